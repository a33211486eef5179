// ssm_q4_rows.hip -- ssm_q4_linear of include/ssm_block.h for up to four tokens (one in fp32): bound by reading the weight once.
//
// A wave takes NT tiles of 16 rows by some blocks of 128 columns: a load of 1 KB for each, in one piece, four blocks on their way at
// once, and the tokens' own values from the caches.  bf16 and e4m3 tokens are multiplied on the matrix cores (16 x 16 outputs:
// 16 rows, up to 16 tokens); that most of a product is idle costs nothing: at 5 TB/s a SIMD has 113 cycles for 512 weights, of
// which bf16 uses 32 (products 16, conversions 16).  An fp32 token would have to be split in three there by every lane, so its
// products are fp32 multiply-adds: a lane has one row and a quarter of the columns.  The waves of a workgroup share a tile's
// columns and join their sums in LDS, in order.
#include "ssm_q4_linear.h"

namespace ssm {
namespace block {
namespace {

template <int X, int NT, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void q4_rows(const LinearArgs a, int split) {
  constexpr int ES = x_size<X>(), N = 2 * ES;  // 16-byte pieces of a group's 32 columns of a token
  constexpr int AHEAD = X == X_F32 ? 2 : 4;    // blocks on their way at once
  __shared__ float part[WAVES][4][NT * 16 + 1];
  const int wave = threadIdx.x / 64, lane = threadIdx.x % 64, n = lane % 16, q = lane / 16;
  const int per = WAVES / split, share = wave % split;  // groups of NT tiles of a workgroup
  const int64_t mt = ((int64_t)blockIdx.x * per + wave / split) * NT;
  const int lo = (int)(a.kt * share / split), hi = mt < a.mt ? (int)(a.kt * (share + 1) / split) : lo;
  const char* cp[NT];
  const char* sp[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int64_t m = mt + i < a.mt ? mt + i : a.mt - 1;  // past the last: any, not stored
    cp[i] = a.codes + (m * a.kt * 64 + lane) * 16;
    sp[i] = a.scales + (m * a.k4 * 64 + lane) * 4;
  }
  f32x4 acc[NT] = {};  // on the matrix cores: token i of lane n's row, in the first quarter of the wave
  float sum[NT] = {};  // fp32: of lane n's row and the groups q
  const auto blocks = [&](int kb, auto count) {
    constexpr int B = decltype(count)::value;
    u32x4 c[B][NT], x[B][N];
    unsigned s[NT], s_next[NT];  // a byte for each of four blocks
    const int from = kb & 3, next = from + B > 4;
    // in the order of their use: loads come back in order
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      s[i] = *reinterpret_cast<const unsigned*>(sp[i] + (int64_t)(kb >> 2) * 256);
      s_next[i] = *reinterpret_cast<const unsigned*>(sp[i] + (int64_t)((kb >> 2) + next) * 256);
    }
#pragma unroll
    for (int b = 0; b < B; ++b) {
#pragma unroll
      for (int i = 0; i < NT; ++i) c[b][i] = *reinterpret_cast<const u32x4*>(cp[i] + (int64_t)(kb + b) * 1024);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int64_t k = (int64_t)(kb + b) * 128 + q * 32 + i * (16 / ES);
        // token n / 4 in lanes 0, 4, 8 and 12: its outputs are the first of a lane's four; fp32: the one token in all lanes
        const bool live = X == X_F32 || (n % 4 == 0 && n / 4 < a.T);
        x[b][i] = u32x4{0, 0, 0, 0};
        if (live && k < a.K) x[b][i] = *reinterpret_cast<const u32x4*>(a.x.p + (X == X_F32 ? 0 : n / 4 * a.x.stride) + k * ES);
      }
    }
    const auto product = [&](auto block) {
      constexpr int b = decltype(block)::value;
      if constexpr (X == X_F32) {
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float e = pow2(s[i] >> (8 * b) & 0xFFu);
            const unsigned u = c[b][i][j];
            const auto w0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(u, e, 0), w1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(u, e, 1),
                       w2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(u, e, 2), w3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(u, e, 3);
            const float w[8] = {w0[0], w0[1], w1[0], w1[1], w2[0], w2[1], w3[0], w3[1]};
#pragma unroll
            for (int v = 0; v < 8; ++v) sum[i] = fmaf(w[v], __uint_as_float(x[b][2 * j + v / 4][v % 4]), sum[i]);
          }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const bf16x8 xv = X == X_BF16 ? __builtin_bit_cast(bf16x8, x[b][j % N])
                                        : widen8(x[b][j / 2][j % 2 * 2], x[b][j / 2][j % 2 * 2 + 1]);
#pragma unroll
          for (int i = 0; i < NT; ++i)
            acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xv, weights8(c[b][i][j], pow2(s[i] >> (8 * b) & 0xFFu)), acc[i], 0, 0, 0);
        }
      }
    };
#pragma unroll
    for (int i = 0; i < NT; ++i) s[i] = __builtin_amdgcn_alignbyte(s_next[i], s[i], from);  // of blocks kb .. kb + B - 1
    product(std::integral_constant<int, 0>());
    if constexpr (B > 1) product(std::integral_constant<int, 1>());
    if constexpr (B > 2) product(std::integral_constant<int, 2>()), product(std::integral_constant<int, 3>());
  };
  int kb = lo;
  for (; kb + AHEAD <= hi; kb += AHEAD) blocks(kb, std::integral_constant<int, AHEAD>());
  if constexpr (AHEAD == 4)
    if (kb + 2 <= hi) blocks(kb, std::integral_constant<int, 2>()), kb += 2;
  if (kb < hi) blocks(kb, std::integral_constant<int, 1>());
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    if constexpr (X == X_F32) {
      float v = sum[i];
      v += __shfl_xor(v, 16, 64);
      v += __shfl_xor(v, 32, 64);
      if (q == 0) part[wave][0][i * 16 + n] = v;
    } else {
      part[wave][q][i * 16 + n] = acc[i][0];  // row 4 q of the outputs is token q
    }
  }
  __syncthreads();
  const int cols = per * NT * 16;
  for (int o = threadIdx.x; o < cols * (int)a.T; o += 64 * WAVES) {
    const int col = o % cols, t = o / cols, group = col / (NT * 16);
    const int64_t m = (int64_t)blockIdx.x * cols + col;
    if (m >= a.M) continue;
    float v = 0.0f;
    for (int i = 0; i < split; ++i) v += part[group * split + i][t][col % (NT * 16)];
    store_one<X>(a, t, m, v);
  }
}

template <int X, int NT, int WAVES>
hipError_t launch_waves(const LinearArgs& a, hipStream_t s) {
  int split = 1;
  while (split < WAVES && split < a.kt) split *= 2;
  const int64_t per = WAVES / split * NT;
  q4_rows<X, NT, WAVES><<<dim3((unsigned)((a.mt + per - 1) / per)), dim3(64 * WAVES), 0, s>>>(a, split);
  return hipGetLastError();
}

// Waves and rows of a workgroup, one bf16 token by 4096 columns, us: up to 8192 rows eight waves on 16 rows (4096 rows 3.9, four
// waves on 32 5.1; 8192 rows 5.8 and 6.4), which has a wave for each block of columns; past that four waves on 32 rows,
// with less to join (16384 rows 8.4, eight on 16 9.3; 32768 14.4 and 16.0; 65536 by 2560 17.2 and 29.6, 5.2 TB/s).
template <int X>
hipError_t launch(const LinearArgs& a, hipStream_t s) {
  return a.mt <= 512 ? launch_waves<X, 1, 8>(a, s) : launch_waves<X, 2, 4>(a, s);
}

}  // namespace

hipError_t launch_q4_rows(const LinearArgs& a, int x, hipStream_t s) {
  return x == X_F32 ? launch<X_F32>(a, s) : x == X_BF16 ? launch<X_BF16>(a, s) : launch<X_E4M3>(a, s);
}

}  // namespace block
}  // namespace ssm
