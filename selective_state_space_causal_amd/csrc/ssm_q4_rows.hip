// ssm_q4_rows.hip -- ssm_q4_linear of include/ssm_block.h for up to 16 tokens: bound by reading the weight once.
//
// A wave takes 16 rows of the weight by 512 columns at a time: four loads of 1 KB and one of 256 bytes, each in one piece, and
// the tokens' own values from the caches.  The products run on the matrix cores (16 x 16 outputs: the 16 rows, up to 16
// tokens), bf16 and fp32 tokens with the weights widened to bf16 (one conversion for two of them), e4m3 tokens with the codes
// as they are.  Fewer than 16 tokens leave part of a product idle, which costs nothing here: at 5 TB/s a SIMD has 113 cycles
// for 512 weights, of which bf16 uses 32 (products 16, conversions 16).  The waves of a workgroup share a tile's columns and
// join their sums in LDS, in order.
#include "ssm_q4_linear.h"

namespace ssm {
namespace block {
namespace {

constexpr int WAVES = 8;

template <int X, typename OUT>
__global__ __launch_bounds__(64 * WAVES) void q4_rows(const LinearArgs a, int split) {
  __shared__ float part[WAVES][16][17];
  const int wave = threadIdx.x / 64, lane = threadIdx.x % 64, n = lane % 16, q = lane / 16;
  const int per = WAVES / split;  // row tiles of a workgroup
  const int64_t mt = (int64_t)blockIdx.x * per + wave / split;
  f32x4 acc = {0, 0, 0, 0};
  if (mt < a.mt) {
    const bool live = n < a.T;  // this lane's token
    const char* xp = a.x.p + n * a.x.stride;
    for (int64_t s = wave % split; s < a.k4; s += split) {
      const char* cp = a.codes + ((mt * a.kt + s * 4) * 64 + lane) * 16;
      u32x4 c[4];
#pragma unroll
      for (int b = 0; b < 4; ++b) c[b] = s * 4 + b < a.kt ? *reinterpret_cast<const u32x4*>(cp + b * 1024) : u32x4{0, 0, 0, 0};
      const unsigned scales = *reinterpret_cast<const unsigned*>(a.scales + ((mt * a.k4 + s) * 64 + lane) * 4);
      if constexpr (X == X_E4M3) {
        u32x4 x[4][2];
#pragma unroll
        for (int b = 0; b < 4; ++b)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int64_t k = s * 512 + b * 128 + h * 64 + q * 16;
            x[b][h] = u32x4{0, 0, 0, 0};
            if (live && k < a.K) x[b][h] = *reinterpret_cast<const u32x4*>(xp + k);
          }
        const auto product = [&](int b, auto sel) {
          const i32x8 xv = __builtin_bit_cast(i32x8, __builtin_shufflevector(x[b][0], x[b][1], 0, 1, 2, 3, 4, 5, 6, 7));
          const i32x8 wv = {(int)c[b][0], (int)c[b][1], (int)c[b][2], (int)c[b][3], 0, 0, 0, 0};
          acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(xv, wv, acc, 0, 4, 0, 0x7F7F7F7F, decltype(sel)::value, (int)scales);
        };
        product(0, std::integral_constant<int, 0>());
        product(1, std::integral_constant<int, 1>());
        product(2, std::integral_constant<int, 2>());
        product(3, std::integral_constant<int, 3>());
      } else {
        constexpr int ES = x_size<X>(), N = 2 * ES;  // 16-byte pieces of a lane's 32 columns
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          u32x4 x[N];
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const int64_t k = s * 512 + b * 128 + q * 32 + i * (16 / ES);
            x[i] = u32x4{0, 0, 0, 0};
            if (live && k < a.K) x[i] = *reinterpret_cast<const u32x4*>(xp + k * ES);
          }
          const float scale = pow2(scales >> (8 * b) & 0xFFu);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const bf16x8 w = weights8(c[b][j], scale);
            if constexpr (X == X_BF16) {
              acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x[j]), w, acc, 0, 0, 0);
            } else if constexpr (X == X_WIDE) {
              acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen8(x[j / 2][j % 2 * 2], x[j / 2][j % 2 * 2 + 1]), w, acc, 0, 0, 0);
            } else {
              float f[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(x[2 * j + i / 4][i % 4]);
              bf16x8 p[3];
              three_parts(f, p);
#pragma unroll
              for (int i = 2; i >= 0; --i) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(p[i], w, acc, 0, 0, 0);
            }
          }
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) part[wave][4 * q + i][n] = acc[i];
  __syncthreads();
  for (int o = threadIdx.x; o < per * 16 * (int)a.T; o += 64 * WAVES) {
    const int col = o % (per * 16), t = o / (per * 16);
    const int64_t m = (int64_t)blockIdx.x * per * 16 + col;
    if (m >= a.M) continue;
    float sum = 0.0f;
    for (int i = 0; i < split; ++i) sum += part[col / 16 * split + i][t][col % 16];
    if constexpr (x_scaled<X>()) sum *= a.x_scale[t];
    reinterpret_cast<OUT*>(a.out.p + t * a.out.stride)[m] = from_f32<OUT>(sum);
  }
}

template <int X, typename OUT>
hipError_t launch(const LinearArgs& a, hipStream_t s) {
  int split = 1;
  while (split < WAVES && split < a.k4) split *= 2;
  const int per = WAVES / split;
  const dim3 grid((unsigned)((a.mt + per - 1) / per)), tb(64 * WAVES);
  q4_rows<X, OUT><<<grid, tb, 0, s>>>(a, split);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_q4_rows(const LinearArgs& a, int x_dtype, int out_dtype, hipStream_t s) {
  const bool bf16 = out_dtype == SSM_BF16;
  if (x_dtype == X_F32) return bf16 ? launch<X_F32, bf16_t>(a, s) : launch<X_F32, float>(a, s);
  if (x_dtype == X_BF16) return bf16 ? launch<X_BF16, bf16_t>(a, s) : launch<X_BF16, float>(a, s);
  return bf16 ? launch<X_E4M3, bf16_t>(a, s) : launch<X_WIDE, float>(a, s);
}

}  // namespace block
}  // namespace ssm
