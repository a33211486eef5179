// ssm_q4_few.hip -- ssm_q4_linear of include/ssm_block.h for up to 32 tokens (16 in fp32) and, but for fp32, not too many rows
// (few_takes): bound by reading the weight once and by the tokens' way to every CU.
//
// As in ssm_q4_rows.hip a wave takes NT tiles of 16 rows, and the waves of a workgroup share their columns; here a wave brings the
// tokens of its own columns straight from memory to an LDS ring of its own, in whole lines, and no wave waits for another until
// the sums are joined.  (Read to registers as operands, tokens come in pieces of 16 bytes of 16 rows, a quarter of the lines'
// rate: 16 bf16 tokens by 4096 x 4096 take 6.2 us so and 5.0 through LDS.)
#include "ssm_q4_linear.h"

namespace ssm {
namespace block {
namespace {

constexpr int WAVES = 8;

// NT tiles of 16 rows and TT of 16 tokens to a wave; `split` waves share a tile's columns.
template <int X, int NT, int TT>
__global__ __launch_bounds__(64 * WAVES) void q4_few(const LinearArgs a, int split) {
  constexpr int RB = 128 * x_size<X>(), STAGE = TT * 16 * RB, LOADS = STAGE / 1024;
  constexpr int ST = 128 * 1024 / (WAVES * STAGE) >= 4 ? 4 : 2;  // steps of 128 columns in the ring
  constexpr int RING = ST * STAGE, PART = TT * 16 * (NT * 16 + 1) * 4;
  static_assert(WAVES * RING <= 160 * 1024 && LOADS * (ST - 1) < 64, "");
  __shared__ __attribute__((aligned(16))) char lds[WAVES * (RING > PART ? RING : PART)];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64, n = lane % 16, q = lane / 16;
  const int per = WAVES / split;  // groups of NT tiles of a workgroup
  const int64_t mt = ((int64_t)blockIdx.x * per + wave / split) * NT;
  const int share = wave % split;
  const int lo = (int)(a.kt * share / split), hi = mt < a.mt ? (int)(a.kt * (share + 1) / split) : lo;
  const int whole = (int)(a.K / 128), last = (int)a.T - 1;
  char* const ring = lds + wave * RING;

  const char* cp[NT];
  const char* sp[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int64_t m = mt + i < a.mt ? mt + i : a.mt - 1;  // past the last: any, not stored
    cp[i] = a.codes + (m * a.kt * 64 + lane) * 16;
    sp[i] = a.scales + (m * a.k4 * 64 + lane) * 4;
  }
  u32x4 c[ST][NT];
  unsigned s[ST][NT];
  // Step kb into place p of the ring; its tokens last, so that a wait for all but the later steps' tokens covers it.
  const auto load = [&](int kb, int p) {
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      c[p][i] = *reinterpret_cast<const u32x4*>(cp[i] + (int64_t)kb * 1024);
      s[p][i] = *reinterpret_cast<const uint8_t*>(sp[i] + (int64_t)(kb >> 2) * 256 + (kb & 3));
    }
    __builtin_amdgcn_sched_barrier(0);
    if (kb < whole) {
      const __amdgpu_buffer_rsrc_t r = resource(a.x.p + (int64_t)kb * RB);
#pragma unroll
      for (int i = 0; i < LOADS; ++i) {
        const int at = i * 1024 + lane * 16, t = at / RB;
        const int off = min(t, last) * (int)a.x.stride + ((at % RB / 16) ^ swap_of<X>(t)) * 16;  // below 2^31: 31 rows of 2^23 bytes
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, LDS_PTR(void, ring + p * STAGE + i * 1024), 16, off, 0, 0, 0);
      }
    } else {  // the last step of an odd width: zeros past the last column
#pragma unroll 1
      for (int i = 0; i < LOADS; ++i) {
        const int at = i * 1024 + lane * 16, t = at / RB, piece = (at % RB / 16) ^ swap_of<X>(t);
        const int64_t k = (int64_t)kb * RB + piece * 16;
        u32x4 v = {0, 0, 0, 0};
        if (k < a.K * x_size<X>()) v = *reinterpret_cast<const u32x4*>(a.x.p + min(t, last) * a.x.stride + k);
        *reinterpret_cast<u32x4*>(ring + p * STAGE + at) = v;
      }
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  f32x4 acc[TT][NT] = {};
  const auto multiply = [&](int p) {
    const char* rows = ring + p * STAGE + n * RB;
    const int swap = swap_of<X>(n);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      bf16x8 x[TT][planes<X>()];
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        Eight<X> e;
        e.read(rows + t * 16 * RB, 4 * q + j, swap);
        e.parts(x[t]);
      }
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const bf16x8 w = weights8(c[p][i][j], pow2(s[p][i]));
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
          for (int k = planes<X>() - 1; k >= 0; --k)
            acc[t][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[t][k], w, acc[t][i], 0, 0, 0);
      }
    }
  };
#pragma unroll
  for (int p = 0; p < ST - 1; ++p)
    if (lo + p < hi) load(lo + p, p);
  for (int kb = lo; kb < hi; kb += ST) {
#pragma unroll
    for (int p = 0; p < ST; ++p) {
      if (kb + p >= hi) break;
      const int ahead = kb + p + ST - 1;
      if (ahead < hi) load(ahead, (p + ST - 1) % ST);
      // Its own tokens are there once at most the later steps' are on their way; the end of the columns waits for all.
      if (ahead < hi && ahead < whole)
        __builtin_amdgcn_s_waitcnt(0x0F70 | ((ST - 1) * LOADS & 15) | ((ST - 1) * LOADS >> 4 << 14));
      else
        __builtin_amdgcn_s_waitcnt(0x0F70);
      asm volatile("" ::: "memory");  // no read of the ring moves up
      __builtin_amdgcn_sched_barrier(0);
      multiply(p);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  __syncthreads();  // every wave is done with its ring
  float(*part)[TT * 16][NT * 16 + 1] = reinterpret_cast<float(*)[TT * 16][NT * 16 + 1]>(lds);
#pragma unroll
  for (int t = 0; t < TT; ++t)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) part[wave][t * 16 + 4 * q + i][j * 16 + n] = acc[t][j][i];
  __syncthreads();
  const int cols = per * NT * 16;
  for (int o = threadIdx.x; o < cols * (int)a.T; o += 64 * WAVES) {
    const int col = o % cols, t = o / cols;
    const int64_t m = (int64_t)blockIdx.x * cols + col;
    if (m >= a.M) continue;
    float sum = 0.0f;
    for (int i = 0; i < split; ++i) sum += part[col / (NT * 16) * split + i][t][col % (NT * 16)];
    store_one<X>(a, t, m, sum);
  }
}

template <int X, int NT, int TT>
hipError_t launch_tiles(const LinearArgs& a, hipStream_t s) {
  int split = 1;
  while (split < WAVES && split < a.kt) split *= 2;
  const int64_t per = WAVES / split * NT;
  q4_few<X, NT, TT><<<dim3((unsigned)((a.mt + per - 1) / per)), dim3(64 * WAVES), 0, s>>>(a, split);
  return hipGetLastError();
}

// Rows to a workgroup: as few as fill the CUs once (16 bf16 tokens by 4096 x 4096 with 16, 32 or 64 rows: 5.0, 5.8, 7.9 us).
template <int X, int TT>
hipError_t launch_rows(const LinearArgs& a, hipStream_t s) {
  if constexpr (X == X_F32)
    if (a.mt > 512) return launch_tiles<X, 4, TT>(a, s);
  if constexpr (x_size<X>() > 1)
    if (a.mt > 256) return launch_tiles<X, 2, TT>(a, s);
  return launch_tiles<X, 1, TT>(a, s);
}

template <int X>
hipError_t launch(const LinearArgs& a, hipStream_t s) {
  if constexpr (X != X_F32)
    if (a.T > 16) return launch_rows<X, 2>(a, s);
  return launch_rows<X, 1>(a, s);
}

}  // namespace

hipError_t launch_q4_few(const LinearArgs& a, int x, hipStream_t s) {
  return x == X_F32 ? launch<X_F32>(a, s) : x == X_BF16 ? launch<X_BF16>(a, s) : launch<X_E4M3>(a, s);
}

}  // namespace block
}  // namespace ssm
