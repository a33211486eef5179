// ssm_q4_linear.h -- what ssm_q4_linear's kernels (ssm_q4_rows.hip, ssm_q4_tiles.hip) share.
#pragma once
#include "ssm_block.h"

namespace ssm {
namespace block {

typedef int i32x8 __attribute__((ext_vector_type(8)));

struct LinearArgs {
  Rows x, out;
  const char* codes;
  const char* scales;
  const float* x_scale;  // e4m3 tokens
  float* partial;        // [splits, T, Mp] sums of parts of K
  int64_t Mp;            // M, a multiple of 4
  bool wide;             // output rows are aligned to 16 bytes
  int64_t T, M, K, kt, k4;  // tiles along K: of 128 and of 512 columns
  int64_t mt;               // tiles of 16 rows
};

// How tokens are multiplied.  e4m3 tokens go into the instruction that takes codes as they are (X_E4M3); for an output in fp32
// they are widened to bf16 (X_WIDE): that instruction aligns the products of eight columns to the largest of them and keeps
// 2^-13 of it, which is far below a bf16 output's own rounding (4.5e-6 of a result of 1552 columns, against 2^-9), and not
// what an fp32 output is asked for.
enum { X_F32 = SSM_F32, X_BF16 = SSM_BF16, X_E4M3 = SSM_E4M3, X_WIDE = 3 };

template <int X>
constexpr int x_size() {  // bytes of a token's value in memory
  return X == X_F32 ? 4 : X == X_BF16 ? 2 : 1;
}
template <int X>
constexpr bool x_scaled() {
  return X == X_E4M3 || X == X_WIDE;
}

__device__ __forceinline__ float pow2(unsigned e) { return __uint_as_float(e << 23); }

// Eight codes times s in bf16, exactly.
__device__ __forceinline__ bf16x8 weights8(unsigned c, float s) {
  const auto two = [](auto v) { return __builtin_bit_cast(unsigned, v); };
  return __builtin_bit_cast(bf16x8, u32x4{two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 0)),
                                          two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 1)),
                                          two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 2)),
                                          two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 3))});
}

// Eight e4m3 values in bf16, exactly.
__device__ __forceinline__ bf16x8 widen8(unsigned lo, unsigned hi) {
  const auto two = [](auto v) { return __builtin_bit_cast(unsigned, v); };
  return __builtin_bit_cast(bf16x8, u32x4{two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false)),
                                          two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true)),
                                          two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false)),
                                          two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true))});
}

// x = p[0] + p[1] + p[2], bf16 each, to 2^-27 of x: a part is rounded to nearest, so what it leaves is at most 2^-9 of it, and
// exact in fp32.
__device__ __forceinline__ void three_parts(const float (&x)[8], bf16x8 (&p)[3]) {
  float r[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = x[i];
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[i] = pack_bf16(r[2 * i], r[2 * i + 1]);
      r[2 * i] -= __uint_as_float(w[i] << 16);
      r[2 * i + 1] -= __uint_as_float(w[i] & 0xFFFF0000u);
    }
    p[k] = __builtin_bit_cast(bf16x8, w);
  }
}

// Few tokens: ssm_q4_rows.hip.  Any number: ssm_q4_tiles.hip.
constexpr int64_t ROWS_MAX_TOKENS = 16;
hipError_t launch_q4_rows(const LinearArgs& a, int x_dtype, int out_dtype, hipStream_t s);
hipError_t launch_q4_tiles(const LinearArgs& a, int x_dtype, int out_dtype, hipStream_t s);
int q4_tiles_splits(int64_t T, int x_dtype, int64_t M, int64_t K);

}  // namespace block
}  // namespace ssm
