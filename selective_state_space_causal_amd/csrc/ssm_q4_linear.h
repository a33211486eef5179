// ssm_q4_linear.h -- what ssm_q4_linear's kernels (ssm_q4_rows.hip, ssm_q4_few.hip, ssm_q4_tiles.hip) share.
#pragma once
#include <type_traits>

#include "ssm_block.h"

#define LDS_PTR(T, p) ((__attribute__((address_space(3))) T*)(p))

namespace ssm {
namespace block {

struct LinearArgs {
  Rows x, out;
  const char* codes;
  const char* scales;
  const float* x_scale;     // e4m3 tokens
  int64_t T, M, K, kt, k4;  // tiles along K: of 128 and of 512 columns
  int64_t mt;               // tiles of 16 rows
  bool out_bf16;
  bool wide;                // output rows are aligned to 16 bytes
};

// Tokens by their type.  e4m3 ones are widened to bf16, which is exact, as the codes are.  (The instruction that takes 8- and 4-bit
// values as they are does not sum in fp32: it aligns the products of eight columns to the largest of them and drops what is
// below 2^-13 of it.  Beside a column of 448 that another one cancels, results of 9.16 came out as 9.63 in bf16.)
enum { X_F32 = SSM_F32, X_BF16 = SSM_BF16, X_E4M3 = SSM_E4M3 };

template <int X>
constexpr int x_size() {  // bytes of a token's value
  return X == X_F32 ? 4 : X == X_BF16 ? 2 : 1;
}
template <int X>
constexpr bool x_scaled() {
  return X == X_E4M3;
}
template <int X>
constexpr int planes() {  // bf16 parts of a value
  return X == X_F32 ? 3 : 1;
}

__device__ __forceinline__ float pow2(unsigned e) { return __uint_as_float(e << 23); }

template <typename V>
__device__ __forceinline__ unsigned two(V v) {
  return __builtin_bit_cast(unsigned, v);
}

// Eight codes times s in bf16, exactly.
__device__ __forceinline__ bf16x8 weights8(unsigned c, float s) {
  return __builtin_bit_cast(bf16x8, u32x4{two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 0)),
                                          two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 1)),
                                          two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 2)),
                                          two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 3))});
}

// Eight e4m3 values in bf16, exactly.
__device__ __forceinline__ bf16x8 widen8(unsigned lo, unsigned hi) {
  return __builtin_bit_cast(bf16x8, u32x4{two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false)),
                                          two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true)),
                                          two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false)),
                                          two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true))});
}

// x = p[0] + p[1] + p[2], bf16 each, exactly, while no part overflows or is subnormal: a part holds 8 of x's 24 bits, rounded to
// nearest, and what it leaves is exact in fp32, at most half of its last place: 16 bits, then 8.
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

// 2 GiB from p on, for loads straight into LDS; every offset is in bounds by construction.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t resource(const char* p) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(p), (short)0, 0x7FFFFFFF, 0x00020000);
}

// Tokens in LDS: rows of 128 columns.  Piece c (16 bytes) of token t lies at place c ^ swap_of(t) of its row, so that 16
// neighbouring rows' pieces c cover all 64 banks.
template <int X>
__device__ __forceinline__ int swap_of(int t) {
  return x_size<X>() == 1 ? (t >> 1) & 7 : t & 15;
}

// Eight of a token's values in LDS, as bf16 (fp32 ones in three parts); `eighth`: which eight of the row's 128.
template <int X>
struct Eight;
template <>
struct Eight<X_BF16> {
  bf16x8 v;
  __device__ __forceinline__ void read(const char* row, int eighth, int swap) {
    v = *reinterpret_cast<const bf16x8*>(row + (eighth ^ swap) * 16);
  }
  __device__ __forceinline__ void parts(bf16x8 (&p)[1]) const { p[0] = v; }
};
template <>
struct Eight<X_E4M3> {
  u32x2 v;
  __device__ __forceinline__ void read(const char* row, int eighth, int swap) {
    v = *reinterpret_cast<const u32x2*>(row + (eighth / 2 ^ swap) * 16 + eighth % 2 * 8);
  }
  __device__ __forceinline__ void parts(bf16x8 (&p)[1]) const { p[0] = widen8(v[0], v[1]); }
};
template <>
struct Eight<X_F32> {
  u32x4 v[2];
  __device__ __forceinline__ void read(const char* row, int eighth, int swap) {
#pragma unroll
    for (int i = 0; i < 2; ++i) v[i] = *reinterpret_cast<const u32x4*>(row + ((2 * eighth + i) ^ swap) * 16);
  }
  __device__ __forceinline__ void parts(bf16x8 (&p)[3]) const {
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(v[i / 4][i % 4]);
    three_parts(f, p);
  }
};

// One output: column m of token t.
template <int X>
__device__ __forceinline__ void store_one(const LinearArgs& a, int64_t t, int64_t m, float sum) {
  if constexpr (x_scaled<X>()) sum *= a.x_scale[t];
  char* const p = a.out.p + t * a.out.stride;
  if (a.out_bf16)
    reinterpret_cast<bf16_t*>(p)[m] = from_f32<bf16_t>(sum);
  else
    reinterpret_cast<float*>(p)[m] = sum;
}

hipError_t launch_q4_rows(const LinearArgs& a, int x, hipStream_t s);   // rows_takes
hipError_t launch_q4_few(const LinearArgs& a, int x, hipStream_t s);    // few_takes
hipError_t launch_q4_tiles(const LinearArgs& a, int x, hipStream_t s);  // any call
inline bool rows_takes(const LinearArgs& a, int x) { return a.T <= (x == X_F32 ? 1 : 4); }
// Up to 32 tokens, us in ssm_q4_few.hip and in tiles: where a weight's rows fill the CUs with tiles of 32 x 32, those win, since
// the tokens are read once for 32 rows; with bf16 tokens once there are two to a CU.
//   e4m3   32 by 4096 x 4096 5.7, 6.3; 6144 x 4096 10.9, 6.5; 16384 x 4096 20, 9.6; 16 by 4096 x 4096 4.6, 6.2; 6144 x 4096 6.5, 6.3
//   bf16   32 by 4096 x 4096 6.2, 8.0; 8192 x 8192 11.6, 13.6; 10240 x 2560 8.7, 7.4; 16384 x 4096 12.5, 11.7
//   fp32   16 by 8192 x 4096 11.0, 17.9; 65536 x 2560 41, 51
inline bool few_takes(const LinearArgs& a, int x) {
  return x == X_F32 ? a.T <= 16 : a.T <= 32 && a.mt <= (x == X_BF16 ? 512 : 256);
}

}  // namespace block
}  // namespace ssm
