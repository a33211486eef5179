// ssm_q4.hip -- ssm_q4_quantize and ssm_q4_dequantize of include/ssm_block.h: a weight to 4-bit codes with a power of two
// for each 32 values of a row, and back.
//
// A wave takes a tile of 16 rows by 512 columns; a lane holds the four groups of 32 values whose 16 bytes of codes are its
// own in each 16 x 128 tile, so that codes leave (or enter) in pieces of 1 KB and the four scales as one word.  Both are
// bound by memory: 2 (bf16) or 4 bytes a value on one side, 0.53 on the other.  The conversion instruction rounds to
// nearest, ties to the even code, and holds magnitudes at 6.
#include "ssm_block.h"

namespace ssm {
namespace block {
namespace {

struct Q4Args {
  Rows w;
  char* codes;
  char* scales;
  int64_t M, K, kt, k4;  // tiles along K: of 128 and of 512 columns
  int64_t tiles;         // 16 x 512, all
};

constexpr int WAVES = 4;

__device__ __forceinline__ float pow2(unsigned e) { return __uint_as_float(e << 23); }

template <typename IO>
__global__ __launch_bounds__(64 * WAVES) void quantize_tiles(const Q4Args a) {
  const int64_t tile = (int64_t)blockIdx.x * WAVES + threadIdx.x / 64;
  if (tile >= a.tiles) return;
  const int lane = threadIdx.x % 64, n = lane % 16, q = lane / 16;
  const int64_t mt = tile / a.k4, k4 = tile % a.k4, m = mt * 16 + n;
  constexpr int PIECES = sizeof(IO) * 2;  // of 16 bytes, in 32 values
  u32x4 v[4][PIECES];
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    const int64_t k = k4 * 512 + b * 128 + q * 32;
    const char* p = a.w.p + m * a.w.stride + k * (int64_t)sizeof(IO);
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      v[b][i] = u32x4{0, 0, 0, 0};
      if (m < a.M && k + i * (16 / (int)sizeof(IO)) < a.K) v[b][i] = reinterpret_cast<const u32x4*>(p)[i];
    }
  }
  unsigned scales = 0;
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    float x[32], amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      if constexpr (sizeof(IO) == 2) {
        const unsigned d = v[b][i / 8][i % 8 / 2];
        x[i] = __uint_as_float(i % 2 ? d & 0xFFFF0000u : d << 16);
      } else {
        x[i] = __uint_as_float(v[b][i / 4][i % 4]);
      }
      amax = fmaxf(amax, fabsf(x[i]));
    }
    const bool live = amax >= 0x1p-100f;
    const unsigned n2 = ((__float_as_uint(amax) + 0x200000u) >> 23) - 2;
    const unsigned e = live ? min(n2, 252u) : 127u;
    scales |= e << (8 * b);
    u32x4 c;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float* y = x + 8 * j;
      unsigned d = 0;
      d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, y[0], y[1], pow2(e), 0);
      d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, y[2], y[3], pow2(e), 1);
      d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, y[4], y[5], pow2(e), 2);
      d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, y[6], y[7], pow2(e), 3);
      c[j] = live ? d : 0u;
    }
    if (k4 * 4 + b < a.kt) *reinterpret_cast<u32x4*>(a.codes + ((mt * a.kt + k4 * 4 + b) * 64 + lane) * 16) = c;
  }
  *reinterpret_cast<unsigned*>(a.scales + (tile * 64 + lane) * 4) = scales;
}

template <typename IO>
__global__ __launch_bounds__(64 * WAVES) void dequantize_tiles(const Q4Args a) {
  const int64_t tile = (int64_t)blockIdx.x * WAVES + threadIdx.x / 64;
  if (tile >= a.tiles) return;
  const int lane = threadIdx.x % 64, n = lane % 16, q = lane / 16;
  const int64_t mt = tile / a.k4, k4 = tile % a.k4, m = mt * 16 + n;
  const unsigned scales = *reinterpret_cast<const unsigned*>(a.scales + (tile * 64 + lane) * 4);
  u32x4 c[4];
#pragma unroll
  for (int b = 0; b < 4; ++b)
    if (k4 * 4 + b < a.kt) c[b] = *reinterpret_cast<const u32x4*>(a.codes + ((mt * a.kt + k4 * 4 + b) * 64 + lane) * 16);
  if (m >= a.M) return;
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    const int64_t k = k4 * 512 + b * 128 + q * 32;
    char* p = a.w.p + m * a.w.stride + k * (int64_t)sizeof(IO);
    const float s = pow2(scales >> (8 * b) & 0xFFu);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (k + 8 * j >= a.K) continue;
      if constexpr (sizeof(IO) == 2) {
        const auto two = [](auto v) { return __builtin_bit_cast(unsigned, v); };
        reinterpret_cast<u32x4*>(p)[j] = u32x4{two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[b][j], s, 0)),
                                               two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[b][j], s, 1)),
                                               two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[b][j], s, 2)),
                                               two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[b][j], s, 3))};
      } else {
        const auto v0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[b][j], s, 0), v1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[b][j], s, 1),
                   v2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[b][j], s, 2), v3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[b][j], s, 3);
        reinterpret_cast<f32x4*>(p)[2 * j] = f32x4{v0[0], v0[1], v1[0], v1[1]};
        reinterpret_cast<f32x4*>(p)[2 * j + 1] = f32x4{v2[0], v2[1], v3[0], v3[1]};
      }
    }
  }
}

// The checks of both; writes: whether the weight's codes and scales are the output.
int run(int32_t io_dtype, const ssm_rows* w, const ssm_q4_weight* q, bool writes, void* stream) {
  if (io_dtype != SSM_F32 && io_dtype != SSM_BF16) return SSM_ERR_DTYPE;
  if (const int st = check_q4(q)) return st;
  const int64_t es = size_of(io_dtype), M = q->out_features, K = q->in_features;
  if (const int st = check_rows(w, es, 16)) return st;
  const Span sw = rows_span(w, M, K, es), sc = codes_span(q), ss = scales_span(q);
  if (overlaps(sw, sc) || overlaps(sw, ss) || (writes && overlaps(sc, ss)) || (!writes && !writable(w, M, K))) return SSM_ERR_ALIAS;
  Q4Args a;
  a.w = rows_of(w, es);
  a.codes = static_cast<char*>(q->codes);
  a.scales = static_cast<char*>(q->scales);
  a.M = M;
  a.K = K;
  a.kt = (K + 127) / 128;
  a.k4 = (K + 511) / 512;
  a.tiles = (M + 15) / 16 * a.k4;  // at most 2^27
  const dim3 grid((unsigned)((a.tiles + WAVES - 1) / WAVES)), tb(64 * WAVES);
  const hipStream_t s = ready(stream);
  if (writes) {
    if (io_dtype == SSM_BF16) quantize_tiles<ssm::bf16_t><<<grid, tb, 0, s>>>(a);
    else quantize_tiles<float><<<grid, tb, 0, s>>>(a);
  } else {
    if (io_dtype == SSM_BF16) dequantize_tiles<ssm::bf16_t><<<grid, tb, 0, s>>>(a);
    else dequantize_tiles<float><<<grid, tb, 0, s>>>(a);
  }
  return hipGetLastError() == hipSuccess ? SSM_OK : SSM_ERR_LAUNCH;
}

}  // namespace
}  // namespace block
}  // namespace ssm

extern "C" {

size_t ssm_q4_codes_bytes(int64_t out_features, int64_t in_features) {
  return ssm::block::q4_sizes(out_features, in_features) ? (size_t)ssm::block::q4_codes_bytes(out_features, in_features) : 0;
}

size_t ssm_q4_scales_bytes(int64_t out_features, int64_t in_features) {
  return ssm::block::q4_sizes(out_features, in_features) ? (size_t)ssm::block::q4_scales_bytes(out_features, in_features) : 0;
}

int ssm_q4_quantize(int32_t io_dtype, const ssm_rows* w, const ssm_q4_weight* q, void* stream) {
  return ssm::block::run(io_dtype, w, q, true, stream);
}

int ssm_q4_dequantize(int32_t io_dtype, const ssm_q4_weight* q, const ssm_rows* w, void* stream) {
  return ssm::block::run(io_dtype, w, q, false, stream);
}

}  // extern "C"
