// ssm_q4.hip -- ssm_q4_quantize and ssm_q4_dequantize of include/ssm_block.h: a weight to 4-bit codes with a power of two
// for each 32 values of a row, and back.
//
// A wave takes a tile of 16 rows by 512 columns.  On the weight's side it works in rows: a lane has 8 neighbouring values, four
// lanes a group, and a load or store covers 512 columns of a row in one piece; on the other side codes lie in tiles.  They change
// places in LDS (a quarter of the weight's bytes), where a group's 16 bytes keep together and the 16 groups of a row start on
// different banks.  Both are bound by memory: 2 (bf16) or 4 bytes a value on one side, 0.53 on the other.  (With a lane holding its
// groups' 64 bytes of the weight, loads and stores were pieces of 16 bytes 64 apart: 44 us for 16384 x 4096 either way.)
// The conversion instruction rounds to nearest, ties to the even code, and holds magnitudes at 6.
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

// A tile of codes and scales in LDS, one to a wave.
struct Exchange {
  char codes[16 * 272];   // group (block b, q) of a row: 16 (4 b + q) + 256 bytes of 16 rows and 16 that shift the banks
  unsigned char scales[256];
  __device__ __forceinline__ char* group(int g, int row) { return codes + g * 272 + row * 16; }
};

// What the wave's lanes wrote to LDS is there for all of them (the LDS takes a wave's accesses in order; this holds the compiler).
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
}

// The larger of two values, NaN where one is (fmaxf drops it).
__device__ __forceinline__ float largest(float a, float b) { return __builtin_elementwise_maximum(a, b); }

// The largest of four neighbouring lanes' values, in all of them.
__device__ __forceinline__ float quad_max(float v) {
  // lanes 1 0 3 2, then 2 3 0 1 of each four
  v = largest(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0xB1, 0xF, 0xF, true)));
  return largest(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x4E, 0xF, 0xF, true)));
}

template <typename IO>
__global__ __launch_bounds__(64 * WAVES) void quantize_tiles(const Q4Args a) {
  __shared__ __attribute__((aligned(16))) Exchange exchange[WAVES];
  const int64_t tile = (int64_t)blockIdx.x * WAVES + threadIdx.x / 64;
  if (tile >= a.tiles) return;  // no barrier below: a wave's LDS is its own
  Exchange& x = exchange[threadIdx.x / 64];
  const int lane = threadIdx.x % 64;
  const int64_t mt = tile / a.k4, k4 = tile % a.k4, k = k4 * 512 + lane * 8;
  constexpr int PIECES = sizeof(IO) / 2, ROWS = 16 / PIECES;  // 16-byte pieces of 8 values; rows on their way at once
  for (int r0 = 0; r0 < 16; r0 += ROWS) {
    u32x4 v[ROWS][PIECES];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const int64_t m = mt * 16 + r0 + r;
      const char* p = a.w.p + m * a.w.stride + k * (int64_t)sizeof(IO);
#pragma unroll
      for (int i = 0; i < PIECES; ++i) {
        v[r][i] = u32x4{0, 0, 0, 0};
        if (m < a.M && k < a.K) v[r][i] = reinterpret_cast<const u32x4*>(p)[i];
      }
    }
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      float y[8], amax = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if constexpr (sizeof(IO) == 2)
          y[i] = __uint_as_float(i % 2 ? v[r][0][i / 2] & 0xFFFF0000u : v[r][0][i / 2] << 16);
        else
          y[i] = __uint_as_float(v[r][i / 4][i % 4]);
        amax = largest(amax, fabsf(y[i]));
      }
      amax = quad_max(amax);
      const bool finite = amax < __builtin_inff(), live = finite && amax >= 0x1p-100f;
      const unsigned e = live ? min(((__float_as_uint(amax) + 0x200000u) >> 23) - 2, 252u) : finite ? 127u : 255u;
      unsigned c = 0;
      c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, y[0], y[1], pow2(e), 0);
      c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, y[2], y[3], pow2(e), 1);
      c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, y[4], y[5], pow2(e), 2);
      c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, y[6], y[7], pow2(e), 3);
      const int g = lane / 4;  // 4 b + q
      reinterpret_cast<unsigned*>(x.group(g, r0 + r))[lane % 4] = live ? c : 0u;
      if (lane % 4 == 0) x.scales[(g % 4 * 16 + r0 + r) * 4 + g / 4] = (unsigned char)e;
    }
  }
  wave_sync();
  const int n = lane % 16, q = lane / 16;
#pragma unroll
  for (int b = 0; b < 4; ++b)
    if (k4 * 4 + b < a.kt)
      *reinterpret_cast<u32x4*>(a.codes + ((mt * a.kt + k4 * 4 + b) * 64 + lane) * 16) =
          *reinterpret_cast<const u32x4*>(x.group(4 * b + q, n));
  *reinterpret_cast<unsigned*>(a.scales + (tile * 64 + lane) * 4) = reinterpret_cast<const unsigned*>(x.scales)[lane];
}

template <typename IO>
__global__ __launch_bounds__(64 * WAVES) void dequantize_tiles(const Q4Args a) {
  __shared__ __attribute__((aligned(16))) Exchange exchange[WAVES];
  const int64_t tile = (int64_t)blockIdx.x * WAVES + threadIdx.x / 64;
  if (tile >= a.tiles) return;  // no barrier below: a wave's LDS is its own
  Exchange& x = exchange[threadIdx.x / 64];
  const int lane = threadIdx.x % 64, n = lane % 16, q = lane / 16;
  const int64_t mt = tile / a.k4, k4 = tile % a.k4, k = k4 * 512 + lane * 8;
  u32x4 c[4];
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    c[b] = u32x4{0, 0, 0, 0};
    if (k4 * 4 + b < a.kt) c[b] = *reinterpret_cast<const u32x4*>(a.codes + ((mt * a.kt + k4 * 4 + b) * 64 + lane) * 16);
  }
  reinterpret_cast<unsigned*>(x.scales)[lane] = *reinterpret_cast<const unsigned*>(a.scales + (tile * 64 + lane) * 4);
#pragma unroll
  for (int b = 0; b < 4; ++b) *reinterpret_cast<u32x4*>(x.group(4 * b + q, n)) = c[b];
  wave_sync();
  if (k >= a.K) return;
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    const int64_t m = mt * 16 + r;
    if (m >= a.M) break;
    const int g = lane / 4;
    const unsigned w = reinterpret_cast<const unsigned*>(x.group(g, r))[lane % 4];
    const float s = pow2(x.scales[(g % 4 * 16 + r) * 4 + g / 4]);
    char* p = a.w.p + m * a.w.stride + k * (int64_t)sizeof(IO);
    if constexpr (sizeof(IO) == 2) {
      const auto two = [](auto v) { return __builtin_bit_cast(unsigned, v); };
      *reinterpret_cast<u32x4*>(p) = u32x4{
          two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0)), two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1)),
          two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2)), two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3))};
    } else {
      const auto v0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 0), v1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 1),
                 v2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 2), v3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 3);
      reinterpret_cast<f32x4*>(p)[0] = f32x4{v0[0], v0[1], v1[0], v1[1]};
      reinterpret_cast<f32x4*>(p)[1] = f32x4{v2[0], v2[1], v3[0], v3[1]};
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
