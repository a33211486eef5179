// ssm_norm.hip -- ssm_rms_norm of include/ssm_block.h: h = x + residual, y = (h * weight) / rms(h), in the io dtype or in
// 8 bits with a scale per row.
//
// One pass over the data: a row stays in the registers of the threads that share it (P pieces of 8 values each) from its
// loads to its stores, so that every value is read and written once.  The call is bound by memory for many rows and by
// its latency (a load, one reduction, a store) for few.  The sum of h^2 and the largest |h * weight| go through one
// reduction: r > 0, and rounding keeps order, so max |(h * weight) * r| is exactly (max |h * weight|) * r.
//
// Threads to a row: one for 8 values up to 8192 of them, which makes the chain from the first load to the last store short;
// it is also the faster form for many rows (two pieces to a thread and half the threads, us: 2560 values, 1 row 2.5 against
// 2.2, 2048 rows 9.0 against 7.9; 4096, 1024 rows 7.8 against 6.7; 8192, 2048 rows 27.9 against 25.4).  Up to 128 values 16
// threads, so that a wave has four rows (100000 rows of 128: 18 us, 25 with a wave for each).  A workgroup takes rows in turn
// and loads the next one before it reduces this one.  32768 rows of 4096, bf16 with residual to e4m3: 162 us, 5.8 TB/s,
// more than a copy reaches.
#include "ssm_block.h"

namespace ssm {
namespace block {
namespace {

struct NormArgs {
  Rows x, res, res_out, out;
  const float* w;
  float* scale;
  int64_t T;
  int W;
  float eps;
};

enum { NO_RES = 0, IO_RES = 1, F32_RES = 2 };

// Eight values as they lie in memory.
template <typename IO>
struct Piece {
  u32x4 v[sizeof(IO) / 2];
  __device__ __forceinline__ void load(const char* p) {
#pragma unroll
    for (unsigned i = 0; i < sizeof(IO) / 2; ++i) v[i] = reinterpret_cast<const u32x4*>(p)[i];
  }
  __device__ __forceinline__ float operator[](int i) const {
    if constexpr (sizeof(IO) == 4)
      return __uint_as_float(v[i / 4][i % 4]);
    else
      return __uint_as_float(i % 2 ? v[0][i / 2] & 0xFFFF0000u : v[0][i / 2] << 16);
  }
};

template <typename IO>
__device__ __forceinline__ void store8(char* p, const float (&y)[8]) {
  if constexpr (sizeof(IO) == 4) {
    reinterpret_cast<f32x4*>(p)[0] = f32x4{y[0], y[1], y[2], y[3]};
    reinterpret_cast<f32x4*>(p)[1] = f32x4{y[4], y[5], y[6], y[7]};
  } else {
    *reinterpret_cast<u32x4*>(p) =
        u32x4{pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7])};
  }
}

// Magnitudes of at most 448 and a few roundings of that, far from the 464 where the next code would begin: nothing to clamp, which
// would make a number of a NaN.
__device__ __forceinline__ unsigned codes4(float a, float b, float c, float d) {
  const int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (unsigned)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}

// 448 / x in fp64, x > 0: the reciprocal instruction and two steps of Newton's, each of which squares what is missing.
__device__ __forceinline__ double top_over(double x) {
  double y = __builtin_amdgcn_rcp(x);
  y = fma(fma(-x, y, 1.0), y, y);
  y = fma(fma(-x, y, 1.0), y, y);
  return 448.0 * y;
}

// TPR threads to a row, P pieces of 8 values to a thread; workgroups of max(256, TPR) threads.
template <typename IO, int RES, bool Q8, int TPR, int P>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void rms_rows(const NormArgs a) {
  using R = typename std::conditional<RES == F32_RES, float, IO>::type;
  constexpr int RPB = TPR < 256 ? 256 / TPR : 1, NW = TPR < 64 ? 1 : TPR / 64;
  constexpr bool AHEAD = P <= 2;  // more pieces leave no registers for the next row
  // h * weight: of 8-bit rows in fp64, so that a code is that of the definition (of 134 million none was another, 58 in fp32), where
  // the registers allow (32768 values: 138 us for 1024 rows so, 84 in fp32).  It costs what it costs, us in fp64 and in fp32:
  // 32768 rows without a residual of 1024 39.3, 30.5; of 2048 49.7, 40.9; of 2560 102, 81; of 4096 112, 90; with one of 1024
  // 47.5, 45.0; of 4096 165.8, 164.8; 16384 of 8192 178, 165; one row of 4096 2.7, 2.5.
  using Max = typename std::conditional<Q8 && P == 1, double, float>::type;
  __shared__ float red[2][NW];
  __shared__ Max red_max[2][Q8 ? NW : 1];
  const int tid = threadIdx.x % TPR;
  const int64_t step = (int64_t)gridDim.x * RPB;
  int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;

  bool in[P];
  float w[P][8];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    in[p] = (p * TPR + tid) * 8 < a.W;
    if (AHEAD && in[p]) {
      const float* wp = a.w + (p * TPR + tid) * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i) w[p][i] = wp[i];
    }
  }
  Piece<IO> x[P];
  Piece<R> s[P];
  const auto load = [&](int64_t r) {
#pragma unroll
    for (int p = 0; p < P; ++p)
      if (in[p]) {
        const int64_t e = (p * TPR + tid) * 8;
        x[p].load(a.x.p + r * a.x.stride + e * sizeof(IO));
        if constexpr (RES != NO_RES) s[p].load(a.res.p + r * a.res.stride + e * sizeof(R));
      }
  };
  if (row < a.T) load(row);
  for (int par = 0; row < a.T; row += step, par ^= 1) {
    float h[P][8], ss = 0.0f;
    Max z[P][8], mx = 0;
    if (!AHEAD && row >= step) load(row);  // the first was loaded above
#pragma unroll
    for (int p = 0; p < P; ++p) {
      if (!in[p]) continue;
      const int64_t e = (p * TPR + tid) * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        h[p][i] = x[p][i];
        if constexpr (RES != NO_RES) h[p][i] += s[p][i];
      }
      if constexpr (RES != NO_RES) {
        if constexpr (sizeof(R) == 2) {  // the norm is of the stream as it is stored
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            const unsigned b = pack_bf16(h[p][i], h[p][i + 1]);
            h[p][i] = __uint_as_float(b << 16), h[p][i + 1] = __uint_as_float(b & 0xFFFF0000u);
          }
        }
        store8<R>(a.res_out.p + row * a.res_out.stride + e * sizeof(R), h[p]);
      }
      if constexpr (!AHEAD) {
        const float* wp = a.w + e;
#pragma unroll
        for (int i = 0; i < 8; ++i) w[p][i] = wp[i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        ss = fmaf(h[p][i], h[p][i], ss);
        z[p][i] = (Max)h[p][i] * (Max)w[p][i];
        if constexpr (Q8) mx = fmax(mx, fabs(z[p][i]));
      }
    }
    if (AHEAD && row + step < a.T) load(row + step);
#pragma unroll
    for (int off = TPR < 64 ? TPR / 2 : 32; off >= 1; off >>= 1) {
      ss += __shfl_xor(ss, off, 64);
      if constexpr (Q8) mx = fmax(mx, __shfl_xor(mx, off, 64));
    }
    if constexpr (NW > 1) {  // rows alternate between two buffers: one barrier a row
      if (tid % 64 == 0) {
        red[par][tid / 64] = ss;
        if constexpr (Q8) red_max[par][tid / 64] = mx;
      }
      __syncthreads();
      ss = red[par][0];
      if constexpr (Q8) mx = red_max[par][0];
#pragma unroll
      for (int i = 1; i < NW; ++i) {
        ss += red[par][i];
        if constexpr (Q8) mx = fmax(mx, red_max[par][i]);
      }
    }
    float r = __builtin_amdgcn_rsqf(ss / (float)a.W + a.eps);
    Max m = 0;
    if constexpr (Q8) {
      const float amax = (float)(mx * (Max)r);
      const bool live = !(amax < 0x1p-100f);  // a row with a NaN or an infinity, whose r is NaN or 0, has a scale of NaN
      if (tid == 0) a.scale[row] = live ? amax * (1.0f / 448.0f) : 0.0f;
      // A code is h * weight over the row's largest, r over r: of r its power of two is enough, which rounds nothing (fp64: none).
      if constexpr (sizeof(Max) == 8) {
        m = live ? top_over(mx) : 0.0;
      } else {
        r = __uint_as_float(__float_as_uint(r) & 0x7F800000u);
        m = live ? 448.0f / (mx * r) : 0.0f;
      }
    }
#pragma unroll
    for (int p = 0; p < P; ++p) {
      if (!in[p]) continue;
      const int64_t e = (p * TPR + tid) * 8;
      float y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if constexpr (!Q8)
          y[i] = z[p][i] * r;
        else if constexpr (sizeof(Max) == 8)
          y[i] = (float)(z[p][i] * m);
        else
          y[i] = z[p][i] * r * m;
      }
      if constexpr (Q8)
        *reinterpret_cast<u32x2*>(a.out.p + row * a.out.stride + e) =
            u32x2{codes4(y[0], y[1], y[2], y[3]), codes4(y[4], y[5], y[6], y[7])};
      else
        store8<IO>(a.out.p + row * a.out.stride + e * sizeof(IO), y);
    }
  }
}

template <typename IO, int RES, bool Q8, int TPR, int P>
hipError_t launch(const NormArgs& a, hipStream_t s) {
  constexpr int RPB = TPR < 256 ? 256 / TPR : 1, TPB = TPR < 256 ? 256 : TPR;
  // 2048 threads to a CU; of 512 for many rows half as many, whose rows are fewer places of memory at once; of 256 to 8 bits the
  // registers leave room for 1536, and some of 2048 would wait for the others' end.  Many begin at 2048 rows; us with 2048
  // threads and with fewer, bf16, by rows:
  //   4096 with a residual to e4m3   1000 7.7, 7.3   2000 12.3, 11.5   2500 14.0, 13.6   32768 170, 165
  //   4096 with a residual to bf16   1000 6.5, 6.8   2000 10.7, 10.9   2500 14.8, 14.2   32768 209, 190
  //   4096 without one to bf16       2048 7.2, 7.2   3000 8.9, 9.4     8192 25.4, 24.6   32768 99, 90
  //   1024 with a residual to e4m3   1000 3.8, 3.8   2048 5.3, 5.3     4096 9.1, 7.9     32768 57, 48
  constexpr int MANY = TPB == 512 ? 1024 : TPB == 256 && Q8 ? 1536 : 2048;
  const int64_t want = (a.T + RPB - 1) / RPB, most = 256 * ((a.T >= 2048 ? MANY : 2048) / TPB);
  rms_rows<IO, RES, Q8, TPR, P><<<dim3((unsigned)(want < most ? want : most)), dim3(TPB), 0, s>>>(a);
  return hipGetLastError();
}

template <typename IO, int RES, bool Q8>
hipError_t launch_width(const NormArgs& a, hipStream_t s) {
  if (a.W <= 128) return launch<IO, RES, Q8, 16, 1>(a, s);
  if (a.W <= 512) return launch<IO, RES, Q8, 64, 1>(a, s);
  if (a.W <= 2048) return launch<IO, RES, Q8, 256, 1>(a, s);
  if (a.W <= 4096) return launch<IO, RES, Q8, 512, 1>(a, s);
  if (a.W <= 8192) return launch<IO, RES, Q8, 1024, 1>(a, s);
  if (a.W <= 16384) return launch<IO, RES, Q8, 1024, 2>(a, s);
  return launch<IO, RES, Q8, 1024, 4>(a, s);
}

template <typename IO>
hipError_t launch_norm(const NormArgs& a, int res, bool q8, hipStream_t s) {
  if (res == NO_RES) return q8 ? launch_width<IO, NO_RES, true>(a, s) : launch_width<IO, NO_RES, false>(a, s);
  if (res == IO_RES) return q8 ? launch_width<IO, IO_RES, true>(a, s) : launch_width<IO, IO_RES, false>(a, s);
  if constexpr (sizeof(IO) == 2)
    return q8 ? launch_width<IO, F32_RES, true>(a, s) : launch_width<IO, F32_RES, false>(a, s);
  return hipErrorInvalidValue;
}

}  // namespace
}  // namespace block
}  // namespace ssm

extern "C" int ssm_rms_norm(int64_t tokens, int64_t width, int32_t io_dtype, int32_t residual_dtype, int32_t out_dtype,
                            float eps, const ssm_rows* x, const float* weight, const ssm_rows* residual,
                            const ssm_rows* residual_out, const ssm_rows* out, float* scale, void* stream) {
  using namespace ssm::block;
  if (tokens < 0 || tokens > INT32_MAX || width < 8 || width > SSM_NORM_MAX_WIDTH || width % 8) return SSM_ERR_SHAPE;
  if (!(eps >= 0x1p-126f) || !isfinite(eps)) return SSM_ERR_SHAPE;  // rsq takes no subnormal
  if (io_dtype != SSM_F32 && io_dtype != SSM_BF16) return SSM_ERR_DTYPE;
  if (out_dtype != io_dtype && out_dtype != SSM_E4M3) return SSM_ERR_DTYPE;
  if (residual && residual_dtype != io_dtype && residual_dtype != SSM_F32) return SSM_ERR_DTYPE;
  const bool q8 = out_dtype == SSM_E4M3;
  if (tokens == 0) return SSM_OK;  // its tensors have no addresses
  if ((residual == nullptr) != (residual_out == nullptr) || q8 != (scale != nullptr)) return SSM_ERR_NULL;
  const int64_t T = tokens, W = width, es = size_of(io_dtype), rs = size_of(residual_dtype), os = size_of(out_dtype);
  if (!weight) return SSM_ERR_NULL;
  if (const int st = check_rows(x, es, 16)) return st;
  if (const int st = check_rows(out, os, q8 ? 8 : 16)) return st;
  if (residual) {
    if (const int st = check_rows(residual, rs, 16)) return st;
    if (const int st = check_rows(residual_out, rs, 16)) return st;
  }
  if (!aligned(weight, 16) || (q8 && !aligned(scale, 4))) return SSM_ERR_ALIGN;
  const Span sw = span(weight, W * 4), ss = span(scale, q8 ? T * 4 : 0);
  const auto clear = [&](const ssm_rows* o, int64_t e) {  // of the weight and the scales
    const Span so = rows_span(o, T, W, e);
    return writable(o, T, W) && !overlaps(so, sw) && !overlaps(so, ss);
  };
  if (!clear(out, os) || overlaps(ss, sw) || overlaps(ss, rows_span(x, T, W, es))) return SSM_ERR_ALIAS;
  if (!(same_rows(out, x) && !q8) && rows_overlap(out, W, os, x, W, es, T)) return SSM_ERR_ALIAS;
  if (residual) {
    if (!clear(residual_out, rs) || overlaps(ss, rows_span(residual, T, W, rs))) return SSM_ERR_ALIAS;
    if (rows_overlap(residual_out, W, rs, x, W, es, T) || rows_overlap(residual_out, W, rs, out, W, os, T) ||
        rows_overlap(residual, W, rs, out, W, os, T))
      return SSM_ERR_ALIAS;
    if (!same_rows(residual_out, residual) && rows_overlap(residual_out, W, rs, residual, W, rs, T)) return SSM_ERR_ALIAS;
  }
  NormArgs a = {};
  a.x = rows_of(x, es);
  a.res = rows_of(residual, rs);
  a.res_out = rows_of(residual_out, rs);
  a.out = rows_of(out, os);
  a.w = weight;
  a.scale = scale;
  a.T = T;
  a.W = (int)W;
  a.eps = eps;
  const int res = !residual ? NO_RES : residual_dtype == io_dtype ? IO_RES : F32_RES;
  const hipStream_t s = ready(stream);
  const hipError_t e = io_dtype == SSM_BF16 ? launch_norm<ssm::bf16_t>(a, res, q8, s) : launch_norm<float>(a, res, q8, s);
  return e == hipSuccess ? SSM_OK : SSM_ERR_LAUNCH;
}
