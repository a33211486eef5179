// ssm_q4_tiles.hip -- ssm_q4_linear of include/ssm_block.h for any number of tokens.
//
// A workgroup of four waves makes 128 rows of the weight by BT tokens, 128 columns at a step.  The tokens' tile goes through
// one of two LDS buffers while the other is multiplied; the weight goes from memory straight into the operands: a lane loads the
// groups of its own row, 16 bytes each, and widens them to bf16 (bf16 and fp32 tokens) or hands them to the instruction that
// takes codes and scales (e4m3 tokens).  32 x 32 products.  LDS pieces of 16 bytes are exchanged within a token's row so that
// the lanes of a read fall on different banks.  Where there are too few tiles for the CUs, several workgroups share a tile's
// columns, write fp32 sums to the workspace, and a second launch adds them in order.
#include "ssm_q4_linear.h"

namespace ssm {
namespace block {
namespace {

constexpr int BM = 128, THREADS = 256;

// fp32 tokens lie in LDS as three planes of bf16 parts.
template <int X>
constexpr int planes() {
  return X == X_F32 ? 3 : 1;
}
template <int X>
constexpr int row_bytes() {
  return X == X_E4M3 ? 128 : 256;
}

// Place of piece c (16 bytes) of token row t in a plane: 16 neighbouring rows' pieces c cover all 64 banks.
template <int X>
__device__ __forceinline__ int place(int t, int c) {
  if constexpr (X == X_E4M3)
    return t * 128 + ((c ^ ((t >> 1) & 7)) * 16);
  else
    return t * 256 + ((c ^ (t & 15)) * 16);
}

template <int X, int BT, typename OUT>
__global__ __launch_bounds__(THREADS, 2) void q4_tiles(const LinearArgs a, int splits) {
  constexpr int ES = x_size<X>(), PL = planes<X>(), RB = row_bytes<X>(), PLANE = BT * RB, TILE = PLANE * PL;
  constexpr int WT = BT == 128 ? 2 : 1, WM = 4 / WT;      // waves along tokens and along rows
  constexpr int NT = BT / WT / 32, NM = BM / WM / 32;     // a wave's 32 x 32 tiles
  constexpr int PIECES = BT * 128 * ES / 16 / THREADS;    // 16-byte loads of a thread for a step's tokens
  static_assert(PIECES >= 1, "");
  static_assert(2 * TILE <= 160 * 1024, "");
  __shared__ __attribute__((aligned(16))) char lds[2 * TILE];

  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64, l32 = lane % 32, h = lane / 32;
  const int64_t tiles_t = (a.T + BT - 1) / BT;
  const int64_t tile = blockIdx.x, t0 = tile % tiles_t * BT, m0 = tile / tiles_t * BM;
  const int wt = wave % WT * (NT * 32), wm = wave / WT * (NM * 32);
  // this workgroup's share of the steps
  const int64_t k_lo = a.kt * blockIdx.y / splits, k_hi = a.kt * (blockIdx.y + 1) / splits;

  // a lane's rows of the weight
  const char* cp[NM];
  const char* sp[NM];
#pragma unroll
  for (int i = 0; i < NM; ++i) {
    int64_t mt = (m0 + wm + i * 32) / 16 + l32 / 16;
    if (mt >= a.mt) mt = a.mt - 1;  // past the last row: any, not stored
    cp[i] = a.codes + (mt * a.kt * 64 + h * 16 + l32 % 16) * 16;
    sp[i] = a.scales + (mt * a.k4 * 64 + h * 16 + l32 % 16) * 4;
  }

  u32x4 xr[PIECES];
  u32x4 c[2][NM][2];
  unsigned s[2][NM][2];
  const auto load_x = [&](int64_t kb) {
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      const int p = i * THREADS + threadIdx.x, t = p / (8 * ES), at = p % (8 * ES);  // 8 * ES pieces to a token's 128 columns
      const int64_t k = kb * 128 + at * (16 / ES);
      xr[i] = u32x4{0, 0, 0, 0};
      if (t0 + t < a.T && k < a.K) xr[i] = *reinterpret_cast<const u32x4*>(a.x.p + (t0 + t) * a.x.stride + k * ES);
    }
  };
  const auto store_x = [&](char* buf) {
    if constexpr (X != X_F32) {
#pragma unroll
      for (int i = 0; i < PIECES; ++i) {
        const int p = i * THREADS + threadIdx.x, t = p / (8 * ES), at = p % (8 * ES);
        if constexpr (X == X_WIDE) {
          *reinterpret_cast<bf16x8*>(buf + place<X>(t, 2 * at)) = widen8(xr[i][0], xr[i][1]);
          *reinterpret_cast<bf16x8*>(buf + place<X>(t, 2 * at + 1)) = widen8(xr[i][2], xr[i][3]);
        } else {
          *reinterpret_cast<u32x4*>(buf + place<X>(t, at)) = xr[i];
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < PIECES; ++i) {  // 4 values: half a piece of each plane
        const int p = i * THREADS + threadIdx.x, t = p / 32, at = p % 32;
        float r[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) r[e] = __uint_as_float(xr[i][e]);
#pragma unroll
        for (int k = 0; k < 3; ++k) {
          const u32x2 w = {pack_bf16(r[0], r[1]), pack_bf16(r[2], r[3])};
          *reinterpret_cast<u32x2*>(buf + k * PLANE + place<X>(t, at / 2) + at % 2 * 8) = w;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            r[2 * e] -= __uint_as_float(w[e] << 16);
            r[2 * e + 1] -= __uint_as_float(w[e] & 0xFFFF0000u);
          }
        }
      }
    }
  };
  const auto load_w = [&](int64_t kb, u32x4 (&cc)[NM][2], unsigned (&ss)[NM][2]) {
#pragma unroll
    for (int i = 0; i < NM; ++i)
#pragma unroll
      for (int v = 0; v < 2; ++v) {  // groups 2 v + h of the 128 columns
        cc[i][v] = *reinterpret_cast<const u32x4*>(cp[i] + kb * 1024 + v * 512);
        ss[i][v] = *reinterpret_cast<const uint8_t*>(sp[i] + (kb >> 2) * 256 + v * 128 + (kb & 3));
      }
  };

  f32x16 acc[NT][NM] = {};
  const auto multiply = [&](const char* buf, const u32x4 (&cc)[NM][2], const unsigned (&ss)[NM][2]) {
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      if constexpr (X == X_E4M3) {
        i32x8 w[NM];
#pragma unroll
        for (int i = 0; i < NM; ++i) w[i] = i32x8{(int)cc[i][v][0], (int)cc[i][v][1], (int)cc[i][v][2], (int)cc[i][v][3], 0, 0, 0, 0};
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const int row = wt + t * 32 + l32;
          const u32x4 lo = *reinterpret_cast<const u32x4*>(buf + place<X>(row, 4 * v + h));
          const u32x4 hi = *reinterpret_cast<const u32x4*>(buf + place<X>(row, 4 * v + 2 + h));
          const i32x8 x = __builtin_bit_cast(i32x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
#pragma unroll
          for (int i = 0; i < NM; ++i)
            acc[t][i] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, w[i], acc[t][i], 0, 4, 0, 0x7F7F7F7F, 0, (int)ss[i][v]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          bf16x8 w[NM];
#pragma unroll
          for (int i = 0; i < NM; ++i) w[i] = weights8(cc[i][v][j], pow2(ss[i][v]));
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int k = PL - 1; k >= 0; --k) {
              const bf16x8 x = *reinterpret_cast<const bf16x8*>(buf + k * PLANE + place<X>(wt + t * 32 + l32, 4 * (2 * v + h) + j));
#pragma unroll
              for (int i = 0; i < NM; ++i) acc[t][i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x, w[i], acc[t][i], 0, 0, 0);
            }
        }
      }
    }
  };

  if (k_lo < k_hi) {
    load_x(k_lo);
    load_w(k_lo, c[0], s[0]);
    store_x(lds);
    __syncthreads();
    for (int64_t kb = k_lo; kb < k_hi; kb += 2) {
      if (kb + 1 < k_hi) {
        load_x(kb + 1);
        load_w(kb + 1, c[1], s[1]);
      }
      multiply(lds, c[0], s[0]);
      if (kb + 1 >= k_hi) break;
      store_x(lds + TILE);
      __syncthreads();
      if (kb + 2 < k_hi) {
        load_x(kb + 2);
        load_w(kb + 2, c[0], s[0]);
      }
      multiply(lds + TILE, c[1], s[1]);
      if (kb + 2 < k_hi) store_x(lds);
      __syncthreads();
    }
  }

  // a lane holds row l32 of the weight, for tokens 8 (i / 4) + 4 h + i % 4
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int64_t row = t0 + wt + t * 32 + 8 * (i / 4) + 4 * h + i % 4;
      if (row >= a.T) continue;
#pragma unroll
      for (int j = 0; j < NM; ++j) {
        const int64_t m = m0 + wm + j * 32 + l32;
        if (m >= a.M) continue;
        float y = acc[t][j][i];
        if (splits > 1) {
          a.partial[(blockIdx.y * a.T + row) * a.M + m] = y;
        } else {
          if constexpr (x_scaled<X>()) y *= a.x_scale[row];
          reinterpret_cast<OUT*>(a.out.p + row * a.out.stride)[m] = from_f32<OUT>(y);
        }
      }
    }
}

template <bool SCALED, typename OUT>
__global__ __launch_bounds__(256) void q4_join(const LinearArgs a, int splits) {
  const int64_t n = a.T * a.M, step = (int64_t)gridDim.x * 256;
  for (int64_t o = (int64_t)blockIdx.x * 256 + threadIdx.x; o < n; o += step) {
    const int64_t t = o / a.M, m = o % a.M;
    float y = 0.0f;
    for (int i = 0; i < splits; ++i) y += a.partial[i * n + o];
    if constexpr (SCALED) y *= a.x_scale[t];
    reinterpret_cast<OUT*>(a.out.p + t * a.out.stride)[m] = from_f32<OUT>(y);
  }
}

template <int X, int BT, typename OUT>
hipError_t launch(const LinearArgs& a, int splits, hipStream_t s) {
  const int64_t tiles = (a.T + BT - 1) / BT * ((a.M + BM - 1) / BM);
  q4_tiles<X, BT, OUT><<<dim3((unsigned)tiles, (unsigned)splits), dim3(THREADS), 0, s>>>(a, splits);
  if (const hipError_t e = hipGetLastError()) return e;
  if (splits > 1) {
    const int64_t want = (a.T * a.M + 255) / 256;
    q4_join<x_scaled<X>(), OUT><<<dim3((unsigned)(want < 4096 ? want : 4096)), dim3(256), 0, s>>>(a, splits);
  }
  return hipGetLastError();
}

int tokens_of(int64_t T, int x_dtype) {
  if (T <= 32) return 32;
  if (T <= 64 || x_dtype == X_F32) return 64;
  return 128;
}

template <int X, typename OUT>
hipError_t launch_tokens(const LinearArgs& a, int splits, hipStream_t s) {
  const int bt = tokens_of(a.T, X);
  if (bt == 32) return launch<X, 32, OUT>(a, splits, s);
  if constexpr (X != X_F32)
    if (bt == 128) return launch<X, 128, OUT>(a, splits, s);
  return launch<X, 64, OUT>(a, splits, s);
}

}  // namespace

hipError_t launch_q4_tiles(const LinearArgs& a, int x_dtype, int out_dtype, int splits, hipStream_t s) {
  const bool bf16 = out_dtype == SSM_BF16;
  if (x_dtype == X_F32) return bf16 ? launch_tokens<X_F32, bf16_t>(a, splits, s) : launch_tokens<X_F32, float>(a, splits, s);
  if (x_dtype == X_BF16) return bf16 ? launch_tokens<X_BF16, bf16_t>(a, splits, s) : launch_tokens<X_BF16, float>(a, splits, s);
  return bf16 ? launch_tokens<X_E4M3, bf16_t>(a, splits, s) : launch_tokens<X_WIDE, float>(a, splits, s);
}

// Workgroups that share a tile's columns: two workgroups to a CU are wanted, and four steps of 128 columns at least for each.
int q4_tiles_splits(int64_t T, int x_dtype, int64_t M, int64_t K) {
  const int bt = tokens_of(T, x_dtype);
  const int64_t tiles = (T + bt - 1) / bt * ((M + BM - 1) / BM), steps = (K + 127) / 128;
  int64_t n = 512 / tiles;
  if (n > steps / 4) n = steps / 4;
  return n < 1 ? 1 : n > 16 ? 16 : (int)n;
}

}  // namespace block
}  // namespace ssm

extern "C" {

size_t ssm_q4_linear_workspace_bytes(int64_t tokens, int32_t x_dtype, int64_t out_features, int64_t in_features) {
  using namespace ssm::block;
  if (tokens < 1 || tokens >= MAX_TOKENS || !q4_sizes(out_features, in_features)) return 0;
  if (x_dtype != SSM_F32 && x_dtype != SSM_BF16 && x_dtype != SSM_E4M3) return 0;
  if (tokens <= ROWS_MAX_TOKENS || tokens * out_features > MAX_OUTPUTS) return 0;
  const int splits = q4_tiles_splits(tokens, x_dtype, out_features, in_features);
  return splits > 1 ? (size_t)splits * tokens * out_features * 4 : 0;
}

int ssm_q4_linear(int64_t tokens, int32_t x_dtype, int32_t out_dtype, const ssm_rows* x, const float* x_scale,
                  const ssm_q4_weight* q, const ssm_rows* out, void* workspace, size_t workspace_bytes, void* stream) {
  using namespace ssm::block;
  if (tokens < 0 || tokens >= MAX_TOKENS) return SSM_ERR_SHAPE;
  if (x_dtype != SSM_F32 && x_dtype != SSM_BF16 && x_dtype != SSM_E4M3) return SSM_ERR_DTYPE;
  if (out_dtype != SSM_F32 && out_dtype != SSM_BF16) return SSM_ERR_DTYPE;
  if (const int st = check_q4(q)) return st;
  if (tokens * q->out_features > MAX_OUTPUTS) return SSM_ERR_SHAPE;
  if (tokens == 0) return SSM_OK;  // its tensors have no addresses
  if ((x_dtype == SSM_E4M3) != (x_scale != nullptr)) return SSM_ERR_NULL;
  const int64_t T = tokens, M = q->out_features, K = q->in_features, es = size_of(x_dtype), os = size_of(out_dtype);
  if (const int st = check_rows(x, es, 16)) return st;
  if (const int st = check_rows(out, os, os)) return st;
  if (!aligned(x_scale, 4)) return SSM_ERR_ALIGN;
  const size_t need = ssm_q4_linear_workspace_bytes(T, x_dtype, M, K);
  if (need && (!workspace || workspace_bytes < need)) return SSM_ERR_WORKSPACE;
  if (need && !aligned(workspace, 16)) return SSM_ERR_ALIGN;
  const Span so = rows_span(out, T, M, os), sw = span(workspace, (int64_t)need);
  const Span ins[3] = {codes_span(q), scales_span(q), span(x_scale, x_scale ? T * 4 : 0)};
  for (const Span& i : ins)
    if (overlaps(so, i) || overlaps(sw, i)) return SSM_ERR_ALIAS;
  if (!writable(out, T, M) || overlaps(so, sw) || overlaps(sw, rows_span(x, T, K, es)) || rows_overlap(out, M, os, x, K, es, T))
    return SSM_ERR_ALIAS;
  LinearArgs a = {};
  a.x = rows_of(x, es);
  a.out = rows_of(out, os);
  a.codes = static_cast<const char*>(q->codes);
  a.scales = static_cast<const char*>(q->scales);
  a.x_scale = x_scale;
  a.partial = static_cast<float*>(workspace);
  a.T = T;
  a.M = M;
  a.K = K;
  a.kt = (K + 127) / 128;
  a.k4 = (K + 511) / 512;
  a.mt = (M + 15) / 16;
  const hipStream_t s = ready(stream);
  const hipError_t e = T <= ROWS_MAX_TOKENS ? launch_q4_rows(a, x_dtype, out_dtype, s)
                                            : launch_q4_tiles(a, x_dtype, out_dtype, q4_tiles_splits(T, x_dtype, M, K), s);
  return e == hipSuccess ? SSM_OK : SSM_ERR_LAUNCH;
}

}  // extern "C"
