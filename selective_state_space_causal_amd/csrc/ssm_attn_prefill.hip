// ssm_attn_prefill.hip -- ssm_attn_prefill of include/ssm_attn.h: softmax attention over packed
// prompts, one pass over the keys with the running maximum and sum of each row's softmax.
//
// Rows.  The query heads that share a key head are packed into the rows of a tile: row r of a sequence
// is token r / G, query head kv_head * G + r % G (G = query heads per key head).  A key tile is then
// read once for all G heads, and a short sequence fills a tile G times better.
//
// Products.  Scores are computed transposed, S^T = K Q^T, with 32x32 matrix instructions: a lane then
// holds scores of ONE row (column lane & 31), 16 keys of every 32, the other 16 being in lane ^ 32.
// Row maxima and sums are therefore taken inside a lane, with a single exchange of the two halves, and
// the weights are already in the layout of the second product's right operand, O^T = V^T P^T: the
// order of the keys inside a product is free as long as V is read in the same order.  V's operand needs
// keys along a lane's registers, and V is stored with channels along a row: bf16 uses the LDS read that
// transposes 16-bit elements.
#include "ssm_attn.h"

namespace ssm {
namespace attn {
namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
#define LDS_PTR(T, p) ((__attribute__((address_space(3))) T*)(p))

struct PrefillArgs {
  View q, k, v, out;
  float* lse;
  const int32_t* cu_q;
  const int32_t* cu_k;
  int B, Tq, Tk, Hq, Hkv, G, D;
  int causal;
  float scale_log2;  // scale * log2(e)
  int64_t work;      // upper bound of tiles of all key heads
};

// The sequence and tile that hold tile `idx` of the packed batch (false past the end).  Each wave finds
// it by itself: 64 sequences at a time, a prefix sum of their tile counts over the lanes.
__device__ __forceinline__ bool find_tile(const PrefillArgs& a, int QT, int64_t idx, int& b, int& tile, int& tiles,
                                          int& q0, int& lq) {
  const int lane = threadIdx.x & 63;
  int64_t base = 0;
  for (int b0 = 0; b0 < a.B; b0 += 64) {
    const int bb = b0 + lane;
    int start = 0, len = 0;
    if (bb < a.B) {
      start = min(max(a.cu_q[bb], 0), a.Tq);
      len = max(min(a.cu_q[bb + 1], a.Tq) - start, 0);
    }
    const int n = (int)(((int64_t)len * a.G + QT - 1) / QT);
    int incl = n;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
      const int up = __shfl_up(incl, m);
      if (lane >= m) incl += up;
    }
    const int total = __shfl(incl, 63);
    if (idx < base + total) {
      const int want = (int)(idx - base);
      const int first = __ffsll((unsigned long long)__ballot(incl > want)) - 1;
      b = __builtin_amdgcn_readfirstlane(b0 + first);
      tiles = __builtin_amdgcn_readfirstlane(__shfl(n, first));
      tile = __builtin_amdgcn_readfirstlane(want - (__shfl(incl, first) - tiles));
      q0 = __builtin_amdgcn_readfirstlane(__shfl(start, first));
      lq = __builtin_amdgcn_readfirstlane(__shfl(len, first));
      return true;
    }
    base += total;
  }
  return false;
}

// The two halves' values of one row joined: max / sum over lane and lane ^ 32.
__device__ __forceinline__ float half_max(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float half_sum(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// One key tile in LDS: KT rows of DP elements, in 16-byte chunks whose place in the row is exchanged
// by the row number so that lanes reading the same chunk of neighbouring rows use different banks.
template <typename IO, int DP>
struct Tile;

template <int DP>
struct Tile<bf16_t, DP> {
  static constexpr int CH = DP / 8;  // chunks of a row
  __device__ static int k_at(int row, int ch) { return (row * CH + (ch ^ (row & 7))) * 16; }
  __device__ static int v_at(int row, int ch) { return (row * CH + (ch ^ ((row & 3) << 1))) * 16; }
};
template <int DP>
struct Tile<float, DP> {
  static constexpr int CH = DP / 4;
  __device__ static int k_at(int row, int ch) { return (row * CH + (ch ^ (row & 7))) * 16; }
  __device__ static int v_at(int row, int ch) { return (row * CH + ch) * 16; }
};

template <typename IO, int DP, int NW, int KT>
__global__ __launch_bounds__(NW * 64, DP <= 128 && sizeof(IO) == 2 ? 2 : 1) void attn_prefill(PrefillArgs a) {
  constexpr bool BF = sizeof(IO) == 2;
  constexpr int ES = sizeof(IO), QT = NW * 32, T = Tile<IO, DP>::CH, EPC = 16 / ES, NS = KT / 32, ND = DP / 32;
  typedef Tile<IO, DP> L;
  __shared__ __attribute__((aligned(16))) char kt[KT * DP * ES];
  __shared__ __attribute__((aligned(16))) char vt[KT * DP * ES];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 31, half = lane >> 5;

  for (int64_t idx = blockIdx.x; idx < a.work; idx += gridDim.x) {
    const int h = (int)(idx % a.Hkv);
    int b, tile, tiles, q0, lq;
    if (!find_tile(a, QT, idx / a.Hkv, b, tile, tiles, q0, lq)) break;  // later ones are past the end too
    tile = tiles - 1 - tile;  // causal: the tiles with the most keys first
    const int k0 = min(max(a.cu_k[b], 0), a.Tk);
    const int lk = max(min(a.cu_k[b + 1], a.Tk) - k0, 0);
    const int rows = lq * a.G, r0 = tile * QT + wave * 32;
    const int r = r0 + col, rc = min(r, rows - 1);
    const int tok = rc / a.G, g = rc - tok * a.G;
    // Keys that a row sees: [0, seen).
    const auto seen_by = [&](int token) { return a.causal ? min(max(token + 1 + lk - lq, 0), lk) : lk; };
    const int seen = seen_by(tok);
    const int wave_first = __builtin_amdgcn_readfirstlane(seen_by(min(r0, rows - 1) / a.G));
    const int wave_last = __builtin_amdgcn_readfirstlane(seen_by(min(r0 + 31, rows - 1) / a.G));
    const int block_last = seen_by(min(tile * QT + QT - 1, rows - 1) / a.G);

    // Q as the right operand: a lane's row, in the order that the K reads below use.
    constexpr int NQ = BF ? DP / 16 : DP / 8;
    u32x4 qf[NQ];
    const char* qp = a.q.p + (int64_t)(q0 + tok) * a.q.ts + (int64_t)(h * a.G + g) * a.q.hs;
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      const int ch = 2 * i + half;
      qf[i] = ch * EPC < a.D ? *reinterpret_cast<const u32x4*>(qp + ch * 16) : u32x4{0, 0, 0, 0};
    }
    f32x16 o[ND] = {};
    float m = -INFINITY, l = 0.0f;

    const char* kp = a.k.p + (int64_t)k0 * a.k.ts + (int64_t)h * a.k.hs;
    const char* vp = a.v.p + (int64_t)k0 * a.v.ts + (int64_t)h * a.v.hs;
    for (int j0 = 0; j0 < block_last; j0 += KT) {
      __syncthreads();
      for (int c = threadIdx.x; c < KT * T; c += NW * 64) {
        const int row = c / T, ch = c - row * T;
        const int64_t key = min(j0 + row, lk - 1);  // rows past the end repeat the last key: finite, masked below
        const bool in = ch * EPC < a.D;
        const u32x4 z = {0, 0, 0, 0};
        *reinterpret_cast<u32x4*>(kt + L::k_at(row, ch)) =
            in ? *reinterpret_cast<const u32x4*>(kp + key * a.k.ts + ch * 16) : z;
        *reinterpret_cast<u32x4*>(vt + L::v_at(row, ch)) =
            in ? *reinterpret_cast<const u32x4*>(vp + key * a.v.ts + ch * 16) : z;
      }
      __syncthreads();
      if (j0 >= wave_last) continue;

      f32x16 s[NS];
#pragma unroll
      for (int n = 0; n < NS; ++n) {
        s[n] = f32x16{};
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
          const u32x4 kf = *reinterpret_cast<const u32x4*>(kt + L::k_at(n * 32 + col, 2 * i + half));
          if constexpr (BF) {
            s[n] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, kf),
                                                           __builtin_bit_cast(bf16x8, qf[i]), s[n], 0, 0, 0);
          } else {
            const f32x4 kx = __builtin_bit_cast(f32x4, kf), qx = __builtin_bit_cast(f32x4, qf[i]);
#pragma unroll
            for (int j = 0; j < 4; ++j) s[n] = __builtin_amdgcn_mfma_f32_32x32x2f32(kx[j], qx[j], s[n], 0, 0, 0);
          }
        }
      }
      if (j0 + KT > wave_first) {  // some row of the wave does not see some key of the tile
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int key = j0 + n * 32 + 8 * (i / 4) + 4 * half + i % 4;
            s[n][i] = key < seen ? s[n][i] : -INFINITY;
          }
      }
      float mx = m;
#pragma unroll
      for (int n = 0; n < NS; ++n)
#pragma unroll
        for (int i = 0; i < 16; ++i) mx = fmaxf(mx, s[n][i]);
      mx = half_max(mx);
      const float mc = mx == -INFINITY ? 0.0f : mx * a.scale_log2;  // a row that has seen nothing yet: all weights 0
      const float alpha = hw_exp2(fmaf(m, a.scale_log2, -mc));
      m = mx;
      float sum = 0.0f;
#pragma unroll
      for (int n = 0; n < NS; ++n)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          s[n][i] = hw_exp2(fmaf(s[n][i], a.scale_log2, -mc));
          sum += s[n][i];
        }
      l = l * alpha + sum;  // this half's keys only; joined at the end
#pragma unroll
      for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[d][i] *= alpha;

      if constexpr (BF) {
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
          for (int t = 0; t < 2; ++t) {  // 16 keys: this half holds keys 4 half + {0..3, 8..11} of them
            u32x4 pf;
#pragma unroll
            for (int i = 0; i < 4; ++i) pf[i] = pack_bf16(s[n][8 * t + 2 * i], s[n][8 * t + 2 * i + 1]);
            // The transposing read: 16 lanes give 4 rows of 16 channels and get 4 rows of one channel each.
            const int row = n * 32 + 16 * t + 4 * half + (lane & 15) / 4;
#pragma unroll
            for (int d = 0; d < ND; ++d) {
              const int e = d * 32 + (col & 16) + (lane & 3) * 4;
              union {
                s16x4 x[2];
                bf16x8 v;
              } vf;
              vf.x[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(LDS_PTR(s16x4, vt + L::v_at(row, e / 8) + (e & 4) * 2));
              vf.x[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(LDS_PTR(s16x4, vt + L::v_at(row + 8, e / 8) + (e & 4) * 2));
              o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf.v, __builtin_bit_cast(bf16x8, pf), o[d], 0, 0, 0);
            }
          }
      } else {
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int row = n * 32 + 8 * (i / 4) + 4 * half + i % 4;
#pragma unroll
            for (int d = 0; d < ND; ++d) {
              const int e = d * 32 + col;
              const float vx = *reinterpret_cast<const float*>(vt + L::v_at(row, e / 4) + (e & 3) * 4);
              o[d] = __builtin_amdgcn_mfma_f32_32x32x2f32(vx, s[n][i], o[d], 0, 0, 0);
            }
          }
      }
    }

    l = half_sum(l);
    if (r < rows) {
      const float inv = l > 0.0f ? 1.0f / l : 0.0f;
      const int head = h * a.G + g;
      char* op = a.out.p + (int64_t)(q0 + tok) * a.out.ts + (int64_t)head * a.out.hs;
#pragma unroll
      for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int e = d * 32 + 8 * i + 4 * half;
          if (e >= a.D) continue;
          const float x0 = o[d][4 * i] * inv, x1 = o[d][4 * i + 1] * inv, x2 = o[d][4 * i + 2] * inv,
                      x3 = o[d][4 * i + 3] * inv;
          if constexpr (BF)
            *reinterpret_cast<u32x2*>(op + e * 2) = u32x2{pack_bf16(x0, x1), pack_bf16(x2, x3)};
          else
            *reinterpret_cast<f32x4*>(op + e * 4) = f32x4{x0, x1, x2, x3};
        }
      if (a.lse && half == 0)
        a.lse[(int64_t)(q0 + tok) * a.Hq + head] =
            l > 0.0f ? (m * a.scale_log2 + __builtin_amdgcn_logf(l)) * kLn2 : -INFINITY;
    }
  }
}

constexpr int64_t MAX_GRID = int64_t(1) << 22;  // keeps a launch within 2^31 work-items

template <typename IO, int DP, int NW, int KT>
hipError_t launch(PrefillArgs& a, hipStream_t s) {
  const int64_t tiles = (int64_t)a.Tq * a.G / (NW * 32) + a.B;  // sum of ceil(rows / QT) over the sequences
  a.work = tiles * a.Hkv;
  const dim3 grid((unsigned)(a.work < MAX_GRID ? a.work : MAX_GRID)), tb(NW * 64);
  attn_prefill<IO, DP, NW, KT><<<grid, tb, 0, s>>>(a);
  return hipGetLastError();
}

template <typename IO, int KT>
hipError_t launch_dim(PrefillArgs& a, hipStream_t s) {
  if (a.D <= 64) return launch<IO, 64, 4, KT>(a, s);
  if (a.D <= 128) return launch<IO, 128, 4, KT>(a, s);
  if (a.D <= 192) return launch<IO, 192, 4, KT>(a, s);
  return launch<IO, 256, 4, KT>(a, s);
}

}  // namespace
}  // namespace attn
}  // namespace ssm

extern "C" int ssm_attn_prefill(const ssm_attn_dims* d, const ssm_view* q, const ssm_view* k, const ssm_view* v,
                                const int32_t* cu_q, const int32_t* cu_k, const ssm_view* out, float* lse,
                                void* stream) {
  using namespace ssm::attn;
  if (!d) return SSM_ERR_NULL;
  int64_t es;
  if (const int st = check_io(d->io_dtype, &es)) return st;
  if (const int st = check_heads(d->q_heads, d->head_dim)) return st;
  if (const int st = check_heads(d->kv_heads, d->head_dim)) return st;
  if (d->q_heads % d->kv_heads) return SSM_ERR_SHAPE;
  if (d->batch < 1 || d->batch > SSM_ATTN_MAX_BATCH) return SSM_ERR_SHAPE;
  if (d->q_tokens < 0 || d->k_tokens < 0 || d->k_tokens > MAX_TOKENS) return SSM_ERR_SHAPE;
  if (d->q_tokens > MAX_TOKENS / (d->q_heads / d->kv_heads)) return SSM_ERR_SHAPE;
  if (!isfinite(d->scale) || !(d->scale > 0.0f) || (d->causal != 0 && d->causal != 1)) return SSM_ERR_SHAPE;
  if (d->q_tokens == 0) return SSM_OK;
  if (!cu_q || !cu_k) return SSM_ERR_NULL;
  if (const int st = check_view(q, es)) return st;
  if (const int st = check_view(out, es)) return st;
  const int64_t Tq = d->q_tokens, Tk = d->k_tokens, D = d->head_dim, Hq = d->q_heads, Hkv = d->kv_heads;
  if (Tk) {
    if (const int st = check_view(k, es)) return st;
    if (const int st = check_view(v, es)) return st;
  }
  if (!aligned(cu_q, 4) || !aligned(cu_k, 4) || !aligned(lse, 4)) return SSM_ERR_ALIGN;
  if (!writable(out, Tq, Hq, D) || views_overlap(out, Tq, Hq, q, Tq, Hq, D, es)) return SSM_ERR_ALIAS;
  const Span so = view_span(out, Tq, Hq, D, es), sl = span(lse, lse ? Tq * Hq * 4 : 0);
  const Span s_cu[2] = {span(cu_q, (d->batch + 1) * 4), span(cu_k, (d->batch + 1) * 4)};
  for (const Span& c : s_cu)
    if (overlaps(so, c) || overlaps(sl, c)) return SSM_ERR_ALIAS;
  if (overlaps(so, sl) || overlaps(sl, view_span(q, Tq, Hq, D, es))) return SSM_ERR_ALIAS;
  if (Tk) {
    if (views_overlap(out, Tq, Hq, k, Tk, Hkv, D, es) || views_overlap(out, Tq, Hq, v, Tk, Hkv, D, es))
      return SSM_ERR_ALIAS;
    if (overlaps(sl, view_span(k, Tk, Hkv, D, es)) || overlaps(sl, view_span(v, Tk, Hkv, D, es))) return SSM_ERR_ALIAS;
  }
  PrefillArgs a = {};
  a.q = bytes_view(q, es);
  a.out = bytes_view(out, es);
  if (Tk) {
    a.k = bytes_view(k, es);
    a.v = bytes_view(v, es);
  }
  a.lse = lse;
  a.cu_q = cu_q;
  a.cu_k = cu_k;
  a.B = (int)d->batch;
  a.Tq = (int)Tq;
  a.Tk = (int)Tk;
  a.Hq = d->q_heads;
  a.Hkv = d->kv_heads;
  a.G = d->q_heads / d->kv_heads;
  a.D = d->head_dim;
  a.causal = d->causal;
  a.scale_log2 = d->scale * 1.4426950408889634f;
  if (!isfinite(a.scale_log2) || !(a.scale_log2 > 0.0f)) return SSM_ERR_SHAPE;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const hipError_t e = d->io_dtype == SSM_BF16 ? launch_dim<ssm::bf16_t, 64>(a, s) : launch_dim<float, 32>(a, s);
  return e == hipSuccess ? SSM_OK : SSM_ERR_LAUNCH;
}
