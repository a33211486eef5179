// ssm_attn_decode.hip -- ssm_attn_decode_step of include/ssm_attn.h: one query token per sequence
// against the paged key/value cache.
//
// The cache is read once, and that bounds it.  The query heads of a key head (up to 16 at a time) are
// the columns of 16x16 matrix products, so a key is read once for all of them: S^T = K Q^T, then
// O^T = V^T P^T with the softmax's running maximum and sum.  A wave works on 32 keys at a time.  Row m of
// score tile t stands for key 8 (m / 4) + 4 t + m % 4 of the 32, which gives lane quarter w the weights
// of keys 8 w .. 8 w + 7 in order: what the second product's right operand wants.  Its left operand
// needs V with keys along a lane's registers; the wave passes V through its own LDS and the LDS read that
// transposes (16-bit and 8-bit elements).  The long axis is split over waves; their partial results
// (maximum, sum, unnormalised output, fp32) are joined by a second kernel in split order.
#include "ssm_attn.h"

namespace ssm {
namespace attn {
namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef int i32x2 __attribute__((ext_vector_type(2)));
#define LDS_PTR(T, p) ((__attribute__((address_space(3))) T*)(p))

constexpr int STEP = 32;  // keys of a wave's step
constexpr int COLS = 16;  // query heads of a wave

struct DecodeArgs {
  View q, out;
  float* lse;
  Cache c;
  const int32_t* table;
  const int32_t* lens;
  int64_t W;  // table width
  int B, Hq, G, groups;  // groups: 16-head groups of a key head
  int splits;
  float scale_log2;
  float* po;  // [B, Hq, splits, D]
  float* ml;  // [B, Hq, splits, 2]: maximum (of scores * log2 e), sum
};

__device__ __forceinline__ int sequence_length(const DecodeArgs& a, int b) {
  const int64_t cap = a.W << a.c.page_shift;
  const int64_t n = a.lens[b];
  return (int)(n < 0 ? 0 : n > cap ? cap : n);
}

// Eight codes as bf16 (exact: an int8 or e4m3 value has at most 7 significant bits).
template <int KV>
__device__ __forceinline__ u32x4 widen_bf16(u32x2 w) {
  u32x4 r;
  if constexpr (KV == SSM_KV_I8) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const unsigned x = w[j / 2] >> (16 * (j & 1));
      r[j] = pack_bf16((float)(int8_t)x, (float)(int8_t)(x >> 8));
    }
  } else {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      r[2 * j] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[j], 1.0f, false));
      r[2 * j + 1] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[j], 1.0f, true));
    }
  }
  return r;
}

// Code j of a word as fp32.
template <int KV>
__device__ __forceinline__ f32x4 widen_f32(unsigned w) {
  if constexpr (KV == SSM_KV_I8) {
    return f32x4{(float)(int8_t)w, (float)(int8_t)(w >> 8), (float)(int8_t)(w >> 16), (float)(int8_t)(w >> 24)};
  } else {
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
    return f32x4{lo[0], lo[1], hi[0], hi[1]};
  }
}

__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// CS: bytes of a cached element.  NW waves of a workgroup, each a split of its own.
template <typename IO, int KV, int DP, int NW>
__global__ __launch_bounds__(NW * 64) void attn_decode(DecodeArgs a) {
  constexpr bool BF = sizeof(IO) == 2;
  constexpr int CS = KV == SSM_KV_IO ? sizeof(IO) : 1, ND = DP / 16;
  __shared__ __attribute__((aligned(16))) char lds[NW][STEP * DP * CS];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 15, w4 = lane >> 4;
  char* vt = lds[wave];
  const int split = blockIdx.x * NW + wave, b = blockIdx.z;
  const int kh = blockIdx.y / a.groups, g0 = (blockIdx.y - kh * a.groups) * COLS;
  if (split >= a.splits) return;
  const int D = a.c.D, len = sequence_length(a, b);
  const int page_mask = (1 << a.c.page_shift) - 1;
  // Equal shares of whole steps.
  const int steps = (len + STEP - 1) / STEP, share = (steps + a.splits - 1) / a.splits;
  const int first = min((int64_t)split * share, (int64_t)steps) * STEP;
  const int last = (int)min((int64_t)len, (int64_t)first + (int64_t)share * STEP);

  const int g = g0 + col;
  const bool live = g < a.G;
  const int head = kh * a.G + min(g, a.G - 1);
  const char* qp = a.q.p + (int64_t)b * a.q.ts + (int64_t)head * a.q.hs;
  constexpr int NQ = BF ? DP / 32 : DP / 16, QC = 16 / (int)sizeof(IO);
  u32x4 qf[NQ];
#pragma unroll
  for (int i = 0; i < NQ; ++i) {
    const int e = (4 * i + w4) * QC;
    qf[i] = e < D ? *reinterpret_cast<const u32x4*>(qp + e * (int)sizeof(IO)) : u32x4{0, 0, 0, 0};
  }
  f32x4 o[ND] = {};
  float m = -INFINITY, l = 0.0f;
  const int32_t* table = a.table + (int64_t)b * a.W;

  // Row of the cache that holds a key of this head, or -1.
  const auto row_of = [&](int key) -> int64_t {
    if (key >= last) return -1;
    const int64_t page = table[key >> a.c.page_shift];
    if (page < 0 || page >= (a.c.slots >> a.c.page_shift)) return -1;
    return ((page * a.c.heads + kh) << a.c.page_shift) + (key & page_mask);
  };

  for (int j0 = first; j0 < last; j0 += STEP) {
    // V rows into LDS, zeros where no key is.
    constexpr int VB = CS == 1 ? 8 : 16, VC = DP * CS / VB;  // bytes of a piece, pieces of a row
#pragma unroll 4
    for (int c = lane; c < STEP * VC; c += 64) {
      const int row = c / VC, piece = c - row * VC;
      const int64_t at = row_of(j0 + row);
      const bool in = at >= 0 && piece * VB < D * CS;
      if constexpr (CS == 1) {
        u32x2 x = {0, 0};
        if (in) x = *reinterpret_cast<const u32x2_a4*>(a.c.v + at * D + piece * 8);
        *reinterpret_cast<u32x2*>(vt + row * DP + piece * 8) = x;
      } else {
        u32x4 x = {0, 0, 0, 0};
        if (in) x = *reinterpret_cast<const u32x4*>(a.c.v + at * D * CS + piece * 16);
        *reinterpret_cast<u32x4*>(vt + row * DP * CS + piece * 16) = x;
      }
    }
    wave_lds_fence();

    f32x4 s[2] = {};
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int64_t at = row_of(j0 + 8 * (col >> 2) + 4 * t + (col & 3));
      const char* kp = a.c.k + (at < 0 ? 0 : at) * D * CS;  // an unseen key's scores are replaced below
#pragma unroll
      for (int i = 0; i < NQ; ++i) {
        const int e = (4 * i + w4) * QC;
        if constexpr (BF) {
          u32x4 kf = {0, 0, 0, 0};
          if (e < D) {
            if constexpr (CS == 1) kf = widen_bf16<KV>(*reinterpret_cast<const u32x2_a4*>(kp + e));
            else kf = *reinterpret_cast<const u32x4*>(kp + e * CS);
          }
          s[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, kf),
                                                         __builtin_bit_cast(bf16x8, qf[i]), s[t], 0, 0, 0);
        } else {
          f32x4 kx = {0, 0, 0, 0};
          if (e < D) {
            if constexpr (CS == 1) kx = widen_f32<KV>(*reinterpret_cast<const unsigned*>(kp + e));
            else kx = *reinterpret_cast<const f32x4*>(kp + e * CS);
          }
          const f32x4 qx = __builtin_bit_cast(f32x4, qf[i]);
#pragma unroll
          for (int j = 0; j < 4; ++j) s[t] = __builtin_amdgcn_mfma_f32_16x16x4f32(kx[j], qx[j], s[t], 0, 0, 0);
        }
      }
    }
    // This lane's keys: j0 + 8 w4 + 4 t + i, all on one page (pages are multiples of 16 tokens).
    const int key0 = j0 + 8 * w4;
    const int64_t at0 = row_of(key0);
    f32x4 sk[2] = {{1, 1, 1, 1}, {1, 1, 1, 1}}, sv[2] = {{1, 1, 1, 1}, {1, 1, 1, 1}};
    if constexpr (KV != SSM_KV_IO) {
      if (at0 >= 0) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          sk[t] = *reinterpret_cast<const f32x4*>(a.c.ks + at0 + 4 * t);
          sv[t] = *reinterpret_cast<const f32x4*>(a.c.vs + at0 + 4 * t);
        }
      }
    }
    float mx = m;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool seen = at0 >= 0 && key0 + 4 * t + i < last;
        s[t][i] = seen ? s[t][i] * sk[t][i] * a.scale_log2 : -INFINITY;
        sv[t][i] = seen ? sv[t][i] : 0.0f;
        mx = fmaxf(mx, s[t][i]);
      }
    mx = fmaxf(mx, __shfl_xor(mx, 16));
    mx = fmaxf(mx, __shfl_xor(mx, 32));
    const float mc = mx == -INFINITY ? 0.0f : mx;
    const float alpha = hw_exp2(m - mc);
    m = mx;
    float sum = 0.0f;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float p = hw_exp2(s[t][i] - mc);
        sum += p;
        s[t][i] = p * sv[t][i];
      }
    l = l * alpha + sum;  // this quarter's keys only; joined at the end
#pragma unroll
    for (int d = 0; d < ND; ++d) o[d] *= alpha;

    if constexpr (BF) {
      const u32x4 pf = {pack_bf16(s[0][0], s[0][1]), pack_bf16(s[0][2], s[0][3]), pack_bf16(s[1][0], s[1][1]),
                        pack_bf16(s[1][2], s[1][3])};
#pragma unroll
      for (int d = 0; d < ND; ++d) {
        u32x4 vf;
        if constexpr (CS == 1) {
          // 16 lanes give 8 rows of 16 codes and get 8 rows of one channel each
          const i32x2 x = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
              LDS_PTR(i32x2, vt + (8 * w4 + (col >> 1)) * DP + d * 16 + (col & 1) * 8));
          vf = widen_bf16<KV>(u32x2{(unsigned)x[0], (unsigned)x[1]});
        } else {
          union {
            s16x4 x[2];
            u32x4 v;
          } u;
          const char* p = vt + ((8 * w4 + (col >> 2)) * DP + d * 16 + (col & 3) * 4) * 2;
          u.x[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(LDS_PTR(s16x4, p));
          u.x[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(LDS_PTR(s16x4, p + 4 * DP * 2));
          vf = u.v;
        }
        o[d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, vf), __builtin_bit_cast(bf16x8, pf),
                                                       o[d], 0, 0, 0);
      }
    } else {
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = 8 * w4 + 4 * t + i;
#pragma unroll
          for (int d = 0; d < ND; ++d) {
            const char* p = vt + (row * DP + d * 16 + col) * CS;
            float x;
            if constexpr (CS == 4) x = *reinterpret_cast<const float*>(p);
            else x = widen_f32<KV>(*reinterpret_cast<const uint8_t*>(p))[0];
            o[d] = __builtin_amdgcn_mfma_f32_16x16x4f32(x, s[t][i], o[d], 0, 0, 0);
          }
        }
    }
    wave_lds_fence();
  }

  l += __shfl_xor(l, 16);
  l += __shfl_xor(l, 32);
  if (!live) return;
  if (a.splits == 1) {
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
    char* op = a.out.p + (int64_t)b * a.out.ts + (int64_t)head * a.out.hs;
#pragma unroll
    for (int d = 0; d < ND; ++d) {
      const int e = d * 16 + 4 * w4;
      if (e >= D) continue;
      const f32x4 x = o[d] * inv;
      if constexpr (BF) *reinterpret_cast<u32x2*>(op + e * 2) = u32x2{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3])};
      else *reinterpret_cast<f32x4*>(op + e * 4) = x;
    }
    if (a.lse && w4 == 0)
      a.lse[(int64_t)b * a.Hq + head] = l > 0.0f ? (m + __builtin_amdgcn_logf(l)) * kLn2 : -INFINITY;
  } else {
    const int64_t at = ((int64_t)b * a.Hq + head) * a.splits + split;
    if (l > 0.0f) {
      float* op = a.po + at * D;
#pragma unroll
      for (int d = 0; d < ND; ++d)
        if (d * 16 + 4 * w4 < D) *reinterpret_cast<f32x4*>(op + d * 16 + 4 * w4) = o[d];
    }
    if (w4 == 0) {
      a.ml[2 * at] = m;
      a.ml[2 * at + 1] = l;
    }
  }
}

// Joins the splits of one (sequence, head): a workgroup of 256 threads, thread e of the first D owning
// channel e, the splits in order.
template <typename IO>
__global__ __launch_bounds__(256) void attn_decode_join(DecodeArgs a) {
  const int64_t row = blockIdx.x;  // b * Hq + head
  const float* ml = a.ml + row * a.splits * 2;
  float m = -INFINITY;
  for (int s = 0; s < a.splits; ++s) m = fmaxf(m, ml[2 * s]);
  const float mc = m == -INFINITY ? 0.0f : m;
  float l = 0.0f, x = 0.0f;
  const int e = threadIdx.x;
  for (int s = 0; s < a.splits; ++s) {
    const float ls = ml[2 * s + 1];
    if (!(ls > 0.0f)) continue;  // no key: no output was written
    const float w = hw_exp2(ml[2 * s] - mc);
    l += w * ls;
    if (e < a.c.D) x += w * a.po[(row * a.splits + s) * a.c.D + e];
  }
  const int b = (int)(row / a.Hq), head = (int)(row - (int64_t)b * a.Hq);
  if (e < a.c.D) {
    char* op = a.out.p + (int64_t)b * a.out.ts + (int64_t)head * a.out.hs;
    const float y = l > 0.0f ? x / l : 0.0f;
    if constexpr (sizeof(IO) == 2) reinterpret_cast<uint16_t*>(op)[e] = (uint16_t)pack_bf16(y, 0.0f);
    else reinterpret_cast<float*>(op)[e] = y;
  }
  if (a.lse && e == 0) a.lse[row] = l > 0.0f ? (m + __builtin_amdgcn_logf(l)) * kLn2 : -INFINITY;
}

constexpr int TARGET_WAVES = 4096;  // 16 waves for each of the 256 CUs
constexpr int MIN_SHARE = 64;       // keys of a split that are worth one
constexpr int MAX_SPLITS = 1024;

int splits_of(int64_t batch, int q_heads, const ssm_kv_cache* c, int64_t table_width) {
  const int64_t groups = (q_heads / c->kv_heads + COLS - 1) / COLS;
  const int64_t have = batch * c->kv_heads * groups, longest = table_width * c->page_size;
  int64_t s = (TARGET_WAVES + have - 1) / have;
  const int64_t most = (longest + MIN_SHARE - 1) / MIN_SHARE;
  if (s > most) s = most;
  if (s > MAX_SPLITS) s = MAX_SPLITS;
  return (int)(s < 1 ? 1 : s);
}

template <typename IO, int KV, int DP>
hipError_t launch_dp(const DecodeArgs& a, hipStream_t s) {
  constexpr int CS = KV == SSM_KV_IO ? sizeof(IO) : 1;
  constexpr int NW = STEP * DP * CS * 4 <= 65536 ? 4 : 2;  // 64 KB of LDS
  const dim3 grid((a.splits + NW - 1) / NW, a.c.heads * a.groups, a.B), tb(NW * 64);
  attn_decode<IO, KV, DP, NW><<<grid, tb, 0, s>>>(a);
  hipError_t e = hipGetLastError();
  if (e == hipSuccess && a.splits > 1) {
    attn_decode_join<IO><<<dim3((unsigned)((int64_t)a.B * a.Hq)), dim3(256), 0, s>>>(a);
    e = hipGetLastError();
  }
  return e;
}

template <typename IO, int KV>
hipError_t launch_kv(const DecodeArgs& a, hipStream_t s) {
  if (a.c.D <= 64) return launch_dp<IO, KV, 64>(a, s);
  if (a.c.D <= 128) return launch_dp<IO, KV, 128>(a, s);
  if (a.c.D <= 192) return launch_dp<IO, KV, 192>(a, s);
  return launch_dp<IO, KV, 256>(a, s);
}

template <typename IO>
hipError_t launch_decode_attn(const DecodeArgs& a, int kv, hipStream_t s) {
  if (kv == SSM_KV_IO) return launch_kv<IO, SSM_KV_IO>(a, s);
  if (kv == SSM_KV_I8) return launch_kv<IO, SSM_KV_I8>(a, s);
  return launch_kv<IO, SSM_KV_E4M3>(a, s);
}

// Sizes of a decode call.
int check_decode_sizes(int64_t batch, int32_t q_heads, const ssm_kv_cache* c, int64_t table_width) {
  if (const int st = check_heads(q_heads, c->head_dim)) return st;
  if (const int st = check_heads(c->kv_heads, c->head_dim)) return st;
  if (q_heads % c->kv_heads) return SSM_ERR_SHAPE;
  if (batch < 1 || batch > SSM_ATTN_MAX_BATCH) return SSM_ERR_SHAPE;
  if (c->page_size < SSM_KV_MIN_PAGE || c->page_size > SSM_KV_MAX_PAGE || (c->page_size & (c->page_size - 1)))
    return SSM_ERR_SHAPE;
  // a sequence's keys, rounded up to steps and shares, stay below 2^31
  if (table_width < 1 || table_width > ((int64_t)INT32_MAX - (1 << 20)) / c->page_size) return SSM_ERR_SHAPE;
  return SSM_OK;
}

}  // namespace
}  // namespace attn
}  // namespace ssm

extern "C" {

size_t ssm_attn_decode_workspace_bytes(int64_t batch, int32_t q_heads, const ssm_kv_cache* cache,
                                       int64_t table_width) {
  using namespace ssm::attn;
  if (!cache || check_decode_sizes(batch, q_heads, cache, table_width) != SSM_OK) return 0;
  const int s = splits_of(batch, q_heads, cache, table_width);
  return s == 1 ? 0 : (size_t)batch * q_heads * s * (cache->head_dim + 2) * sizeof(float);
}

int ssm_attn_decode_step(int64_t batch, int32_t q_heads, int32_t io_dtype, float scale, const ssm_kv_cache* cache,
                         const ssm_view* q, const int32_t* table, int64_t table_width, const int32_t* lens,
                         const ssm_view* out, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  using namespace ssm::attn;
  int64_t es, cs;
  if (const int st = check_io(io_dtype, &es)) return st;
  if (const int st = check_cache(cache, es, &cs)) return st;
  if (const int st = check_decode_sizes(batch, q_heads, cache, table_width)) return st;
  if (!isfinite(scale) || !(scale > 0.0f)) return SSM_ERR_SHAPE;
  if (!table || !lens) return SSM_ERR_NULL;
  if (const int st = check_view(q, es)) return st;
  if (const int st = check_view(out, es)) return st;
  if (!aligned(table, 4) || !aligned(lens, 4) || !aligned(lse, 4)) return SSM_ERR_ALIGN;
  const size_t need = ssm_attn_decode_workspace_bytes(batch, q_heads, cache, table_width);
  if (need && (!workspace || workspace_bytes < need)) return SSM_ERR_WORKSPACE;
  if (need && !aligned(workspace, 16)) return SSM_ERR_ALIGN;
  const int64_t B = batch, D = cache->head_dim, H = q_heads;
  if (!writable(out, B, H, D) || views_overlap(out, B, H, q, B, H, D, es)) return SSM_ERR_ALIAS;
  const Span so = view_span(out, B, H, D, es), sl = span(lse, lse ? B * H * 4 : 0), sw = span(workspace, (int64_t)need);
  const Span ins[3] = {view_span(q, B, H, D, es), span(table, B * table_width * 4), span(lens, B * 4)};
  const CacheSpans spans = cache_spans(cache, cs);
  if (overlaps(so, sl) || overlaps(so, sw) || overlaps(sl, sw)) return SSM_ERR_ALIAS;
  if (overlaps(so, ins[1]) || overlaps(so, ins[2])) return SSM_ERR_ALIAS;
  for (const Span& s : ins)
    if (overlaps(sl, s) || overlaps(sw, s)) return SSM_ERR_ALIAS;
  if (cache_overlaps(spans, so) || cache_overlaps(spans, sl) || cache_overlaps(spans, sw)) return SSM_ERR_ALIAS;
  DecodeArgs a = {};
  a.q = bytes_view(q, es);
  a.out = bytes_view(out, es);
  a.lse = lse;
  a.c = cache_of(cache);
  a.table = table;
  a.lens = lens;
  a.W = table_width;
  a.B = (int)batch;
  a.Hq = q_heads;
  a.G = q_heads / cache->kv_heads;
  a.groups = (a.G + COLS - 1) / COLS;
  a.splits = splits_of(batch, q_heads, cache, table_width);
  a.scale_log2 = scale * 1.4426950408889634f;
  if (!isfinite(a.scale_log2) || !(a.scale_log2 > 0.0f)) return SSM_ERR_SHAPE;
  a.po = static_cast<float*>(workspace);
  a.ml = a.po + (int64_t)batch * q_heads * a.splits * cache->head_dim;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const hipError_t e = io_dtype == SSM_BF16 ? launch_decode_attn<ssm::bf16_t>(a, cache->kv_dtype, s)
                                            : launch_decode_attn<float>(a, cache->kv_dtype, s);
  return e == hipSuccess ? SSM_OK : SSM_ERR_LAUNCH;
}

}  // extern "C"
