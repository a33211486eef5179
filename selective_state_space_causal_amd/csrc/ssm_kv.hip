// ssm_kv.hip -- rotary positions and the paged key/value cache of include/ssm_attn.h.
//
// kv_rows does ssm_rope and ssm_kv_write: a workgroup takes some tokens, computes cos and sin of their
// pairs once into LDS (they are shared by all heads of a token), and walks the tokens' rows (q heads,
// k heads, v heads).  A row is held by LPR lanes, each with 2 * VW of its elements in registers:
// the two halves of VW rotated pairs, or 2 * VW neighbouring elements.  So a row is read once, rotated,
// its |x| maximum taken over the LPR lanes, quantised and written, without a second pass.  What bounds
// it is memory: each row is read and written once.
#include "ssm_attn.h"

namespace ssm {
namespace attn {
namespace {

constexpr int TPB = 256;
constexpr int MAX_ANGLES = 1024;  // cos / sin pairs of one workgroup's tokens in LDS (8 KB)
constexpr int64_t MAX_GRID = int64_t(1) << 20;  // keeps a launch within 2^28 work-items

struct RowArgs {
  View q, qo, k, ko, v;
  int64_t T;
  int Hq, Hk, Hv;
  int D, pairs, interleaved;
  float mscale;
  const int64_t* pos;
  const double* freq;
  Cache c;
  const int64_t* slots;
  int tpb;  // tokens of a workgroup
};

// cos and sin of position * freq.  The angle in turns is position * freq / (2 pi), kept as a sum of two
// fp64 (the products' rounding errors by fused multiply-adds, 1 / (2 pi) as two fp64), so reducing it
// to [-1/2, 1/2] loses nothing at any position below 2^53.  Then fp32, as the values that are turned are at most that: 2^-25 of
// half a turn is 9e-8 radians, and the result's error relative to fp64 grows from 4.2e-8 (cos and sin in fp64, rounded) to 5.3e-8.
__device__ __forceinline__ void angle(int64_t pos, double freq, float mscale, float& c, float& s) {
#pragma clang fp contract(off)  // each product below is rounded by itself: its error is taken from it
  constexpr double INV_HI = 0x1.45f306dc9c883p-3, INV_LO = -0x1.6b01ec5417056p-57;  // 1 / (2 pi)
  const double x = (double)pos, p = x * freq, pe = fma(x, freq, -p);
  const double t = p * INV_HI, te = fma(p, INV_HI, -t) + fma(p, INV_LO, pe * INV_HI);
  const float turns = (float)((t - rint(t)) + te);
  float sn, cs;
  sincospif(2.0f * turns, &sn, &cs);
  c = cs * mscale;
  s = sn * mscale;
}

// A pair turned by (c, s), each value one product and one fused multiply-add in every kernel: rope and kv_write give
// the same bits.
__device__ __forceinline__ void turn(float& x, float& y, float c, float s) {
  const float p = fmaf(x, c, -(y * s));
  y = fmaf(y, c, x * s);
  x = p;
}

template <typename IO, int VW>
__device__ __forceinline__ void load_vec(const char* p, float (&x)[VW]) {
  if constexpr (sizeof(IO) == 2) {
    if constexpr (VW == 1) {
      x[0] = to_f32(*reinterpret_cast<const bf16_t*>(p));
    } else {
      unsigned w[VW / 2];
      if constexpr (VW == 8) {
        const u32x4 t = *reinterpret_cast<const u32x4*>(p);
        w[0] = t[0], w[1] = t[1], w[2] = t[2], w[3] = t[3];
      } else {
        const u32x2 t = *reinterpret_cast<const u32x2*>(p);
        w[0] = t[0], w[1] = t[1];
      }
#pragma unroll
      for (int j = 0; j < VW / 2; ++j) {
        x[2 * j] = __uint_as_float(w[j] << 16);
        x[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
      }
    }
  } else {
    if constexpr (VW == 1) {
      x[0] = *reinterpret_cast<const float*>(p);
    } else {
#pragma unroll
      for (int j = 0; j < VW / 4; ++j) {
        const f32x4 t = reinterpret_cast<const f32x4*>(p)[j];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[4 * j + i] = t[i];
      }
    }
  }
}

template <typename IO, int VW>
__device__ __forceinline__ void store_vec(char* p, const float (&x)[VW]) {
  if constexpr (sizeof(IO) == 2) {
    if constexpr (VW == 1) {
      *reinterpret_cast<uint16_t*>(p) = (uint16_t)pack_bf16(x[0], 0.0f);
    } else if constexpr (VW == 4) {
      *reinterpret_cast<u32x2*>(p) = u32x2{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3])};
    } else {
      *reinterpret_cast<u32x4*>(p) =
          u32x4{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7])};
    }
  } else {
    if constexpr (VW == 1) {
      *reinterpret_cast<float*>(p) = x[0];
    } else {
#pragma unroll
      for (int j = 0; j < VW / 4; ++j)
        reinterpret_cast<f32x4*>(p)[j] = f32x4{x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]};
    }
  }
}

// Rounded to the io dtype and widened again.
template <typename IO>
__device__ __forceinline__ float through_io(float x) {
  if constexpr (sizeof(IO) == 2)
    return __uint_as_float(pack_bf16(x, 0.0f) << 16);
  else
    return x;
}

// Four scaled values as four codes.
template <int KV>
__device__ __forceinline__ unsigned codes4(float a, float b, float c, float d) {
  if constexpr (KV == SSM_KV_I8) {
    const auto one = [](float x) { return (unsigned)(int)rintf(fminf(fmaxf(x, -127.0f), 127.0f)) & 0xFFu; };
    return one(a) | one(b) << 8 | one(c) << 16 | one(d) << 24;
  } else {
    const auto in = [](float x) { return fminf(fmaxf(x, -448.0f), 448.0f); };
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(in(a), in(b), 0, false);
    return (unsigned)__builtin_amdgcn_cvt_pk_fp8_f32(in(c), in(d), w, true);
  }
}

template <int KV, int VW>
__device__ __forceinline__ void store_codes(char* p, const float (&x)[VW], float m) {
  if constexpr (VW == 1) {
    *p = (char)codes4<KV>(x[0] * m, 0.0f, 0.0f, 0.0f);
  } else if constexpr (VW == 4) {
    *reinterpret_cast<unsigned*>(p) = codes4<KV>(x[0] * m, x[1] * m, x[2] * m, x[3] * m);
  } else {
    *reinterpret_cast<u32x2_a4*>(p) = u32x2{codes4<KV>(x[0] * m, x[1] * m, x[2] * m, x[3] * m),
                                            codes4<KV>(x[4] * m, x[5] * m, x[6] * m, x[7] * m)};
  }
}

// LPR: lanes of a row, a power of two with LPR * NIT * 2 VW >= D.
template <typename IO, int VW, int KV, bool ROPE, bool CACHE, int LPR, int NIT>
__global__ __launch_bounds__(TPB) void kv_rows(RowArgs a) {
  constexpr int ES = sizeof(IO);
  __shared__ float cs[ROPE ? MAX_ANGLES : 1], sn[ROPE ? MAX_ANGLES : 1];
  const int lig = threadIdx.x % LPR, group = threadIdx.x / LPR;
  const int nrow = a.Hq + a.Hk + a.Hv, units = a.D / (2 * VW), rot_units = ROPE ? a.pairs / VW : 0;
  for (int64_t t0 = (int64_t)blockIdx.x * a.tpb; t0 < a.T; t0 += (int64_t)gridDim.x * a.tpb) {
    const int ntok = (int)(a.T - t0 < a.tpb ? a.T - t0 : a.tpb);
    if constexpr (ROPE) {
      __syncthreads();
      for (int i = threadIdx.x; i < ntok * a.pairs; i += TPB) {
        const int tok = i / a.pairs;
        angle(a.pos[t0 + tok], a.freq[i - tok * a.pairs], a.mscale, cs[i], sn[i]);
      }
      __syncthreads();
    }
    for (int r = group; r < ntok * nrow; r += TPB / LPR) {
      const int tok = r / nrow, h = r - tok * nrow;
      const int64_t t = t0 + tok;
      const bool is_q = h < a.Hq, is_k = !is_q && h < a.Hq + a.Hk;
      const int hh = is_q ? h : is_k ? h - a.Hq : h - a.Hq - a.Hk;
      const View& src = is_q ? a.q : is_k ? a.k : a.v;
      const char* sp = src.p + t * src.ts + hh * src.hs;
      float xa[NIT][VW], xb[NIT][VW];
      int at[NIT], bt[NIT];
      float amax = 0.0f;
#pragma unroll
      for (int n = 0; n < NIT; ++n) {
        const int u = lig + n * LPR;
        const bool in = u < units, rot = ROPE && u < rot_units && (is_q || is_k);
        const bool apart = rot && !a.interleaved;
        at[n] = apart ? u * VW : 2 * u * VW;
        bt[n] = apart ? a.pairs + u * VW : (2 * u + 1) * VW;
        if (!in) continue;
        load_vec<IO, VW>(sp + at[n] * ES, xa[n]);
        load_vec<IO, VW>(sp + bt[n] * ES, xb[n]);
        if (rot) {
          const float* c = cs + tok * a.pairs + u * VW;
          const float* s = sn + tok * a.pairs + u * VW;
          if (a.interleaved) {
            float y[2 * VW];
#pragma unroll
            for (int j = 0; j < VW; ++j) y[j] = xa[n][j], y[VW + j] = xb[n][j];
#pragma unroll
            for (int j = 0; j < VW; ++j) turn(y[2 * j], y[2 * j + 1], c[j], s[j]);
#pragma unroll
            for (int j = 0; j < VW; ++j) xa[n][j] = y[j], xb[n][j] = y[VW + j];
          } else {
#pragma unroll
            for (int j = 0; j < VW; ++j) turn(xa[n][j], xb[n][j], c[j], s[j]);
          }
        }
      }
      if (is_q || (is_k && a.ko.p)) {  // rotated rows in the io dtype
        const View& dst = is_q ? a.qo : a.ko;
        char* dp = dst.p + t * dst.ts + hh * dst.hs;
#pragma unroll
        for (int n = 0; n < NIT; ++n)
          if (lig + n * LPR < units) {
            store_vec<IO, VW>(dp + at[n] * ES, xa[n]);
            store_vec<IO, VW>(dp + bt[n] * ES, xb[n]);
          }
      }
      if constexpr (CACHE) {
        if (is_q) continue;
        const int64_t slot = a.slots[t];
        if (slot < 0 || slot >= a.c.slots) continue;
        const int64_t page = slot >> a.c.page_shift, off = slot & ((1 << a.c.page_shift) - 1);
        const int64_t row = ((page * a.Hk + hh) << a.c.page_shift) + off;
        char* base = is_k ? a.c.k : a.c.v;
        if constexpr (KV == SSM_KV_IO) {
          char* dp = base + row * a.D * ES;
#pragma unroll
          for (int n = 0; n < NIT; ++n)
            if (lig + n * LPR < units) {
              store_vec<IO, VW>(dp + at[n] * ES, xa[n]);
              store_vec<IO, VW>(dp + bt[n] * ES, xb[n]);
            }
        } else {
#pragma unroll
          for (int n = 0; n < NIT; ++n)
            if (lig + n * LPR < units) {
#pragma unroll
              for (int j = 0; j < VW; ++j) {
                if constexpr (ROPE) xa[n][j] = through_io<IO>(xa[n][j]), xb[n][j] = through_io<IO>(xb[n][j]);
                amax = fmaxf(amax, fmaxf(fabsf(xa[n][j]), fabsf(xb[n][j])));
              }
            }
#pragma unroll
          for (int m = 1; m < LPR; m <<= 1) amax = fmaxf(amax, __shfl_xor(amax, m));
          constexpr float TOP = KV == SSM_KV_I8 ? 127.0f : 448.0f;
          const bool live = amax >= 0x1p-100f;
          const float m = live ? (1.0f / amax) * TOP : 0.0f;
          char* dp = base + row * a.D;
#pragma unroll
          for (int n = 0; n < NIT; ++n)
            if (lig + n * LPR < units) {
              store_codes<KV, VW>(dp + at[n], xa[n], m);
              store_codes<KV, VW>(dp + bt[n], xb[n], m);
            }
          if (lig == 0) (is_k ? a.c.ks : a.c.vs)[row] = live ? amax * (1.0f / TOP) : 0.0f;
        }
      }
    }
  }
}

template <typename IO, int KV, bool ROPE, bool CACHE>
hipError_t launch_rows(RowArgs& a, hipStream_t s) {
  // The widest vectors that the pairs and the rest of a head divide into: 8 elements where pairs and
  // D / 2 - pairs are multiples of 8 (16 bytes of bf16), else 4, else single elements.
  const int rest = a.D / 2 - a.pairs;
  const int vw = a.pairs % 8 == 0 && rest % 8 == 0 ? 8 : a.pairs % 4 == 0 && rest % 4 == 0 ? 4 : 1;
  // Tokens of a workgroup: up to 8 while that leaves four workgroups for each of the 256 CUs, and no more than the
  // angle table holds.  Token by token the rows of a packed projection are read in memory's order: 32768 tokens take 45 us
  // written (8 + 8 heads, int8) and 35 us rotated (8 + 2 heads); head by head, 16 or 32 tokens at a time, 48 to 58 and 40,
  // though the cache's lines are then written whole.
  const int cap = ROPE ? MAX_ANGLES / a.pairs : 16;
  int tpb = 1;
  while (tpb * 2 <= cap && tpb < 8 && a.T / (tpb * 2) >= 1024) tpb *= 2;
  a.tpb = tpb;
  const int64_t want = (a.T + tpb - 1) / tpb;
  const dim3 grid((unsigned)(want < MAX_GRID ? want : MAX_GRID)), tb(TPB);
  const int units = a.D / (2 * vw);
  if (vw == 8) {
    if (units <= 8) kv_rows<IO, 8, KV, ROPE, CACHE, 8, 1><<<grid, tb, 0, s>>>(a);
    else kv_rows<IO, 8, KV, ROPE, CACHE, 16, 1><<<grid, tb, 0, s>>>(a);
  } else if (vw == 4) {
    if (units <= 16) kv_rows<IO, 4, KV, ROPE, CACHE, 16, 1><<<grid, tb, 0, s>>>(a);
    else kv_rows<IO, 4, KV, ROPE, CACHE, 32, 1><<<grid, tb, 0, s>>>(a);
  } else {
    kv_rows<IO, 1, KV, ROPE, CACHE, 64, 2><<<grid, tb, 0, s>>>(a);
  }
  return hipGetLastError();
}

template <typename IO>
hipError_t launch_write(RowArgs& a, int kv, bool rope, hipStream_t s) {
  if (rope) {
    if (kv == SSM_KV_IO) return launch_rows<IO, SSM_KV_IO, true, true>(a, s);
    if (kv == SSM_KV_I8) return launch_rows<IO, SSM_KV_I8, true, true>(a, s);
    return launch_rows<IO, SSM_KV_E4M3, true, true>(a, s);
  }
  if (kv == SSM_KV_IO) return launch_rows<IO, SSM_KV_IO, false, true>(a, s);
  if (kv == SSM_KV_I8) return launch_rows<IO, SSM_KV_I8, false, true>(a, s);
  return launch_rows<IO, SSM_KV_E4M3, false, true>(a, s);
}

// ---- reading back ----

constexpr int HEADS = 4;  // heads of a workgroup (65536 tokens, 8 + 8 heads: 1 95 us, 2 77.5, 4 76.7, 8 79)

struct ReadArgs {
  View k, v;
  Cache c;
  const int64_t* slots;
  int64_t T;
};

// Eight codes times the row's scale.
template <int KV>
__device__ __forceinline__ void widen8(u32x2 w, float s, float (&x)[8]) {
  if constexpr (KV == SSM_KV_I8) {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = (float)(int8_t)(w[j / 4] >> (8 * (j % 4))) * s;
  } else {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[j], false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[j], true);
      x[4 * j] = lo[0] * s, x[4 * j + 1] = lo[1] * s, x[4 * j + 2] = hi[0] * s, x[4 * j + 3] = hi[1] * s;
    }
  }
}

// LPR lanes read a row, eight elements each; a workgroup has TPB / LPR neighbouring tokens, which mostly lie
// side by side in the cache (whole lines of codes and of scales), and HEADS heads of them at once.  Memory bounds
// it: 65536 tokens of 8 heads of 128 from int8 to bf16 take 77 us, 5.3 TB/s (a large copy here does 4.8).
template <typename IO, int KV, int LPR>
__global__ __launch_bounds__(TPB) void kv_read_rows(ReadArgs a) {
  constexpr int TOK = TPB / LPR;
  const int lig = threadIdx.x % LPR, nrow = 2 * a.c.heads, parts = (nrow + HEADS - 1) / HEADS;
  if (lig >= a.c.D / 8) return;
  const int64_t blocks = (a.T + TOK - 1) / TOK * parts;
  for (int64_t u = blockIdx.x; u < blocks; u += gridDim.x) {
    const int64_t block = u / parts, t = block * TOK + threadIdx.x / LPR;
    const int h0 = (int)(u - block * parts) * HEADS;
    if (t >= a.T) continue;
    const int64_t slot = a.slots[t];
    const bool held = slot >= 0 && slot < a.c.slots;
    const int64_t page = held ? slot >> a.c.page_shift : 0, off = held ? slot & ((1 << a.c.page_shift) - 1) : 0;
    u32x4 w[HEADS][KV == SSM_KV_IO ? sizeof(IO) / 2 : 1];
    float scale[HEADS];
#pragma unroll
    for (int i = 0; i < HEADS; ++i) {  // every load first; heads past the last repeat it
      const int h = min(h0 + i, nrow - 1);
      const bool is_k = h < a.c.heads;
      const int64_t row = ((page * a.c.heads + (is_k ? h : h - a.c.heads)) << a.c.page_shift) + off;
      const char* p = (is_k ? a.c.k : a.c.v) + (row * a.c.D + lig * 8) * (KV == SSM_KV_IO ? (int)sizeof(IO) : 1);
      if constexpr (KV == SSM_KV_IO) {
#pragma unroll
        for (int j = 0; j < (int)sizeof(IO) / 2; ++j) w[i][j] = reinterpret_cast<const u32x4*>(p)[j];
      } else {
        const u32x2 x = *reinterpret_cast<const u32x2_a4*>(p);
        w[i][0][0] = x[0], w[i][0][1] = x[1];
        scale[i] = (is_k ? a.c.ks : a.c.vs)[row];
      }
    }
#pragma unroll
    for (int i = 0; i < HEADS; ++i) {
      const int h = h0 + i;
      if (h >= nrow) break;
      const bool is_k = h < a.c.heads;
      const View& dst = is_k ? a.k : a.v;
      char* dp = dst.p + t * dst.ts + (is_k ? h : h - a.c.heads) * dst.hs + lig * 8 * (int)sizeof(IO);
      if constexpr (KV == SSM_KV_IO) {
#pragma unroll
        for (int j = 0; j < (int)sizeof(IO) / 2; ++j)
          reinterpret_cast<u32x4*>(dp)[j] = held ? w[i][j] : u32x4{0, 0, 0, 0};
      } else {
        float x[8];
        widen8<KV>(u32x2{w[i][0][0], w[i][0][1]}, scale[i], x);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = held ? x[j] : 0.0f;
        store_vec<IO, 8>(dp, x);
      }
    }
  }
}

template <typename IO, int KV>
hipError_t launch_read(const ReadArgs& a, hipStream_t s) {
  const int units = a.c.D / 8;
  const int lpr = units <= 8 ? 8 : units <= 16 ? 16 : 32, tok = TPB / lpr;
  const int64_t want = (a.T + tok - 1) / tok * ((2 * a.c.heads + HEADS - 1) / HEADS);
  const dim3 grid((unsigned)(want < MAX_GRID ? want : MAX_GRID)), tb(TPB);
  if (lpr == 8) kv_read_rows<IO, KV, 8><<<grid, tb, 0, s>>>(a);
  else if (lpr == 16) kv_read_rows<IO, KV, 16><<<grid, tb, 0, s>>>(a);
  else kv_read_rows<IO, KV, 32><<<grid, tb, 0, s>>>(a);
  return hipGetLastError();
}

int check_rope(const ssm_rope_desc* r, int32_t head_dim) {
  if (!r || !r->positions || !r->freq) return SSM_ERR_NULL;
  if (r->pairs < 1 || 2 * (int64_t)r->pairs > head_dim || !isfinite(r->mscale)) return SSM_ERR_SHAPE;
  if (r->interleaved != 0 && r->interleaved != 1) return SSM_ERR_SHAPE;
  if (!aligned(r->positions, 8) || !aligned(r->freq, 8)) return SSM_ERR_ALIGN;
  return SSM_OK;
}

bool same_view(const ssm_view* a, const ssm_view* b) {
  return a->data == b->data && a->token_stride == b->token_stride && a->head_stride == b->head_stride;
}

void set_rope(RowArgs& a, const ssm_rope_desc* r) {
  a.pairs = r->pairs;
  a.interleaved = r->interleaved;
  a.mscale = r->mscale;
  a.pos = r->positions;
  a.freq = r->freq;
}

}  // namespace
}  // namespace attn
}  // namespace ssm

extern "C" {

int ssm_rope(int64_t tokens, int32_t q_heads, int32_t k_heads, int32_t head_dim, int32_t io_dtype,
             const ssm_rope_desc* rope, const ssm_view* q, const ssm_view* q_out, const ssm_view* k,
             const ssm_view* k_out, void* stream) {
  using namespace ssm::attn;
  int64_t es;
  if (tokens < 0 || tokens > MAX_TOKENS) return SSM_ERR_SHAPE;
  if (const int st = check_io(io_dtype, &es)) return st;
  if (const int st = check_heads(q_heads, head_dim)) return st;
  if (k_heads < 0 || k_heads > SSM_ATTN_MAX_HEADS) return SSM_ERR_SHAPE;
  if (!rope) return SSM_ERR_NULL;
  if (tokens == 0) return SSM_OK;
  if (const int st = check_rope(rope, head_dim)) return st;
  if (const int st = check_view(q, es)) return st;
  if (const int st = check_view(q_out, es)) return st;
  if (k_heads) {
    if (const int st = check_view(k, es)) return st;
    if (const int st = check_view(k_out, es)) return st;
  }
  const int64_t T = tokens, D = head_dim;
  if (!writable(q_out, T, q_heads, D) || (k_heads && !writable(k_out, T, k_heads, D))) return SSM_ERR_ALIAS;
  if (!same_view(q, q_out) && views_overlap(q, T, q_heads, q_out, T, q_heads, D, es)) return SSM_ERR_ALIAS;
  if (k_heads) {
    if (!same_view(k, k_out) && views_overlap(k, T, k_heads, k_out, T, k_heads, D, es)) return SSM_ERR_ALIAS;
    if (views_overlap(q_out, T, q_heads, k_out, T, k_heads, D, es) || views_overlap(q_out, T, q_heads, k, T, k_heads, D, es) ||
        views_overlap(q, T, q_heads, k_out, T, k_heads, D, es))
      return SSM_ERR_ALIAS;
  }
  const ssm_view* outs[2] = {q_out, k_heads ? k_out : nullptr};
  for (int i = 0; i < 2; ++i) {
    if (!outs[i]) continue;
    const Span so = view_span(outs[i], T, i ? k_heads : q_heads, D, es);
    if (overlaps(so, span(rope->positions, T * 8)) || overlaps(so, span(rope->freq, rope->pairs * (int64_t)8)))
      return SSM_ERR_ALIAS;
  }
  RowArgs a = {};
  a.q = bytes_view(q, es);
  a.qo = bytes_view(q_out, es);
  if (k_heads) {
    a.k = bytes_view(k, es);
    a.ko = bytes_view(k_out, es);
  }
  a.T = T;
  a.Hq = q_heads;
  a.Hk = k_heads;
  a.D = head_dim;
  set_rope(a, rope);
  const hipStream_t s = ready(stream);
  const hipError_t e = io_dtype == SSM_BF16 ? launch_rows<ssm::bf16_t, SSM_KV_IO, true, false>(a, s)
                                            : launch_rows<float, SSM_KV_IO, true, false>(a, s);
  return e == hipSuccess ? SSM_OK : SSM_ERR_LAUNCH;
}

int ssm_kv_write(int64_t tokens, int32_t io_dtype, const ssm_kv_cache* cache, const int64_t* slots,
                 const ssm_view* k, const ssm_view* v, const ssm_rope_desc* rope, int32_t q_heads,
                 const ssm_view* q, const ssm_view* q_out, const ssm_view* k_out, void* stream) {
  using namespace ssm::attn;
  int64_t es, cs;
  if (tokens < 0 || tokens > MAX_TOKENS) return SSM_ERR_SHAPE;
  if (const int st = check_io(io_dtype, &es)) return st;
  if (const int st = check_cache(cache, es, &cs)) return st;
  if (q_heads < 0 || q_heads > SSM_ATTN_MAX_HEADS) return SSM_ERR_SHAPE;
  if (!rope && (q_heads || k_out)) return SSM_ERR_SHAPE;
  if (tokens == 0) return SSM_OK;
  const int64_t T = tokens, D = cache->head_dim, H = cache->kv_heads;
  if (!slots) return SSM_ERR_NULL;
  if (const int st = check_view(k, es)) return st;
  if (const int st = check_view(v, es)) return st;
  if (rope)
    if (const int st = check_rope(rope, cache->head_dim)) return st;
  if (q_heads) {
    if (const int st = check_view(q, es)) return st;
    if (const int st = check_view(q_out, es)) return st;
  }
  if (k_out)
    if (const int st = check_view(k_out, es)) return st;
  if (!aligned(slots, 8)) return SSM_ERR_ALIGN;
  // outputs: the cache, q_out, k_out
  const CacheSpans spans = cache_spans(cache, cs);
  if (cache_overlaps_itself(spans)) return SSM_ERR_ALIAS;
  const Span ins[4] = {span(slots, T * 8), rope ? span(rope->positions, T * 8) : Span{0, 0},
                       rope ? span(rope->freq, rope->pairs * (int64_t)8) : Span{0, 0}, Span{0, 0}};
  for (const Span& s : ins)
    if (cache_overlaps(spans, s)) return SSM_ERR_ALIAS;
  if (cache_overlaps(spans, view_span(k, T, H, D, es)) || cache_overlaps(spans, view_span(v, T, H, D, es)))
    return SSM_ERR_ALIAS;
  struct Out {
    const ssm_view* o;
    const ssm_view* from;
    int64_t heads;
  } outs[2] = {{q_heads ? q_out : nullptr, q, q_heads}, {k_out, k, H}};
  if (q_heads && cache_overlaps(spans, view_span(q, T, q_heads, D, es))) return SSM_ERR_ALIAS;
  for (const Out& o : outs) {
    if (!o.o) continue;
    if (!writable(o.o, T, o.heads, D)) return SSM_ERR_ALIAS;
    const Span so = view_span(o.o, T, o.heads, D, es);
    if (cache_overlaps(spans, so)) return SSM_ERR_ALIAS;
    for (const Span& s : ins)
      if (overlaps(so, s)) return SSM_ERR_ALIAS;
    if (!same_view(o.o, o.from) && views_overlap(o.o, T, o.heads, o.from, T, o.heads, D, es)) return SSM_ERR_ALIAS;
    if (views_overlap(o.o, T, o.heads, v, T, H, D, es)) return SSM_ERR_ALIAS;
  }
  if (q_heads && views_overlap(q_out, T, q_heads, k, T, H, D, es)) return SSM_ERR_ALIAS;
  if (q_heads && k_out &&
      (views_overlap(q_out, T, q_heads, k_out, T, H, D, es) || views_overlap(q, T, q_heads, k_out, T, H, D, es)))
    return SSM_ERR_ALIAS;
  RowArgs a = {};
  a.k = bytes_view(k, es);
  a.v = bytes_view(v, es);
  a.ko = bytes_view(k_out, es);
  if (q_heads) {
    a.q = bytes_view(q, es);
    a.qo = bytes_view(q_out, es);
  }
  a.T = T;
  a.Hq = q_heads;
  a.Hk = a.Hv = cache->kv_heads;
  a.D = cache->head_dim;
  if (rope) set_rope(a, rope);
  a.c = cache_of(cache);
  a.slots = slots;
  const hipStream_t s = ready(stream);
  const hipError_t e = io_dtype == SSM_BF16 ? launch_write<ssm::bf16_t>(a, cache->kv_dtype, rope != nullptr, s)
                                            : launch_write<float>(a, cache->kv_dtype, rope != nullptr, s);
  return e == hipSuccess ? SSM_OK : SSM_ERR_LAUNCH;
}

int ssm_kv_read(int64_t tokens, int32_t io_dtype, const ssm_kv_cache* cache, const int64_t* slots,
                const ssm_view* k_out, const ssm_view* v_out, void* stream) {
  using namespace ssm::attn;
  int64_t es, cs;
  if (tokens < 0 || tokens > MAX_TOKENS) return SSM_ERR_SHAPE;
  if (const int st = check_io(io_dtype, &es)) return st;
  if (const int st = check_cache(cache, es, &cs)) return st;
  if (tokens == 0) return SSM_OK;
  if (!slots) return SSM_ERR_NULL;
  if (const int st = check_view(k_out, es)) return st;
  if (const int st = check_view(v_out, es)) return st;
  if (!aligned(slots, 8)) return SSM_ERR_ALIGN;
  const int64_t T = tokens, D = cache->head_dim, H = cache->kv_heads;
  const CacheSpans spans = cache_spans(cache, cs);
  const ssm_view* outs[2] = {k_out, v_out};
  for (const ssm_view* o : outs) {
    if (!writable(o, T, H, D)) return SSM_ERR_ALIAS;
    const Span so = view_span(o, T, H, D, es);
    if (cache_overlaps(spans, so) || overlaps(so, span(slots, T * 8))) return SSM_ERR_ALIAS;
  }
  if (views_overlap(k_out, T, H, v_out, T, H, D, es)) return SSM_ERR_ALIAS;
  ReadArgs a = {};
  a.k = bytes_view(k_out, es);
  a.v = bytes_view(v_out, es);
  a.c = cache_of(cache);
  a.slots = slots;
  a.T = T;
  const hipStream_t s = ready(stream);
  hipError_t e;
  if (io_dtype == SSM_BF16)
    e = cache->kv_dtype == SSM_KV_IO   ? launch_read<ssm::bf16_t, SSM_KV_IO>(a, s)
        : cache->kv_dtype == SSM_KV_I8 ? launch_read<ssm::bf16_t, SSM_KV_I8>(a, s)
                                       : launch_read<ssm::bf16_t, SSM_KV_E4M3>(a, s);
  else
    e = cache->kv_dtype == SSM_KV_IO   ? launch_read<float, SSM_KV_IO>(a, s)
        : cache->kv_dtype == SSM_KV_I8 ? launch_read<float, SSM_KV_I8>(a, s)
                                       : launch_read<float, SSM_KV_E4M3>(a, s);
  return e == hipSuccess ? SSM_OK : SSM_ERR_LAUNCH;
}

}  // extern "C"
