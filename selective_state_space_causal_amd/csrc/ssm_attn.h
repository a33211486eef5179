// ssm_attn.h -- what the attention kernels (ssm_kv.hip, ssm_attn_prefill.hip, ssm_attn_decode.hip)
// share: views, vector types, conversions and the host-side checks of include/ssm_attn.h.
#pragma once
#include <hip/hip_runtime.h>
#include <math.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/ssm_attn.h"
#include "ssm_device.h"

namespace ssm {
namespace attn {

typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
// Rows of 8-bit codes start on 8-byte boundaries (head_dim is a multiple of 8): wider accesses
// are declared with the alignment they have; the hardware needs 4 bytes.
typedef unsigned u32x2_a4 __attribute__((ext_vector_type(2), aligned(4)));
typedef unsigned u32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));

struct View {
  char* p;
  int64_t ts, hs;  // strides in bytes
};

inline View bytes_view(const ssm_view* v, int64_t es) {
  if (!v) return View{nullptr, 0, 0};
  return View{static_cast<char*>(v->data), v->token_stride * es, v->head_stride * es};
}

struct Cache {
  char* k;
  char* v;
  float* ks;
  float* vs;
  int64_t slots;   // pages * page_size
  int page_shift;  // log2 page_size
  int heads;
  int D;
};

// Two fp32 values as a packed bf16 pair, rounded to nearest even (one v_cvt_pk_bf16_f32).
__device__ __forceinline__ unsigned pack_bf16(float lo, float hi) {
  bf16x2 r = {(__bf16)lo, (__bf16)hi};
  return __builtin_bit_cast(unsigned, r);
}

// The two 16-bit halves of a and b as pairs (a.lo, b.lo) and (a.hi, b.hi).
__device__ __forceinline__ unsigned pair_lo(unsigned a, unsigned b) { return __builtin_amdgcn_perm(b, a, 0x05040100u); }
__device__ __forceinline__ unsigned pair_hi(unsigned a, unsigned b) { return __builtin_amdgcn_perm(b, a, 0x07060302u); }

// ---- host-side checks: every one before any HIP call ----

inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

struct Span {
  uintptr_t lo, hi;
};
inline Span span(const void* p, int64_t bytes) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return Span{lo, lo + (uintptr_t)(bytes > 0 ? bytes : 0)};
}
inline bool overlaps(Span a, Span b) { return a.lo < b.hi && b.lo < a.hi; }

constexpr int64_t MAX_TOKENS = INT32_MAX;
// Largest strides in elements: 64 tokens of fp32 and 128 of bf16 stay within 2^31 bytes (a tile's offsets are 32-bit), and
// all byte counts within int64.
constexpr int64_t MAX_TOKEN_STRIDE = int64_t(1) << 23, MAX_HEAD_STRIDE = int64_t(1) << 48;

inline int check_io(int32_t io_dtype, int64_t* es) {
  if (io_dtype != SSM_F32 && io_dtype != SSM_BF16) return SSM_ERR_DTYPE;
  *es = io_dtype == SSM_BF16 ? 2 : 4;
  return SSM_OK;
}

inline int check_heads(int32_t heads, int32_t head_dim) {
  if (heads < 1 || heads > SSM_ATTN_MAX_HEADS) return SSM_ERR_SHAPE;
  if (head_dim < 8 || head_dim > SSM_ATTN_MAX_HEAD_DIM || head_dim % 8) return SSM_ERR_SHAPE;
  return SSM_OK;
}

inline int check_view(const ssm_view* v, int64_t es) {
  if (!v || !v->data) return SSM_ERR_NULL;
  if (v->token_stride < 0 || v->head_stride < 0 || v->token_stride > MAX_TOKEN_STRIDE ||
      v->head_stride > MAX_HEAD_STRIDE)
    return SSM_ERR_SHAPE;
  if (!aligned(v->data, 16) || v->token_stride * es % 16 || v->head_stride * es % 16) return SSM_ERR_ALIGN;
  return SSM_OK;
}

inline Span view_span(const ssm_view* v, int64_t tokens, int64_t heads, int64_t D, int64_t es) {
  return span(v->data, ((tokens - 1) * v->token_stride + (heads - 1) * v->head_stride + D) * es);
}

// Whether [pa, pa + wa) and [pb, pb + wb), each repeated at every multiple of `period` bytes, share no byte.
inline bool apart(const void* pa, int64_t wa, const void* pb, int64_t wb, int64_t period) {
  if (wa > period || wb > period) return false;
  const uintptr_t a = reinterpret_cast<uintptr_t>(pa), b = reinterpret_cast<uintptr_t>(pb);
  const int64_t off = b >= a ? (int64_t)((b - a) % (uintptr_t)period)
                             : (int64_t)((period - (int64_t)((a - b) % (uintptr_t)period)) % period);
  return off >= wa && off + wb <= period;  // b's starts past a's, and ends before a's next
}

// Whether two views may touch a common byte.  Views into one packed projection interleave without sharing one: whole
// rows of heads, token by token (q, k and v heads of a token in blocks: equal token strides), or single heads (each head's
// q, k and v next to one another: equal head strides, of which the token strides are multiples).
inline bool views_overlap(const ssm_view* a, int64_t ta, int64_t ha, const ssm_view* b, int64_t tb, int64_t hb,
                          int64_t D, int64_t es) {
  if (!overlaps(view_span(a, ta, ha, D, es), view_span(b, tb, hb, D, es))) return false;
  const int64_t ts = a->token_stride, hs = a->head_stride;
  if (ts == b->token_stride && ts > 0 &&
      apart(a->data, ((ha - 1) * hs + D) * es, b->data, ((hb - 1) * b->head_stride + D) * es, ts * es))
    return false;
  return !(hs == b->head_stride && hs > 0 && ts % hs == 0 && b->token_stride % hs == 0 &&
           apart(a->data, D * es, b->data, D * es, hs * es));
}

// Whether the rows that a view writes are disjoint (a stride of 0 or too small makes them overlap).
inline bool writable(const ssm_view* v, int64_t tokens, int64_t heads, int64_t D) {
  const int64_t ts = v->token_stride, hs = v->head_stride;
  if (heads > 1 && hs < D) return false;
  if (tokens > 1 && ts < D) return false;
  if (heads == 1 || tokens == 1) return true;
  return ts >= (heads - 1) * hs + D || hs >= (tokens - 1) * ts + D;
}

inline int check_cache(const ssm_kv_cache* c, int64_t es, int64_t* code_size) {
  if (!c || !c->k || !c->v) return SSM_ERR_NULL;
  if (const int st = check_heads(c->kv_heads, c->head_dim)) return st;
  if (c->page_size < SSM_KV_MIN_PAGE || c->page_size > SSM_KV_MAX_PAGE || (c->page_size & (c->page_size - 1)))
    return SSM_ERR_SHAPE;
  if (c->pages < 1 || c->pages > INT32_MAX) return SSM_ERR_SHAPE;
  if (c->kv_dtype != SSM_KV_IO && c->kv_dtype != SSM_KV_I8 && c->kv_dtype != SSM_KV_E4M3) return SSM_ERR_DTYPE;
  *code_size = c->kv_dtype == SSM_KV_IO ? es : 1;
  if (c->kv_dtype != SSM_KV_IO && (!c->k_scale || !c->v_scale)) return SSM_ERR_NULL;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 16) || !aligned(c->v_scale, 16))
    return SSM_ERR_ALIGN;
  return SSM_OK;
}

struct CacheSpans {
  Span s[4];
  int n;
};
inline CacheSpans cache_spans(const ssm_kv_cache* c, int64_t code_size) {
  const int64_t rows = c->pages * c->kv_heads * c->page_size;
  CacheSpans r;
  r.n = c->kv_dtype == SSM_KV_IO ? 2 : 4;
  r.s[0] = span(c->k, rows * c->head_dim * code_size);
  r.s[1] = span(c->v, rows * c->head_dim * code_size);
  r.s[2] = span(c->k_scale, rows * 4);
  r.s[3] = span(c->v_scale, rows * 4);
  return r;
}
inline bool cache_overlaps(const CacheSpans& c, Span s) {
  for (int i = 0; i < c.n; ++i)
    if (overlaps(c.s[i], s)) return true;
  return false;
}
inline bool cache_overlaps_itself(const CacheSpans& c) {
  for (int i = 0; i < c.n; ++i)
    for (int j = i + 1; j < c.n; ++j)
      if (overlaps(c.s[i], c.s[j])) return true;
  return false;
}

inline Cache cache_of(const ssm_kv_cache* c) {
  Cache r;
  r.k = static_cast<char*>(c->k);
  r.v = static_cast<char*>(c->v);
  r.ks = c->k_scale;
  r.vs = c->v_scale;
  r.slots = c->pages * c->page_size;
  r.page_shift = __builtin_ctz((unsigned)c->page_size);
  r.heads = c->kv_heads;
  r.D = c->head_dim;
  return r;
}

// The stream of a call whose checks are done.  An error that an earlier, unrelated call left behind is dropped, so that
// what hipGetLastError says after the launch is the launch's own.
inline hipStream_t ready(void* stream) {
  (void)hipGetLastError();
  return static_cast<hipStream_t>(stream);
}

}  // namespace attn
}  // namespace ssm
