/*
 * ssm_attn.h -- C ABI of the attention operators that stand beside the selective-SSM mixer on
 * AMD Instinct MI355X (gfx950).  Part of libssm.so.
 *
 * Hybrid stacks put attention blocks between their selective-SSM mixers.  One rank's attention
 * block needs, between its projections (ssm_proj.h):
 *   ssm_rope               rotary positions of q and k
 *   ssm_kv_write           new keys and values into a paged cache, quantised as they are written,
 *                          with the rotation of q and k in the same pass where asked
 *   ssm_kv_read            cached keys and values back in the io dtype
 *   ssm_attn_prefill       softmax attention over packed prompts of different lengths
 *   ssm_attn_decode_step   one token per sequence against the paged cache
 * As with the scan (ssm.h) the cache is the caller's: prefill writes it, decode resumes from it.
 *
 * Formulas (T tokens; Hq query heads and Hkv key heads, Hq a multiple of Hkv; query head g reads
 * key head g / (Hq / Hkv); D = head_dim):
 *   rotation   pair i < pairs of a head holds (a, b) = (x[2i], x[2i+1]) (interleaved) or
 *              (x[i], x[i + pairs]) (half); with angle w = position * freq[i],
 *              (a, b) <- mscale * (a cos w - b sin w, b cos w + a sin w); the rest of the head
 *              stays as it is.  The angle is reduced as a sum of two fp64, so positions below 2^53
 *              keep their digits; the rest is fp32, rounded once to the io dtype.
 *   attention  s[i, j] = scale * <q_i, k_j>, o_i = sum_j e^(s_ij - m_i) v_j / sum_j e^(s_ij - m_i),
 *              m_i = max_j s_ij, over the keys j that query i sees; lse_i = m_i + ln(sum).  A query
 *              that sees no key gives o_i = 0 and lse_i = -inf.
 *   8-bit rows one fp32 scale per cached row (one token's key or value of one head):
 *              amax = max |x|, s = amax * (1 / top), m = (1 / amax) * top (each operation rounded
 *              to fp32), top = 127 (int8) or 448 (e4m3); code = clamp(x * m, -top, top) rounded to nearest
 *              even; value = code * s.  Rows with amax < 2^-100 get s = 0 and codes 0 (m would
 *              overflow).  x is the io-dtype value (a rotated key is rounded to the io dtype first).
 *
 * Views.  A [T, H, D] tensor is a base pointer with a token and a head stride in elements (the D
 * values of a head are contiguous), so the heads of a packed q/k/v projection are used in place.
 * Base pointers are 16-byte aligned and strides are multiples of 16 bytes, token strides in
 * [0, 2^23] elements, head strides in [0, 2^48].
 *
 * Cache.  k and v are [pages, Hkv, page_size, D] in kv_dtype and k_scale, v_scale
 * [pages, Hkv, page_size] fp32 (8-bit types; NULL otherwise).  page_size is a power of two in
 * [16, 1024].  A token's slot is page * page_size + its place in the page; slots outside
 * [0, pages * page_size) are skipped on write and read back as zeros.  kv_dtype SSM_KV_IO holds
 * the io dtype itself.
 *
 * head_dim is a multiple of 8 in [8, 256].  io dtypes: SSM_F32, SSM_BF16.  Products of bf16 inputs
 * run on the matrix cores with fp32 sums; for the product with v, prompt attention rounds a softmax weight
 * to bf16 (2^-8 relative, the size of the output's own rounding), and decode holds it as the sum of two bf16
 * (2^-17).  fp32 inputs keep fp32's accuracy throughout: prompt attention multiplies them as three bf16
 * parts each (what is left out is below 2^-25 of a product); decode against an 8-bit cache multiplies q and the
 * weights as three bf16 parts each (to 2^-27 of them) with the codes, which are exact, and against an fp32 cache on the fp32
 * matrix instructions.  What is split into parts (q, and k and v of a prompt) has magnitudes up to 2^127, and sums of
 * products stay below 2^128 before the scale of a cached row and `scale` are applied.  Softmax maxima, sums and the
 * partial results of a split are fp32.
 *
 * Conventions (ownership, ordering, errors before any HIP call, no allocation, no mutable global
 * state, no host synchronisation, the current device) as in ssm.h.  Index arrays (slots,
 * positions, cu_q, cu_k, table, lens) are device memory and are not seen by the host: values out
 * of range are clamped or skipped as stated at each call, never followed.  Non-finite values in
 * q, or in the keys and values that a sequence holds, are outside the contract; what lies in a
 * cache or tensor past a sequence's length is never used, whatever it holds.
 */
#ifndef SSM_ATTN_H
#define SSM_ATTN_H

#include <stddef.h>
#include <stdint.h>

#include "ssm.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SSM_ATTN_MAX_HEAD_DIM 256
#define SSM_ATTN_MAX_HEADS 1024    /* largest head count */
#define SSM_ATTN_MAX_BATCH 65535   /* most sequences of one call */
#define SSM_KV_MIN_PAGE 16
#define SSM_KV_MAX_PAGE 1024

typedef enum { SSM_KV_IO = 0, SSM_KV_I8 = 1, SSM_KV_E4M3 = 2 } ssm_kv_dtype;

/* A [T, H, D] tensor on the device; strides in elements. */
typedef struct {
  void* data;
  int64_t token_stride;
  int64_t head_stride;
} ssm_view;

typedef struct {
  void* k;           /* [pages, kv_heads, page_size, head_dim] */
  void* v;
  float* k_scale;    /* [pages, kv_heads, page_size], or NULL for SSM_KV_IO */
  float* v_scale;
  int64_t pages;
  int32_t page_size;
  int32_t kv_heads;
  int32_t head_dim;
  int32_t kv_dtype;  /* ssm_kv_dtype */
} ssm_kv_cache;

typedef struct {
  const int64_t* positions; /* device [T] */
  const double* freq;       /* device [pairs]: radians per position */
  int32_t pairs;            /* rotated pairs of a head, 1 <= pairs, 2 * pairs <= head_dim */
  int32_t interleaved;      /* 0: pairs (i, i + pairs); 1: pairs (2i, 2i + 1) */
  float mscale;             /* factor on cos and sin (1 = none) */
} ssm_rope_desc;

/*
 * Rotate q [T, q_heads, D] into q_out and k [T, k_heads, D] into k_out.  q_out may be q itself and
 * k_out k (in place: same data and strides); no other overlap of an output is allowed.  k_heads 0
 * with NULL views: q alone.  tokens 0 is a call that does nothing.
 */
int ssm_rope(int64_t tokens, int32_t q_heads, int32_t k_heads, int32_t head_dim, int32_t io_dtype,
             const ssm_rope_desc* rope, const ssm_view* q, const ssm_view* q_out, const ssm_view* k,
             const ssm_view* k_out, void* stream);

/*
 * Write the keys and values of T tokens (k, v [T, kv_heads, D]) to the slots of the cache.
 * With rope, keys are rotated on the way (and stored in k_out too where it is given), and q
 * [T, q_heads, D] is rotated into q_out in the same launch (q_heads 0: no q).  Without rope, q_heads
 * is 0 and k_out NULL.  Two tokens with the same slot race: undefined which of them is kept.
 */
int ssm_kv_write(int64_t tokens, int32_t io_dtype, const ssm_kv_cache* cache, const int64_t* slots,
                 const ssm_view* k, const ssm_view* v, const ssm_rope_desc* rope, int32_t q_heads,
                 const ssm_view* q, const ssm_view* q_out, const ssm_view* k_out, void* stream);

/* Read the rows at T slots back: k_out, v_out [T, kv_heads, D] in io_dtype (for SSM_KV_IO the cache's own). */
int ssm_kv_read(int64_t tokens, int32_t io_dtype, const ssm_kv_cache* cache, const int64_t* slots,
                const ssm_view* k_out, const ssm_view* v_out, void* stream);

typedef struct {
  int64_t batch;     /* sequences, 1 .. SSM_ATTN_MAX_BATCH */
  int64_t q_tokens;  /* tokens of q and out (all sequences); q_tokens * (q_heads / kv_heads) <= 2^30 - 32 */
  int64_t k_tokens;  /* tokens of k and v, below 2^31 - 2^20 */
  int32_t q_heads;
  int32_t kv_heads;
  int32_t head_dim;
  int32_t io_dtype;
  int32_t causal;    /* 1: the last query of a sequence sees its last key, the one before one key less, ... */
  float scale;       /* factor on the products, finite and > 0 */
} ssm_attn_dims;

/*
 * Attention over packed sequences.  cu_q, cu_k: device int32 [batch + 1], ascending from 0: sequence b
 * holds q rows cu_q[b] .. cu_q[b+1] - 1 and k, v rows cu_k[b] .. cu_k[b+1] - 1 (either may be empty;
 * with more keys than queries the queries are the sequence's last tokens, a prompt's next chunk).
 * Entries are clamped to [0, tokens].  Rows of no sequence are left untouched.
 * out [q_tokens, q_heads, D]; lse fp32 [q_tokens, q_heads] or NULL.  out and lse may not overlap the
 * inputs or each other.
 */
int ssm_attn_prefill(const ssm_attn_dims* dims, const ssm_view* q, const ssm_view* k, const ssm_view* v,
                     const int32_t* cu_q, const int32_t* cu_k, const ssm_view* out, float* lse, void* stream);

/* Device workspace in bytes that ssm_attn_decode_step needs (0 = none, or invalid sizes). */
size_t ssm_attn_decode_workspace_bytes(int64_t batch, int32_t q_heads, const ssm_kv_cache* cache,
                                       int64_t table_width);

/*
 * One query token per sequence (q, out [batch, q_heads, D]) against its lens[b] cached tokens.
 * table: device int32 [batch, table_width], the pages of each sequence in order; lens: device int32
 * [batch], clamped to [0, table_width * page_size].  Tokens on a page outside [0, pages) are not
 * seen.  lse fp32 [batch, q_heads] or NULL.  The long axis is split over workgroups; the partial
 * results (fp32) go through the workspace and are joined in a fixed order: a call's bits do not depend
 * on timing.  Its contents need no initialisation.
 */
int ssm_attn_decode_step(int64_t batch, int32_t q_heads, int32_t io_dtype, float scale, const ssm_kv_cache* cache,
                         const ssm_view* q, const int32_t* table, int64_t table_width, const int32_t* lens,
                         const ssm_view* out, float* lse, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* SSM_ATTN_H */
