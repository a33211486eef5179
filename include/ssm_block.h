/*
 * ssm_block.h -- C ABI of the operators between a stack's residual stream and its mixers' projections,
 * on AMD Instinct MI355X (gfx950).  Part of libssm.so.
 *
 * A block of a stack (a selective-SSM mixer, ssm_layer.h, or an attention block, ssm_attn.h) starts with
 * the sum of the residual stream and a norm, and its input and output projections are most of the bytes
 * that a decoded token reads.  One rank runs there:
 *   ssm_rms_norm           the residual's addition and the root-mean-square norm, in the io dtype or in
 *                          8 bits with a scale per token
 *   ssm_q4_quantize        a projection's weight in 4 bits with a power of two for each 32 values
 *   ssm_q4_dequantize      such a weight back in the io dtype
 *   ssm_q4_linear          products of tokens with such a weight
 *
 * Formulas.
 *   norm       h = x + residual, summed in fp32 and rounded once to the residual's dtype (h = x where
 *              there is no residual); r = 1 / sqrt(mean(h^2) + eps); y = (h * weight) * r, fp32, rounded
 *              once to the output's dtype.  (The sum of h^2 is fp32: magnitudes stay below 2^56.)
 *   8-bit rows one fp32 scale per row: amax = max |y|, s = amax * (1 / 448); code = e4m3, nearest even, of
 *              (h * weight) * (448 / max |h * weight|), which is y * (448 / amax) with fewer roundings (in fp64,
 *              rounded to fp32 before; rows of more than 8192 values in fp32); value = code * s.  Rows with amax < 2^-100
 *              get s = 0 and codes 0.  A row with a NaN or an infinity gets s = NaN: all of it reads back as NaN.
 *   4-bit      w[m, k] = c * 2^(e - 127): c one of 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives (e2m1:
 *              sign, two bits of exponent, one of mantissa, in code order), e a byte for each 32 values of
 *              a row (k / 32).  Quantising: amax = max |w| of the group, rounded to three significant bits
 *              (half away from zero, bit pattern + 2^21), falls in 2^n .. 2^(n+1); e = n - 2 + 127, at most
 *              252; code = w * 2^(127 - e) to nearest, ties to the even code, at most 6 in magnitude.
 *              Groups with amax < 2^-100 get codes 0 and e = 127; what rounds to zero keeps its sign.
 *              Groups with a NaN or an infinity get codes 0 and e = 255, for which every value is NaN.
 *              Every value is exact in bf16 for e in [2, 252]; other bytes are outside the contract.
 *   linear     out[t, m] = x_scale[t] * sum_k x[t, k] w[m, k] (no x_scale for bf16 and fp32 tokens), sums
 *              in fp32.  Products are exact: bf16 tokens (and e4m3 tokens widened to it) multiply the
 *              exact 4-bit values on the matrix cores, fp32 tokens as three bf16 parts (whose sum is the
 *              token, for magnitudes from 2^-99 to 2^127).
 *              No sum is split differently from one call to the next: a call's bits depend on its sizes
 *              and values alone.
 *
 * 4-bit layout, for W [M, K] row-major in the formulas (M = out_features, K = in_features):
 *   codes  [ceil(M / 16), ceil(K / 128), 64, 16] bytes: tile (m / 16, k / 128), in it lane
 *          (k % 128) / 32 * 16 + m % 16, in it byte (k % 32) / 2, low nibble for even k
 *   scales [ceil(M / 16), ceil(K / 512), 64, 4] bytes: tile (m / 16, k / 512), the same lane, byte
 *          (k / 128) % 4
 * Places past M hold anything; places past K hold codes 0 and scales 127 (ssm_q4_quantize writes both so).
 * A tile is what one wave loads at once, and a lane's 16 bytes one group, with one scale.
 *
 * Rows.  A [T, D] tensor is a base pointer and a row stride in elements (ssm_rows), the D values of a row
 * contiguous.  Row strides lie in [0, 2^22] (written rows may not overlap: at least D where T > 1).
 * Alignment: bases and row strides multiples of 16 bytes (8 bytes for e4m3 rows that ssm_rms_norm writes;
 * out of ssm_q4_linear: its dtype's own size).
 *
 * Conventions (ownership, ordering, errors before any HIP call, no allocation, no mutable global state,
 * no host synchronisation, the current device) as in ssm.h.  Outputs may not overlap inputs or each
 * other, except where said.  0 tokens: a call that does nothing.  Non-finite inputs stay in their row
 * (ssm_rms_norm, a token's row of ssm_q4_linear) and are not lost there: the norm in the io dtype and the
 * products give what the formulas give (an infinity among fp32 tokens may give NaN), the norm in 8 bits
 * and a weight in 4 bits what is said above.
 */
#ifndef SSM_BLOCK_H
#define SSM_BLOCK_H

#include <stddef.h>
#include <stdint.h>

#include "ssm.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SSM_E4M3 2                /* beside ssm_dtype's SSM_F32 and SSM_BF16: rows in 8 bits */
#define SSM_NORM_MAX_WIDTH 32768
#define SSM_Q4_GROUP 32
#define SSM_Q4_MAX_FEATURES (1 << 20) /* largest in_features and out_features; their product at most 2^38 */

/* A [T, D] tensor on the device; the stride in elements. */
typedef struct {
  void* data;
  int64_t stride;
} ssm_rows;

/* A 4-bit weight on the device (layout above). */
typedef struct {
  void* codes;  /* ssm_q4_codes_bytes() */
  void* scales; /* ssm_q4_scales_bytes() */
  int64_t out_features; /* M in [1, SSM_Q4_MAX_FEATURES] */
  int64_t in_features;  /* K, a multiple of 16 in [16, SSM_Q4_MAX_FEATURES] */
} ssm_q4_weight;

/*
 * x [tokens, width] (io_dtype SSM_F32 or SSM_BF16), weight fp32 [width], width a multiple of 8 up to
 * SSM_NORM_MAX_WIDTH; eps finite and at least 2^-126.
 * residual, residual_out [tokens, width] in residual_dtype (io_dtype, or SSM_F32): both or neither (NULL).
 * residual_out may be residual itself (in place: same data and stride).
 * out [tokens, width] in out_dtype: io_dtype, or SSM_E4M3 with scale fp32 [tokens] (NULL otherwise).
 * out may be x itself where out_dtype is io_dtype.
 */
int ssm_rms_norm(int64_t tokens, int64_t width, int32_t io_dtype, int32_t residual_dtype, int32_t out_dtype, float eps,
                 const ssm_rows* x, const float* weight, const ssm_rows* residual, const ssm_rows* residual_out,
                 const ssm_rows* out, float* scale, void* stream);

/* Bytes of a weight's codes and scales (0 for invalid sizes). */
size_t ssm_q4_codes_bytes(int64_t out_features, int64_t in_features);
size_t ssm_q4_scales_bytes(int64_t out_features, int64_t in_features);

/* w [M, K] in io_dtype into q (every byte of codes and scales is written). */
int ssm_q4_quantize(int32_t io_dtype, const ssm_rows* w, const ssm_q4_weight* q, void* stream);

/* q back into w [M, K] in io_dtype. */
int ssm_q4_dequantize(int32_t io_dtype, const ssm_q4_weight* q, const ssm_rows* w, void* stream);

/*
 * out [tokens, M] (out_dtype SSM_F32 or SSM_BF16) from x [tokens, K] (x_dtype SSM_F32, SSM_BF16, or SSM_E4M3 with
 * x_scale fp32 [tokens]; NULL otherwise).  tokens below 2^24, tokens * M at most 2^35.
 */
int ssm_q4_linear(int64_t tokens, int32_t x_dtype, int32_t out_dtype, const ssm_rows* x, const float* x_scale,
                  const ssm_q4_weight* q, const ssm_rows* out, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* SSM_BLOCK_H */
