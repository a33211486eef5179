// ssm_block.h -- what the kernels of include/ssm_block.h share (ssm_norm.hip, ssm_q4.hip; ssm_q4_rows.hip, ssm_q4_few.hip and
// ssm_q4_tiles.hip by way of ssm_q4_linear.h): rows, the 4-bit layout and the host-side checks.
#pragma once
#include "../../include/ssm_block.h"
#include "ssm_attn.h"

namespace ssm {
namespace block {

using attn::aligned;
using attn::bf16x8;
using attn::f32x16;
using attn::f32x4;
using attn::overlaps;
using attn::pack_bf16;
using attn::ready;
using attn::Span;
using attn::span;
using attn::u32x2;
using attn::u32x4;

constexpr int64_t MAX_ROW_STRIDE = int64_t(1) << 22;
constexpr int64_t MAX_TOKENS = int64_t(1) << 24;
// Most values of a 4-bit weight, and of a product's output: a launch has fewer than 2^32 work-items (at most one for 16 outputs,
// and those of tiles that are not whole).
constexpr int64_t MAX_WEIGHTS = int64_t(1) << 38, MAX_OUTPUTS = int64_t(1) << 35;

// Rows with a byte stride.
struct Rows {
  char* p;
  int64_t stride;
};
inline Rows rows_of(const ssm_rows* r, int64_t es) {
  return r ? Rows{static_cast<char*>(r->data), r->stride * es} : Rows{nullptr, 0};
}

inline Span rows_span(const ssm_rows* r, int64_t tokens, int64_t width, int64_t es) {
  return span(r->data, ((tokens - 1) * r->stride + width) * es);
}
// Whether two [tokens, .] tensors may touch a common byte; parts of one packed row (equal strides) may lie side by side.
inline bool rows_overlap(const ssm_rows* a, int64_t wa, int64_t ea, const ssm_rows* b, int64_t wb, int64_t eb, int64_t tokens) {
  if (!overlaps(rows_span(a, tokens, wa, ea), rows_span(b, tokens, wb, eb))) return false;
  return !(a->stride * ea == b->stride * eb && a->stride > 0 && attn::apart(a->data, wa * ea, b->data, wb * eb, a->stride * ea));
}
inline bool same_rows(const ssm_rows* a, const ssm_rows* b) { return a->data == b->data && a->stride == b->stride; }

inline int64_t size_of(int32_t dtype) { return dtype == SSM_F32 ? 4 : dtype == SSM_BF16 ? 2 : 1; }

// align: of the base and of the row stride, in bytes.
inline int check_rows(const ssm_rows* r, int64_t es, int64_t align) {
  if (!r || !r->data) return SSM_ERR_NULL;
  if (r->stride < 0 || r->stride > MAX_ROW_STRIDE) return SSM_ERR_SHAPE;
  if (!aligned(r->data, align) || r->stride * es % align) return SSM_ERR_ALIGN;
  return SSM_OK;
}
// Whether the rows that are written are disjoint.
inline bool writable(const ssm_rows* r, int64_t tokens, int64_t width) { return tokens <= 1 || r->stride >= width; }

inline bool q4_sizes(int64_t M, int64_t K) {
  return M >= 1 && M <= SSM_Q4_MAX_FEATURES && K >= 16 && K <= SSM_Q4_MAX_FEATURES && K % 16 == 0 &&
         M * K <= MAX_WEIGHTS;
}
inline int64_t q4_codes_bytes(int64_t M, int64_t K) { return ((M + 15) / 16) * ((K + 127) / 128) * 1024; }
inline int64_t q4_scales_bytes(int64_t M, int64_t K) { return ((M + 15) / 16) * ((K + 511) / 512) * 256; }

inline int check_q4(const ssm_q4_weight* q) {
  if (!q || !q->codes || !q->scales) return SSM_ERR_NULL;
  if (!q4_sizes(q->out_features, q->in_features)) return SSM_ERR_SHAPE;
  if (!aligned(q->codes, 16) || !aligned(q->scales, 16)) return SSM_ERR_ALIGN;
  return SSM_OK;
}
inline Span codes_span(const ssm_q4_weight* q) { return span(q->codes, q4_codes_bytes(q->out_features, q->in_features)); }
inline Span scales_span(const ssm_q4_weight* q) { return span(q->scales, q4_scales_bytes(q->out_features, q->in_features)); }

}  // namespace block
}  // namespace ssm
