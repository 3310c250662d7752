// C entry points of the FP8 format with a scale for each block of 128 and of
// the grouped product over it.
#include "api_checks.h"
#include "fp8.h"

using namespace moeq;

namespace {

constexpr int64_t kMaxFp8Blocks = int64_t(1) << 40;   // of 128 values or fewer: sizes in bytes fit 64 bits

bool tiled(const moeq_qweight* q) { return q->format == MOEQ_FMT_FP8_TILE; }

// may_be_empty: rows == 0 is allowed, and the data pointers may then be null.
moeq_status check_fp8(const moeq_qweight* q, bool may_be_empty = false) {
  if (!q) return MOEQ_EINVAL;
  if (q->format != MOEQ_FMT_FP8_ROW && q->format != MOEQ_FMT_FP8_TILE) return MOEQ_EFORMAT;
  if (q->num_experts <= 0 || q->rows < (may_be_empty ? 0 : 1) || q->cols <= 0) return MOEQ_EINVAL;
  if ((q->rows > 0 && (!q->qdata || !q->scales)) || q->scale_codes) return MOEQ_EINVAL;
  if (q->blocksize != kFp8Block || q->cols % 16 != 0) return MOEQ_EBLOCK;
  if ((int64_t)q->rows * fp8_blocks(q->cols) > kMaxFp8Blocks / q->num_experts) return MOEQ_ESHAPE;
  if (!aligned16(q->qdata) || reinterpret_cast<uintptr_t>(q->scales) % sizeof(float)) return MOEQ_EALIGN;
  return MOEQ_OK;
}

int64_t values(const moeq_qweight* q) { return (int64_t)q->num_experts * q->rows * q->cols; }
Span codes(const moeq_qweight* q) { return {q->qdata, values(q)}; }
Span scales(const moeq_qweight* q) {
  return {q->scales, (int64_t)q->num_experts * (tiled(q) ? fp8_blocks(q->rows) : q->rows) * fp8_blocks(q->cols) * 4};
}

}  // namespace

extern "C" {

moeq_status moeq_quantize_fp8(const uint16_t* w, const moeq_qweight* dst, void* stream) {
  const moeq_status st = check_fp8(dst);
  if (st != MOEQ_OK) return st;
  if (!w) return MOEQ_EINVAL;
  if (!aligned16(w)) return MOEQ_EALIGN;
  const Span in = {w, values(dst) * 2};
  if (overlaps(codes(dst), {in, scales(dst)}) || overlaps(scales(dst), {in})) return MOEQ_EINVAL;
  return device_status(launch_quantize_fp8(w, static_cast<uint8_t*>(dst->qdata), dst->scales, dst->num_experts, dst->rows,
                                           dst->cols, tiled(dst), static_cast<hipStream_t>(stream)));
}

moeq_status moeq_dequantize_fp8(const moeq_qweight* src, uint16_t* out, void* stream) {
  const moeq_status st = check_fp8(src);
  if (st != MOEQ_OK) return st;
  if (!out) return MOEQ_EINVAL;
  if (!aligned16(out)) return MOEQ_EALIGN;
  if (overlaps({out, values(src) * 2}, {codes(src), scales(src)})) return MOEQ_EINVAL;
  return device_status(launch_dequantize_fp8(static_cast<const uint8_t*>(src->qdata), src->scales, out, src->num_experts,
                                             src->rows, src->cols, tiled(src), static_cast<hipStream_t>(stream)));
}

moeq_status moeq_grouped_mm_fp8(const moeq_qweight* x, const moeq_qweight* w, const int32_t* offsets, uint16_t* out,
                                void* stream) {
  moeq_status st = check_fp8(x, true);
  if (st == MOEQ_OK) st = check_fp8(w);
  if (st != MOEQ_OK) return st;
  if (x->format != MOEQ_FMT_FP8_ROW || w->format != MOEQ_FMT_FP8_TILE) return MOEQ_EFORMAT;
  if (x->num_experts != 1 || x->cols != w->cols) return MOEQ_ESHAPE;
  st = check_grouped(x->rows, w->num_experts, w->rows, w->cols);
  if (st != MOEQ_OK) return st;
  if (x->rows == 0) return MOEQ_OK;
  if (!offsets || !out) return MOEQ_EINVAL;
  if (!aligned16(out)) return MOEQ_EALIGN;
  if (overlaps(bf16(out, x->rows, w->rows), {codes(x), scales(x), codes(w), scales(w), ints(offsets, w->num_experts)}))
    return MOEQ_EINVAL;
  const GroupedArgs g = {x->qdata, w->qdata, nullptr, nullptr, offsets, out, x->rows, w->num_experts, w->rows, w->cols};
  return device_status(launch_grouped_mm_fp8(g, x->scales, w->scales, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
