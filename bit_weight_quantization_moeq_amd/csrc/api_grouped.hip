// C entry points of the MXFP4 format, the grouped products and the gradient
// clipping: host-side validation and dispatch.  As in api.hip, every check
// runs before the first HIP call, so a rejected call has no side effect.
#include <algorithm>
#include <initializer_list>
#include <vector>

#include "grouped.h"

using namespace moeq;

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

moeq_status device_status(hipError_t e) { return e == hipSuccess ? MOEQ_OK : MOEQ_EDEVICE; }

constexpr int32_t kMaxDim = 1 << 20;     // N and K of a grouped product
constexpr int64_t kMaxExpertBytes = int64_t(1) << 31;
constexpr int32_t kMaxRows = 1 << 28;    // M of a grouped product
constexpr int64_t kMaxBlocks = int64_t(1) << 40;   // of an MXFP4 tensor: sizes in bytes fit 64 bits

// may_be_empty: rows == 0 is allowed, and the data pointers may then be null.
moeq_status check_mxfp4(const moeq_qweight* q, bool may_be_empty = false) {
  if (!q) return MOEQ_EINVAL;
  if (q->format != MOEQ_FMT_MXFP4) return MOEQ_EFORMAT;
  if (q->num_experts <= 0 || q->rows < (may_be_empty ? 0 : 1) || q->cols <= 0) return MOEQ_EINVAL;
  if ((q->rows > 0 && (!q->qdata || !q->scale_codes)) || q->scales) return MOEQ_EINVAL;
  if (q->blocksize != MOEQ_MXFP4_BLOCKSIZE || q->cols % MOEQ_MXFP4_BLOCKSIZE != 0) return MOEQ_EBLOCK;
  if ((int64_t)q->rows * (q->cols / MOEQ_MXFP4_BLOCKSIZE) > kMaxBlocks / q->num_experts) return MOEQ_ESHAPE;
  if (!aligned16(q->qdata) || !aligned16(q->scale_codes)) return MOEQ_EALIGN;
  return MOEQ_OK;
}

int64_t blocks(const moeq_qweight* q) { return (int64_t)q->num_experts * q->rows * (q->cols / MOEQ_MXFP4_BLOCKSIZE); }

moeq_status check_grouped(int32_t M, int32_t E, int32_t N, int32_t K) {
  if (M < 0 || E < 1 || N < 1 || K < 1) return MOEQ_EINVAL;
  if (E > MOEQ_MAX_EXPERTS || N > kMaxDim || K > kMaxDim || M > kMaxRows) return MOEQ_ESHAPE;
  if (N % 8 != 0 || K % 8 != 0) return MOEQ_ESHAPE;
  if ((int64_t)N * K * 2 >= kMaxExpertBytes) return MOEQ_ESHAPE;
  // The tiles' grids (a quarter more workgroups than tiles) hold less than
  // 2^32 threads: 512 for a tile of 256 x 256, 256 for one of 64 x 128.
  const int64_t threads = int64_t(1) << 32;
  if (((int64_t)M / 256 + E) * (N / 256 + 1) * 640 + 8192 >= threads) return MOEQ_ESHAPE;
  if (K <= 64 && ((int64_t)M / 64 + E) * (N / 128 + 1) * 320 + 8192 >= threads) return MOEQ_ESHAPE;
  return MOEQ_OK;
}

// Whether what a call writes shares memory with one of the others.  The
// kernels' workgroups read their operands while others store their results, so
// such a call would read its own output.
struct Span {
  const void* p;
  int64_t bytes;
};
bool overlaps(const Span& out, std::initializer_list<Span> others) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(out.p), hi = lo + (uintptr_t)out.bytes;
  for (const Span& s : others) {
    const uintptr_t l = reinterpret_cast<uintptr_t>(s.p);
    if (out.bytes > 0 && s.bytes > 0 && lo < l + (uintptr_t)s.bytes && l < hi) return true;
  }
  return false;
}
Span bf16(const uint16_t* p, int64_t rows, int64_t cols) { return {p, rows * cols * 2}; }
Span ints(const int32_t* offsets, int32_t E) { return {offsets, (E + int64_t(1)) * 4}; }
Span codes(const moeq_qweight* q) { return {q->qdata, blocks(q) * (MOEQ_MXFP4_BLOCKSIZE / 2)}; }
Span scale_codes(const moeq_qweight* q) { return {q->scale_codes, blocks(q)}; }

// Whether a tensor that is written overlaps any other one (in place, a
// tensor is one range), or the norm and the workspace.
bool overlapping(const moeq_grad* g, int32_t count, const Span& norm, const Span& workspace) {
  struct Range {
    uintptr_t lo, hi;
    bool written;
  };
  std::vector<Range> r;
  r.reserve(2 * (size_t)count + 2);
  for (const Span& s : {norm, workspace}) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(s.p);
    r.push_back({lo, lo + (uintptr_t)s.bytes, true});
  }
  for (int32_t i = 0; i < count; ++i) {
    if (g[i].numel == 0) continue;
    const uintptr_t size = (uintptr_t)g[i].numel * (g[i].dtype == MOEQ_DTYPE_FP32 ? 4 : 2);
    const uintptr_t src = reinterpret_cast<uintptr_t>(g[i].src), dst = reinterpret_cast<uintptr_t>(g[i].dst);
    r.push_back({dst, dst + size, true});
    if (src != dst) r.push_back({src, src + size, false});
  }
  std::sort(r.begin(), r.end(), [](const Range& a, const Range& b) { return a.lo < b.lo; });
  uintptr_t any = 0, written = 0;  // where the ranges so far end
  for (const Range& x : r) {
    if (x.lo < (x.written ? any : written)) return true;
    any = std::max(any, x.hi);
    if (x.written) written = std::max(written, x.hi);
  }
  return false;
}

}  // namespace

extern "C" {

moeq_status moeq_quantize_mxfp4(const uint16_t* w, const moeq_qweight* dst, void* stream) {
  const moeq_status st = check_mxfp4(dst);
  if (st != MOEQ_OK) return st;
  if (!w) return MOEQ_EINVAL;
  if (!aligned16(w)) return MOEQ_EALIGN;
  const Span in = {w, blocks(dst) * 2 * MOEQ_MXFP4_BLOCKSIZE};
  if (overlaps(codes(dst), {in, scale_codes(dst)}) || overlaps(scale_codes(dst), {in})) return MOEQ_EINVAL;
  return device_status(launch_quantize_mxfp4(w, static_cast<uint8_t*>(dst->qdata), dst->scale_codes, blocks(dst),
                                             static_cast<hipStream_t>(stream)));
}

moeq_status moeq_dequantize_mxfp4(const moeq_qweight* src, uint16_t* out, void* stream) {
  const moeq_status st = check_mxfp4(src);
  if (st != MOEQ_OK) return st;
  if (!out) return MOEQ_EINVAL;
  if (!aligned16(out)) return MOEQ_EALIGN;
  if (overlaps({out, blocks(src) * 2 * MOEQ_MXFP4_BLOCKSIZE}, {codes(src), scale_codes(src)})) return MOEQ_EINVAL;
  return device_status(launch_dequantize_mxfp4(static_cast<const uint8_t*>(src->qdata), src->scale_codes, out,
                                               blocks(src), static_cast<hipStream_t>(stream)));
}

moeq_status moeq_grouped_mm(const uint16_t* x, const uint16_t* w, const int32_t* offsets, int32_t M, int32_t E,
                            int32_t N, int32_t K, uint16_t* out, void* stream) {
  const moeq_status st = check_grouped(M, E, N, K);
  if (st != MOEQ_OK) return st;
  if (M == 0) return MOEQ_OK;
  if (!x || !w || !offsets || !out) return MOEQ_EINVAL;
  if (!aligned16(x) || !aligned16(w) || !aligned16(out)) return MOEQ_EALIGN;
  if (overlaps(bf16(out, M, N), {bf16(x, M, K), bf16(w, (int64_t)E * N, K), ints(offsets, E)})) return MOEQ_EINVAL;
  const GroupedArgs g = {x, w, nullptr, nullptr, offsets, out, M, E, N, K};
  return device_status(launch_grouped_mm(g, static_cast<hipStream_t>(stream)));
}

moeq_status moeq_grouped_mm_grad_input(const uint16_t* dy, const uint16_t* w, const int32_t* offsets, int32_t M,
                                       int32_t E, int32_t N, int32_t K, uint16_t* dx, void* stream) {
  moeq_status st = check_grouped(M, E, N, K);
  if (st == MOEQ_OK) st = check_grouped(M, E, K, N);
  if (st != MOEQ_OK) return st;
  if (M == 0) return MOEQ_OK;
  if (!dy || !w || !offsets || !dx) return MOEQ_EINVAL;
  if (!aligned16(dy) || !aligned16(w) || !aligned16(dx)) return MOEQ_EALIGN;
  if (overlaps(bf16(dx, M, K), {bf16(dy, M, N), bf16(w, (int64_t)E * N, K), ints(offsets, E)})) return MOEQ_EINVAL;
  const GroupedArgs g = {dy, w, nullptr, nullptr, offsets, dx, M, E, K, N};
  return device_status(launch_grouped_mm_grad_input(g, static_cast<hipStream_t>(stream)));
}

size_t moeq_grouped_mm_grad_weight_workspace_bytes(int32_t M, int32_t E, int32_t N, int32_t K) {
  if (check_grouped(M, E, N, K) != MOEQ_OK) return 0;
  return sizeof(float) * (size_t)grad_weight_slots(M, grad_weight_segment(M, N, K)) * N * K;
}

moeq_status moeq_grouped_mm_grad_weight(const uint16_t* dy, const uint16_t* x, const int32_t* offsets, int32_t M,
                                        int32_t E, int32_t N, int32_t K, int32_t dtype, void* dw, void* workspace,
                                        size_t workspace_bytes, void* stream) {
  const moeq_status st = check_grouped(M, E, N, K);
  if (st != MOEQ_OK) return st;
  if (dtype != MOEQ_DTYPE_BF16 && dtype != MOEQ_DTYPE_FP32) return MOEQ_EFORMAT;
  if (!offsets || !dw || (M > 0 && (!dy || !x))) return MOEQ_EINVAL;
  if (!aligned16(dw) || (M > 0 && (!aligned16(dy) || !aligned16(x)))) return MOEQ_EALIGN;
  const size_t need = moeq_grouped_mm_grad_weight_workspace_bytes(M, E, N, K);
  if (need > 0 && (!workspace || workspace_bytes < need)) return MOEQ_EWORKSPACE;
  if (need > 0 && !aligned16(workspace)) return MOEQ_EALIGN;
  const Span out = {dw, (int64_t)E * N * K * (dtype == MOEQ_DTYPE_FP32 ? 4 : 2)}, sums = {workspace, (int64_t)need};
  if (overlaps(out, {bf16(dy, M, N), bf16(x, M, K), ints(offsets, E), sums}) ||
      overlaps(sums, {bf16(dy, M, N), bf16(x, M, K), ints(offsets, E)}))
    return MOEQ_EINVAL;
  GroupedArgs g = {x, dy, nullptr, nullptr, offsets, dw, M, E, N, K};
  g.segment = grad_weight_segment(M, N, K);
  g.slots = (int32_t)grad_weight_slots(M, g.segment);
  g.partial = static_cast<float*>(workspace);
  return device_status(launch_grouped_mm_grad_weight(g, dtype == MOEQ_DTYPE_FP32, static_cast<hipStream_t>(stream)));
}

moeq_status moeq_grouped_mm_mxfp4(const moeq_qweight* x, const moeq_qweight* w, const int32_t* offsets, uint16_t* out,
                                  void* stream) {
  moeq_status st = check_mxfp4(x, true);
  if (st == MOEQ_OK) st = check_mxfp4(w);
  if (st != MOEQ_OK) return st;
  if (x->num_experts != 1 || x->cols != w->cols) return MOEQ_ESHAPE;
  st = check_grouped(x->rows, w->num_experts, w->rows, w->cols);
  if (st != MOEQ_OK) return st;
  if (x->rows == 0) return MOEQ_OK;
  if (!offsets || !out) return MOEQ_EINVAL;
  if (!aligned16(out)) return MOEQ_EALIGN;
  if (overlaps(bf16(out, x->rows, w->rows),
               {codes(x), scale_codes(x), codes(w), scale_codes(w), ints(offsets, w->num_experts)}))
    return MOEQ_EINVAL;
  const GroupedArgs g = {x->qdata, w->qdata, x->scale_codes, w->scale_codes, offsets, out,
                         x->rows, w->num_experts, w->rows, w->cols};
  return device_status(launch_grouped_mm_mxfp4(g, static_cast<hipStream_t>(stream)));
}

size_t moeq_clip_grad_norm_workspace_bytes(int32_t count) {
  return count < 0 ? 0 : sizeof(double) * (size_t)(kClipHead + clip_partials(count));
}

moeq_status moeq_clip_grad_norm(const moeq_grad* grads, int32_t count, double max_norm, float* norm, void* workspace,
                                size_t workspace_bytes, void* stream) {
  if (count < 0 || (count > 0 && !grads) || !norm) return MOEQ_EINVAL;
  if (!(max_norm >= 0.0)) return MOEQ_EINVAL;
  for (int32_t i = 0; i < count; ++i) {
    const moeq_grad& g = grads[i];
    if (g.numel < 0 || g.numel > (int64_t(1) << 37) || (g.numel > 0 && (!g.src || !g.dst))) return MOEQ_EINVAL;
    if (g.dtype != MOEQ_DTYPE_BF16 && g.dtype != MOEQ_DTYPE_FP32) return MOEQ_EFORMAT;
    const uintptr_t size = g.dtype == MOEQ_DTYPE_FP32 ? 4 : 2;
    if (g.numel > 0 && (reinterpret_cast<uintptr_t>(g.src) % size || reinterpret_cast<uintptr_t>(g.dst) % size))
      return MOEQ_EALIGN;
  }
  if (reinterpret_cast<uintptr_t>(norm) % 4) return MOEQ_EALIGN;
  if (!workspace || workspace_bytes < moeq_clip_grad_norm_workspace_bytes(count)) return MOEQ_EWORKSPACE;
  if (!aligned16(workspace)) return MOEQ_EALIGN;
  try {
    if (overlapping(grads, count, {norm, sizeof(float)},
                    {workspace, (int64_t)moeq_clip_grad_norm_workspace_bytes(count)}))
      return MOEQ_EINVAL;
  } catch (...) {   // (no room on the host for the ranges)
    return MOEQ_EWORKSPACE;
  }
  return device_status(launch_clip(grads, count, max_norm, norm, static_cast<double*>(workspace),
                                   static_cast<hipStream_t>(stream)));
}

}  // extern "C"
