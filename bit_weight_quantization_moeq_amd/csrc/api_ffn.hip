// C entry points of the gated feed-forward block over rows sorted by expert.
#include <algorithm>

#include "api_checks.h"
#include "ffn.h"

using namespace moeq;

namespace {

// Of the block's products, in both directions.
moeq_status check_ffn(int32_t M, int32_t E, int32_t H, int32_t I) {
  if (M < 0 || E < 1 || H < 1 || I < 1) return MOEQ_EINVAL;
  if (I > kMaxDim / 2) return MOEQ_ESHAPE;
  moeq_status st = check_grouped(M, E, 2 * I, H);
  if (st == MOEQ_OK) st = check_grouped(M, E, H, 2 * I);
  if (st == MOEQ_OK) st = check_grouped(M, E, H, I);
  if (st == MOEQ_OK) st = check_grouped(M, E, I, H);
  return st;
}

size_t round16(size_t n) { return (n + 15) / 16 * 16; }
size_t rows_bytes(int32_t M, int32_t cols) { return round16((size_t)M * cols * 2); }
size_t sums_bytes(int32_t M, int32_t E, int32_t H, int32_t I) {
  return std::max(moeq_grouped_mm_grad_weight_workspace_bytes(M, E, 2 * I, H),
                  moeq_grouped_mm_grad_weight_workspace_bytes(M, E, H, I));
}

moeq_status check_workspace(const void* workspace, size_t bytes, size_t need) {
  if (need > 0 && (!workspace || bytes < need)) return MOEQ_EWORKSPACE;
  return need > 0 && !aligned16(workspace) ? MOEQ_EALIGN : MOEQ_OK;
}

}  // namespace

extern "C" {

size_t moeq_grouped_ffn_workspace_bytes(int32_t M, int32_t E, int32_t H, int32_t I) {
  return check_ffn(M, E, H, I) == MOEQ_OK ? rows_bytes(M, I) : 0;
}

moeq_status moeq_grouped_ffn(const uint16_t* x, const uint16_t* gate_up, const uint16_t* down, const int32_t* offsets,
                             int32_t M, int32_t E, int32_t H, int32_t I, float* gu_saved, uint16_t* out,
                             void* workspace, size_t workspace_bytes, void* stream) {
  moeq_status st = check_ffn(M, E, H, I);
  if (st != MOEQ_OK) return st;
  if (M == 0) return MOEQ_OK;
  if (!x || !gate_up || !down || !offsets || !out) return MOEQ_EINVAL;
  if (!aligned16(x) || !aligned16(gate_up) || !aligned16(down) || !aligned16(out) || !aligned16(gu_saved))
    return MOEQ_EALIGN;
  const size_t need = moeq_grouped_ffn_workspace_bytes(M, E, H, I);
  st = check_workspace(workspace, workspace_bytes, need);
  if (st != MOEQ_OK) return st;
  const Span in = bf16(x, M, H), w1 = bf16(gate_up, (int64_t)E * 2 * I, H), w2 = bf16(down, (int64_t)E * H, I),
             off = ints(offsets, E), gu = {gu_saved, gu_saved ? (int64_t)M * 2 * I * 4 : 0}, y = bf16(out, M, H),
             ws = {workspace, (int64_t)need};
  if (overlaps(ws, {in, w1, w2, off}) || overlaps(gu, {in, w1, w2, off, ws}) || overlaps(y, {in, w1, w2, off, ws, gu}))
    return MOEQ_EINVAL;
  uint16_t* h = static_cast<uint16_t*>(workspace);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e = launch_glu({x, gate_up, nullptr, nullptr, offsets, h, M, E, I, H}, gu_saved, s);
  if (e == hipSuccess) e = launch_grouped_mm({h, down, nullptr, nullptr, offsets, out, M, E, H, I}, s);
  return device_status(e);
}

size_t moeq_grouped_ffn_backward_workspace_bytes(int32_t M, int32_t E, int32_t H, int32_t I) {
  return check_ffn(M, E, H, I) == MOEQ_OK ? rows_bytes(M, 2 * I) + rows_bytes(M, I) + sums_bytes(M, E, H, I) : 0;
}

moeq_status moeq_grouped_ffn_backward(const uint16_t* grad_out, const uint16_t* x, const uint16_t* gate_up,
                                      const uint16_t* down, const int32_t* offsets, const float* gu_saved, int32_t M,
                                      int32_t E, int32_t H, int32_t I, int32_t dtype, uint16_t* grad_x,
                                      void* grad_gate_up, void* grad_down, void* workspace, size_t workspace_bytes,
                                      void* stream) {
  moeq_status st = check_ffn(M, E, H, I);
  if (st != MOEQ_OK) return st;
  if (dtype != MOEQ_DTYPE_BF16 && dtype != MOEQ_DTYPE_FP32) return MOEQ_EFORMAT;
  if (!offsets || !grad_gate_up || !grad_down) return MOEQ_EINVAL;
  if (M > 0 && (!grad_out || !x || !gate_up || !down || !gu_saved || !grad_x)) return MOEQ_EINVAL;
  if (!aligned16(grad_gate_up) || !aligned16(grad_down)) return MOEQ_EALIGN;
  if (M > 0)
    for (const uint16_t* p : {grad_out, x, gate_up, down, static_cast<const uint16_t*>(grad_x)})
      if (!aligned16(p) || !aligned16(gu_saved)) return MOEQ_EALIGN;
  const size_t need = moeq_grouped_ffn_backward_workspace_bytes(M, E, H, I);
  st = check_workspace(workspace, workspace_bytes, need);
  if (st != MOEQ_OK) return st;
  const int64_t size = dtype == MOEQ_DTYPE_FP32 ? 4 : 2, w1n = (int64_t)E * 2 * I * H, w2n = (int64_t)E * H * I;
  const Span dy = bf16(grad_out, M, H), in = bf16(x, M, H), w1 = {gate_up, M ? w1n * 2 : 0}, w2 = {down, M ? w2n * 2 : 0},
             off = ints(offsets, E), gu = {gu_saved, (int64_t)M * 2 * I * 4}, dx = bf16(grad_x, M, H),
             dw1 = {grad_gate_up, w1n * size}, dw2 = {grad_down, w2n * size}, ws = {workspace, (int64_t)need};
  if (overlaps(ws, {dy, in, w1, w2, off, gu}) || overlaps(dx, {dy, in, w1, w2, off, gu, ws}) ||
      overlaps(dw1, {dy, in, w1, w2, off, gu, ws, dx}) || overlaps(dw2, {dy, in, w1, w2, off, gu, ws, dx, dw1}))
    return MOEQ_EINVAL;

  char* p = static_cast<char*>(workspace);
  uint16_t* dgu = reinterpret_cast<uint16_t*>(p);
  uint16_t* h = reinterpret_cast<uint16_t*>(p + rows_bytes(M, 2 * I));
  float* sums = reinterpret_cast<float*>(p + rows_bytes(M, 2 * I) + rows_bytes(M, I));
  const hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e = hipSuccess;
  if (M > 0) {
    e = launch_glu_backward({grad_out, down, nullptr, nullptr, offsets, h, M, E, I, H}, gu_saved, dgu, s);
    if (e == hipSuccess)
      e = launch_grouped_mm_grad_input({dgu, gate_up, nullptr, nullptr, offsets, grad_x, M, E, H, 2 * I}, s);
  }
  // grad[e] = sum of rows[p] in[p]^T, [N][K]
  auto weight = [&](const uint16_t* rows, const uint16_t* xs, int32_t N, int32_t K, void* grad) {
    if (e != hipSuccess) return;
    GroupedArgs g = {xs, rows, nullptr, nullptr, offsets, grad, M, E, N, K};
    g.segment = grad_weight_segment(M, N, K);
    g.slots = (int32_t)grad_weight_slots(M, g.segment);
    g.partial = sums;
    e = launch_grouped_mm_grad_weight(g, dtype == MOEQ_DTYPE_FP32, s);
  };
  weight(dgu, x, 2 * I, H, grad_gate_up);
  weight(grad_out, h, H, I, grad_down);
  return device_status(e);
}

}  // extern "C"
