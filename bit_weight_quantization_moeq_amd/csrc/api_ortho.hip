// C entry point of the orthogonalised update.
#include <cmath>

#include "api_checks.h"
#include "ortho.h"

using namespace moeq;

namespace {

constexpr int32_t kMaxSide = 1 << 20, kMaxShortSide = 1 << 15;

moeq_status check_ortho(int32_t E, int32_t N, int32_t K) {
  if (E < 1 || N < 1 || K < 1) return MOEQ_EINVAL;
  if (E > 65535 || N > kMaxSide || K > kMaxSide || (N > kMaxShortSide && K > kMaxShortSide)) return MOEQ_ESHAPE;
  // The products' grids (a quarter more workgroups than tiles) hold less than
  // 2^32 threads: 256 for a tile of 64 x 64, of which there are less than 2^14
  // an edge where they serve, 512 for one of 256 x 256.
  const int64_t tiles = ((int64_t)N / 256 + 1) * (K / 256 + 1) * E;
  return tiles >= int64_t(1) << 18 ? MOEQ_ESHAPE : MOEQ_OK;
}

}  // namespace

extern "C" {

size_t moeq_orthogonalize_workspace_bytes(int32_t E, int32_t N, int32_t K) {
  return check_ortho(E, N, K) == MOEQ_OK ? (size_t)ortho_plan(E, N, K).bytes : 0;
}

moeq_status moeq_orthogonalize(const void* g, int32_t dtype, int32_t E, int32_t N, int32_t K, const float* coefficients,
                               int32_t steps, uint16_t* out, void* workspace, size_t workspace_bytes, void* stream) {
  const moeq_status st = check_ortho(E, N, K);
  if (st != MOEQ_OK) return st;
  if (dtype != MOEQ_DTYPE_BF16 && dtype != MOEQ_DTYPE_FP32) return MOEQ_EFORMAT;
  if (!g || !out || !coefficients || steps < 1 || steps > kOrthoMaxSteps) return MOEQ_EINVAL;
  for (int32_t i = 0; i < 3 * steps; ++i)
    if (!std::isfinite(coefficients[i])) return MOEQ_EINVAL;
  const int64_t size = dtype == MOEQ_DTYPE_FP32 ? 4 : 2, values = (int64_t)E * N * K;
  if (reinterpret_cast<uintptr_t>(g) % size != 0 || !aligned16(out)) return MOEQ_EALIGN;
  const OrthoPlan plan = ortho_plan(E, N, K);
  if (!workspace || workspace_bytes < (size_t)plan.bytes) return MOEQ_EWORKSPACE;
  if (!aligned16(workspace)) return MOEQ_EALIGN;
  const Span in = {g, values * size}, ws = {workspace, plan.bytes};
  if (overlaps({out, values * 2}, {in, ws}) || overlaps(ws, {in})) return MOEQ_EINVAL;
  return device_status(launch_orthogonalize(g, dtype == MOEQ_DTYPE_FP32, plan, coefficients, steps, out, workspace,
                                            static_cast<hipStream_t>(stream)));
}

}  // extern "C"
