// Launcher behind the orthogonalised update.
#pragma once

#include "moeq_internal.h"

namespace moeq {

constexpr int kOrthoMaxSteps = 64;

// The working matrices of one call, fp16 but for the partial sums: X and Y [E]
// [xr][xc] in turn (as the input lies, columns padded to a multiple of 8), A and
// P [E][n][nc] with n the shorter side.
struct OrthoPlan {
  int32_t E, N, K, n, m, xc, nc;
  bool tall;             // N > K: A = X^T X, X <- X P; otherwise A = X X^T, X <- P X
  int32_t chunks;        // partial sums of squares per matrix
  int64_t partial, x, y, a, p, bytes;   // offsets into the workspace, and its size
};
OrthoPlan ortho_plan(int32_t E, int32_t N, int32_t K);

// coefficients: [steps][3] on the host.
hipError_t launch_orthogonalize(const void* g, bool fp32, const OrthoPlan& plan, const float* coefficients, int32_t steps,
                                uint16_t* out, void* workspace, hipStream_t s);

}  // namespace moeq
