// Launcher behind the orthogonalised update.
#pragma once

#include <algorithm>

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
constexpr int kOrthoChunk = 1 << 15;   // values per partial sum, at least
constexpr int kOrthoMaxChunks = 64;

inline OrthoPlan ortho_plan(int32_t E, int32_t N, int32_t K) {
  auto pad8 = [](int32_t n) { return (n + 7) / 8 * 8; };
  auto round256 = [](int64_t n) { return (n + 255) / 256 * 256; };
  OrthoPlan p;
  p.E = E;
  p.N = N;
  p.K = K;
  p.tall = N > K;
  p.n = std::min(N, K);
  p.m = std::max(N, K);
  p.xc = pad8(K);
  p.nc = pad8(p.n);
  p.chunks = (int32_t)std::min<int64_t>(kOrthoMaxChunks, ((int64_t)N * K + kOrthoChunk - 1) / kOrthoChunk);
  const int64_t x = round256((int64_t)E * N * p.xc * 2), a = round256((int64_t)E * p.n * p.nc * 2);
  p.partial = 0;
  p.x = round256((int64_t)E * p.chunks * 8);
  p.y = p.x + x;
  p.a = p.y + x;
  p.p = p.a + a;
  p.bytes = p.p + a;
  return p;
}

// coefficients: [steps][3] on the host.
hipError_t launch_orthogonalize(const void* g, bool fp32, const OrthoPlan& plan, const float* coefficients, int32_t steps,
                                uint16_t* out, void* workspace, hipStream_t s);

}  // namespace moeq
