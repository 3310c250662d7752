// Drives the host code of the feed-forward block, the FP8 format and the
// orthogonalised update (no GPU, no kernel launch: the launchers are counting
// stubs), built with AddressSanitizer and UndefinedBehaviorSanitizer on the host
// code.  Pointers handed in are never dereferenced; descriptors and coefficients
// are.  Exits non-zero on the first result that differs from the documented one.
#include <stdio.h>

#include <climits>
#include <cmath>
#include <cstdint>

// The workspaces' own host code is compiled in, but the entry points reach the
// stubs below.
#define launch_grouped_mm launch_grouped_mm_real
#define launch_grouped_mm_mxfp4 launch_grouped_mm_mxfp4_real
#define launch_grouped_mm_grad_input launch_grouped_mm_grad_input_real
#define launch_grouped_mm_grad_weight launch_grouped_mm_grad_weight_real
#include "grouped.hip"
#undef launch_grouped_mm
#undef launch_grouped_mm_mxfp4
#undef launch_grouped_mm_grad_input
#undef launch_grouped_mm_grad_weight
#include "ffn.h"
#include "fp8.h"
#include "ortho.h"

static int launches = 0, failures = 0;

namespace moeq {
static hipError_t hit() {
  ++launches;
  return hipSuccess;
}
hipError_t launch_quantize_mxfp4(const uint16_t*, uint8_t*, uint8_t*, int64_t, hipStream_t) { return hit(); }
hipError_t launch_dequantize_mxfp4(const uint8_t*, const uint8_t*, uint16_t*, int64_t, hipStream_t) { return hit(); }
hipError_t launch_grouped_mm(const GroupedArgs&, hipStream_t) { return hit(); }
hipError_t launch_grouped_mm_mxfp4(const GroupedArgs&, hipStream_t) { return hit(); }
hipError_t launch_grouped_mm_grad_input(const GroupedArgs&, hipStream_t) { return hit(); }
hipError_t launch_grouped_mm_grad_weight(const GroupedArgs& g, bool, hipStream_t) {
  // what the sums of long experts need is there
  if (grad_weight_slots(g.M, g.segment) != g.slots || (g.slots > 0 && !g.partial)) ++failures;
  return hit();
}
int64_t clip_partials(int32_t) { return 1; }
hipError_t launch_clip(const moeq_grad*, int32_t, double, float*, double*, hipStream_t) { return hit(); }
hipError_t launch_glu(const GroupedArgs&, float*, hipStream_t) { return hit(); }
hipError_t launch_glu_backward(const GroupedArgs&, const float*, uint16_t*, hipStream_t) { return hit(); }
hipError_t launch_quantize_fp8(const uint16_t*, uint8_t*, float*, int32_t, int32_t, int32_t, bool, hipStream_t) {
  return hit();
}
hipError_t launch_dequantize_fp8(const uint8_t*, const float*, uint16_t*, int32_t, int32_t, int32_t, bool, hipStream_t) {
  return hit();
}
hipError_t launch_grouped_mm_fp8(const GroupedArgs&, const float*, const float*, hipStream_t) { return hit(); }
hipError_t launch_orthogonalize(const void*, bool, const OrthoPlan&, const float* table, int32_t steps, uint16_t*, void*,
                                hipStream_t) {
  float sum = 0.f;
  for (int32_t i = 0; i < 3 * steps; ++i) sum += table[i];   // (read here, under the sanitizer)
  return sum == sum ? hit() : hipErrorUnknown;
}
}  // namespace moeq

#define EXPECT(call, want)                                                                          \
  do {                                                                                              \
    const long long got_ = (long long)(call), want_ = (long long)(want);                            \
    if (got_ != want_) {                                                                            \
      fprintf(stderr, "%s:%d: %s -> %lld, expected %lld\n", __FILE__, __LINE__, #call, got_, want_); \
      ++failures;                                                                                   \
    }                                                                                               \
  } while (0)

// an address that is only compared, far from the others
template <typename T = uint16_t>
static T* at(int k, uintptr_t add = 0) {
  return reinterpret_cast<T*>((uintptr_t(k) << 52) + (uintptr_t(1) << 51) + add);
}

static const int32_t kEdges[] = {INT_MIN, INT_MIN + 8, -1, 0, 1, 7, 8, 16, 24, 1 << 10, 1 << 19, 1 << 20, (1 << 20) + 8,
                                 1 << 28, 1 << 30, INT_MAX - 7, INT_MAX};

static void feed_forward() {
  // every size that is accepted has a workspace that 64 bits hold, and no other has one
  for (const int32_t M : kEdges)
    for (const int32_t E : {INT_MIN, 0, 1, 64, 1024, 1025, INT_MAX})
      for (const int32_t H : kEdges)
        for (const int32_t I : kEdges) {
          const moeq_status st = moeq_grouped_ffn(at(1), at(2), at(3), at<int32_t>(4), M, E, H, I, at<float>(5), at(6), at<void>(7),
                                                  SIZE_MAX, nullptr);
          const size_t need = moeq_grouped_ffn_workspace_bytes(M, E, H, I);
          const size_t back = moeq_grouped_ffn_backward_workspace_bytes(M, E, H, I);
          const bool fits = st == MOEQ_OK;
          EXPECT(need > 0, fits && M > 0);
          if (back > 0) EXPECT(fits, true);
          if (fits && M > 0) {
            EXPECT(need >= (size_t)M * I * 2 && back >= (size_t)M * I * 6, true);
            EXPECT(moeq_grouped_ffn(at(1), at(2), at(3), at<int32_t>(4), M, E, H, I, nullptr, at(6), at<void>(7), need - 1,
                                    nullptr), MOEQ_EWORKSPACE);
            EXPECT(moeq_grouped_ffn_backward(at(1), at(2), at(3), at(4), at<int32_t>(5), at<float>(6), M, E, H, I, MOEQ_DTYPE_FP32,
                                             at(7), at<void>(8), at<void>(9), at<void>(10), back, nullptr), MOEQ_OK);
          }
        }
  int before = launches;
  EXPECT(moeq_grouped_ffn(at(1), at(2), at(3), at<int32_t>(4), 8, 2, 16, 24, nullptr, at(6), at<void>(7), 1 << 20, nullptr),
         MOEQ_OK);
  EXPECT(launches - before, 2);
  before = launches;
  EXPECT(moeq_grouped_ffn_backward(at(1), at(2), at(3), at(4), at<int32_t>(5), at<float>(6), 8, 2, 16, 24, MOEQ_DTYPE_BF16, at(7),
                                   at<void>(8), at<void>(9), at<void>(10), 1 << 20, nullptr), MOEQ_OK);
  EXPECT(launches - before, 4);
  before = launches;   // no rows: the weights' gradients are zeros
  EXPECT(moeq_grouped_ffn_backward(nullptr, nullptr, nullptr, nullptr, at<int32_t>(5), nullptr, 0, 2, 16, 24,
                                   MOEQ_DTYPE_BF16, nullptr, at<void>(8), at<void>(9), nullptr, 0, nullptr), MOEQ_OK);
  EXPECT(launches - before, 2);
  EXPECT(moeq_grouped_ffn(at(1), at(2), at(3), at<int32_t>(4), 8, 2, 16, 24, nullptr, at(1), at<void>(7), 1 << 20, nullptr),
         MOEQ_EINVAL);
}

static void fp8() {
  for (const int32_t fmt : {MOEQ_FMT_FP8_ROW, MOEQ_FMT_FP8_TILE})
    for (const int32_t E : {INT_MIN, 0, 1, 3, 1 << 20, INT_MAX})
      for (const int32_t R : kEdges)
        for (const int32_t C : {INT_MIN, 0, 8, 16, 128, 1 << 20, INT_MAX - 15, INT_MAX}) {
          const moeq_qweight q = {fmt, E, R, C, 128, at<void>(1), at<float>(2), nullptr};
          const int before = launches;
          const moeq_status st = moeq_quantize_fp8(at(3), &q, nullptr);
          EXPECT(launches - before, st == MOEQ_OK);
          if (st == MOEQ_OK) {
            EXPECT(E > 0 && R > 0 && C > 0 && C % 16 == 0, true);
            EXPECT((double)E * R * C <= std::ldexp(1.0, 47), true);
          }
          EXPECT(moeq_dequantize_fp8(&q, at(3), nullptr), st);
          moeq_qweight x = {MOEQ_FMT_FP8_ROW, 1, R, C, 128, at<void>(4), at<float>(5), nullptr};
          const moeq_qweight w = {MOEQ_FMT_FP8_TILE, 3, 16, C, 128, at<void>(6), at<float>(7), nullptr};
          const moeq_status pr = moeq_grouped_mm_fp8(&x, &w, at<int32_t>(8), at(9), nullptr);
          if (pr == MOEQ_OK) EXPECT(R >= 0 && R <= 1 << 28 && C <= 1 << 20, true);
        }
  EXPECT(moeq_quantize_fp8(at(3), nullptr, nullptr), MOEQ_EINVAL);
  moeq_qweight q = {MOEQ_FMT_FP8_TILE, 2, 130, 272, 128, at<void>(1), at<float>(2), nullptr};
  EXPECT(moeq_quantize_fp8(at(1, 2 * 130 * 272 - 16), &q, nullptr), MOEQ_EINVAL);   // the last codes
  EXPECT(moeq_quantize_fp8(at(2, 2 * 2 * 3 * 4 - 16), &q, nullptr), MOEQ_EINVAL);   // the last scales
  EXPECT(moeq_quantize_fp8(at(2, 2 * 2 * 3 * 4), &q, nullptr), MOEQ_OK);            // right behind them
  q.scales = at<float>(2, 4);
  EXPECT(moeq_quantize_fp8(at(3), &q, nullptr), MOEQ_OK);
}

static void orthogonalize() {
  float* table = new float[3];
  table[0] = 3.4445f, table[1] = -4.775f, table[2] = 2.0315f;
  for (const int32_t E : {INT_MIN, 0, 1, 2, 64, 65535, 65536, INT_MAX})
    for (const int32_t N : kEdges)
      for (const int32_t K : kEdges) {
        const size_t need = moeq_orthogonalize_workspace_bytes(E, N, K);
        const moeq_status st =
            moeq_orthogonalize(at<void>(1), MOEQ_DTYPE_FP32, E, N, K, table, 1, at(2), at<void>(3), SIZE_MAX, nullptr);
        EXPECT(st == MOEQ_OK, need > 0);
        if (need == 0) continue;
        const moeq::OrthoPlan p = moeq::ortho_plan(E, N, K);
        const int64_t x = (int64_t)E * N * p.xc * 2, a = (int64_t)E * p.n * p.nc * 2;
        // the parts lie behind each other, each large enough
        EXPECT(p.chunks >= 1 && p.chunks <= 64 && p.x >= (int64_t)E * p.chunks * 8, true);
        EXPECT(p.y >= p.x + x && p.a >= p.y + x && p.p >= p.a + a && p.bytes >= p.p + a, true);
        EXPECT(p.xc >= K && p.xc % 8 == 0 && p.nc >= p.n && p.nc % 8 == 0 && p.n <= p.m, true);
        EXPECT(moeq_orthogonalize(at<void>(1), MOEQ_DTYPE_FP32, E, N, K, table, 1, at(2), at<void>(3), need - 1, nullptr),
               MOEQ_EWORKSPACE);
      }
  EXPECT(moeq_orthogonalize(at<void>(1), MOEQ_DTYPE_BF16, 1, 4, 4, table, 0, at(2), at<void>(3), SIZE_MAX, nullptr),
         MOEQ_EINVAL);
  EXPECT(moeq_orthogonalize(at<void>(1), MOEQ_DTYPE_BF16, 1, 4, 4, table, 65, at(2), at<void>(3), SIZE_MAX, nullptr),
         MOEQ_EINVAL);
  table[2] = INFINITY;
  EXPECT(moeq_orthogonalize(at<void>(1), MOEQ_DTYPE_BF16, 1, 4, 4, table, 1, at(2), at<void>(3), SIZE_MAX, nullptr),
         MOEQ_EINVAL);
  delete[] table;
}

int main() {
  feed_forward();
  fp8();
  orthogonalize();
  if (failures) return 1;
  printf("all checks passed\n");
  return 0;
}
