// Drives the host code of the grouped products, the MXFP4 format and the
// gradient clipping (no GPU, no kernel launch: the launchers are counting
// stubs), built with AddressSanitizer and UndefinedBehaviorSanitizer on the
// host code.  Pointers handed in are never dereferenced; the descriptors are.
// Exits non-zero on the first result that differs from the documented one.
#include <stdio.h>

#include <climits>
#include <cstdint>
#include <vector>

// The launchers' own host code (table, workspace sizes) is compiled in, but the
// entry points reach the stubs below.
#define launch_clip launch_clip_real
#include "clip.hip"
#undef launch_clip
#define launch_grouped_mm launch_grouped_mm_real
#define launch_grouped_mm_mxfp4 launch_grouped_mm_mxfp4_real
#define launch_grouped_mm_grad_input launch_grouped_mm_grad_input_real
#define launch_grouped_mm_grad_weight launch_grouped_mm_grad_weight_real
#include "grouped.hip"
#undef launch_grouped_mm
#undef launch_grouped_mm_mxfp4
#undef launch_grouped_mm_grad_input
#undef launch_grouped_mm_grad_weight

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
hipError_t launch_grouped_mm_grad_weight(const GroupedArgs&, bool, hipStream_t) { return hit(); }
hipError_t launch_clip(const moeq_grad*, int32_t, double, float*, double*, hipStream_t) { return hit(); }
}  // namespace moeq

#define EXPECT(call, want)                                                                          \
  do {                                                                                              \
    const long long got_ = (long long)(call), want_ = (long long)(want);                            \
    if (got_ != want_) {                                                                            \
      fprintf(stderr, "%s:%d: %s -> %lld, expected %lld\n", __FILE__, __LINE__, #call, got_, want_); \
      ++failures;                                                                                   \
    }                                                                                               \
  } while (0)

// an address that is only compared
template <typename T>
static T* at(uintptr_t a) { return reinterpret_cast<T*>(a); }

constexpr uintptr_t kFar = uintptr_t(1) << 40;   // between the arrays of a call

// Whatever two offsets hold, an expert's rows lie in [0, M).
static void rows_of_an_expert() {
  const int32_t of[] = {INT_MIN, INT_MIN + 1, -5, -1, 0, 1, 7, 8, 9, 1 << 28, INT_MAX - 1, INT_MAX};
  for (const int32_t M : {0, 1, 8, 1 << 28})
    for (const int32_t from : of)
      for (const int32_t to : of) {
        const int64_t lo = from < 0 ? 0 : from < M ? from : M, hi = to < 0 ? 0 : to < M ? to : M;
        const moeq::RowRange r = moeq::row_range(from, to, M);
        EXPECT(r.lo, lo);
        EXPECT(r.n, hi > lo ? hi - lo : 0);
      }
}

static void mxfp4_format() {
  uint16_t* w = at<uint16_t>(kFar);
  moeq_qweight q = {MOEQ_FMT_MXFP4, 3, 5, 64, 32, at<void>(2 * kFar), nullptr, at<uint8_t>(3 * kFar)};
  moeq_qweight bad = q;
  EXPECT(moeq_quantize_mxfp4(w, nullptr, nullptr), MOEQ_EINVAL);
  EXPECT(moeq_dequantize_mxfp4(nullptr, w, nullptr), MOEQ_EINVAL);
  for (int f : {0, 1, 2, 3, 5, -1, INT_MAX}) {
    bad = q; bad.format = f;
    EXPECT(moeq_quantize_mxfp4(w, &bad, nullptr), MOEQ_EFORMAT);
    EXPECT(moeq_dequantize_mxfp4(&bad, w, nullptr), MOEQ_EFORMAT);
  }
  for (int n : {0, -1, INT_MIN}) {
    bad = q; bad.num_experts = n;
    EXPECT(moeq_quantize_mxfp4(w, &bad, nullptr), MOEQ_EINVAL);
    bad = q; bad.rows = n;
    EXPECT(moeq_quantize_mxfp4(w, &bad, nullptr), MOEQ_EINVAL);
    bad = q; bad.cols = n;
    EXPECT(moeq_quantize_mxfp4(w, &bad, nullptr), MOEQ_EINVAL);
  }
  bad = q; bad.cols = 48;
  EXPECT(moeq_quantize_mxfp4(w, &bad, nullptr), MOEQ_EBLOCK);
  bad = q; bad.blocksize = 64;
  EXPECT(moeq_quantize_mxfp4(w, &bad, nullptr), MOEQ_EBLOCK);
  bad = q; bad.scales = at<float>(4 * kFar);
  EXPECT(moeq_quantize_mxfp4(w, &bad, nullptr), MOEQ_EINVAL);
  bad = q; bad.qdata = at<void>(2 * kFar + 8);
  EXPECT(moeq_quantize_mxfp4(w, &bad, nullptr), MOEQ_EALIGN);
  EXPECT(moeq_quantize_mxfp4(at<uint16_t>(kFar + 2), &q, nullptr), MOEQ_EALIGN);
  EXPECT(launches, 0);
  // sizes whose product leaves 64 bits
  for (int e : {1, 1 << 20, INT_MAX}) {
    bad = q; bad.num_experts = e; bad.rows = INT_MAX; bad.cols = INT_MAX / 32 * 32;
    EXPECT(moeq_quantize_mxfp4(w, &bad, nullptr), MOEQ_ESHAPE);
    EXPECT(moeq_dequantize_mxfp4(&bad, w, nullptr), MOEQ_ESHAPE);
    EXPECT(moeq_grouped_mm_mxfp4(&q, &bad, at<int32_t>(4), w, nullptr), MOEQ_ESHAPE);
  }
  EXPECT(launches, 0);
  // as many experts as the field takes
  bad = q; bad.num_experts = INT_MAX; bad.rows = 1; bad.cols = 32;
  EXPECT(moeq_quantize_mxfp4(w, &bad, nullptr), MOEQ_OK);
  // neighbours: the buffers touch, and overlap by one 16-byte step
  const int64_t values = 3 * 5 * 64;
  bad = q; bad.qdata = at<void>(kFar + 2 * values); bad.scale_codes = at<uint8_t>(kFar + 2 * values + values / 2);
  EXPECT(moeq_quantize_mxfp4(w, &bad, nullptr), MOEQ_OK);
  EXPECT(moeq_dequantize_mxfp4(&bad, w, nullptr), MOEQ_OK);
  EXPECT(launches, 3);
  EXPECT(moeq_quantize_mxfp4(w + 8, &bad, nullptr), MOEQ_EINVAL);
  EXPECT(moeq_dequantize_mxfp4(&bad, w + 8, nullptr), MOEQ_EINVAL);
  EXPECT(launches, 3);
}

static void products() {
  launches = 0;
  const int M = 96, E = 4, N = 24, K = 40;
  uint16_t *x = at<uint16_t>(kFar), *w = at<uint16_t>(2 * kFar), *y = at<uint16_t>(3 * kFar);
  const int32_t* off = at<int32_t>(4 * kFar + 4);   // (offsets need no more than their own alignment)
  for (int big : {INT_MAX, INT_MAX - 7, 1 << 30}) {
    EXPECT(moeq_grouped_mm(x, w, off, big, E, N, K, y, nullptr), MOEQ_ESHAPE);
    EXPECT(moeq_grouped_mm(x, w, off, M, big, N, K, y, nullptr), MOEQ_ESHAPE);
    EXPECT(moeq_grouped_mm(x, w, off, M, E, big, K, y, nullptr), MOEQ_ESHAPE);
    EXPECT(moeq_grouped_mm_grad_input(x, w, off, M, E, N, big, y, nullptr), MOEQ_ESHAPE);
    EXPECT(moeq_grouped_mm_grad_weight(x, y, off, M, E, big, K, 1, w, nullptr, 0, nullptr), MOEQ_ESHAPE);
    EXPECT(moeq_grouped_mm_grad_weight_workspace_bytes(big, E, N, K), 0);
    EXPECT(moeq_grouped_mm_grad_weight_workspace_bytes(M, big, N, K), 0);
    EXPECT(moeq_grouped_mm_grad_weight_workspace_bytes(M, E, N, big), 0);
  }
  for (int small : {0, -1, INT_MIN}) {
    EXPECT(moeq_grouped_mm(x, w, off, M, small, N, K, y, nullptr), MOEQ_EINVAL);
    EXPECT(moeq_grouped_mm(x, w, off, M, E, small, K, y, nullptr), MOEQ_EINVAL);
    EXPECT(moeq_grouped_mm_grad_input(x, w, off, M, E, N, small, y, nullptr), MOEQ_EINVAL);
  }
  EXPECT(moeq_grouped_mm(x, w, off, -1, E, N, K, y, nullptr), MOEQ_EINVAL);
  EXPECT(launches, 0);
  EXPECT(moeq_grouped_mm(x, w, off, M, E, N, K, y, nullptr), MOEQ_OK);
  EXPECT(moeq_grouped_mm_grad_input(x, w, off, M, E, N, K, y, nullptr), MOEQ_OK);
  EXPECT(moeq_grouped_mm_grad_weight(x, y, off, M, E, N, K, MOEQ_DTYPE_FP32, w, nullptr, 0, nullptr), MOEQ_OK);
  EXPECT(moeq_grouped_mm_grad_weight(nullptr, nullptr, off, 0, E, N, K, MOEQ_DTYPE_FP32, w, nullptr, 0, nullptr),
         MOEQ_OK);   // zeros
  EXPECT(moeq_grouped_mm_grad_weight(x, x, off, M, E, N, N, MOEQ_DTYPE_BF16, w, nullptr, 0, nullptr), MOEQ_OK);
  EXPECT(launches, 5);
  // a result between two operands that touches both, then one step into each
  uint16_t *y0 = x + M * K, *w0 = y0 + M * N;
  EXPECT(moeq_grouped_mm(x, w0, off, M, E, N, K, y0, nullptr), MOEQ_OK);
  EXPECT(moeq_grouped_mm(x, w0, off, M, E, N, K, y0 - 8, nullptr), MOEQ_EINVAL);
  EXPECT(moeq_grouped_mm(x, w0, off, M, E, N, K, y0 + 8, nullptr), MOEQ_EINVAL);
  // operands may share memory
  EXPECT(moeq_grouped_mm(x, x, off, M, E, N, K, y, nullptr), MOEQ_OK);
  EXPECT(launches, 7);

  // MXFP4: the same for codes and scales; no rows reach no launcher
  moeq_qweight xq = {MOEQ_FMT_MXFP4, 1, M, 64, 32, at<void>(kFar), nullptr, at<uint8_t>(5 * kFar)};
  moeq_qweight wq = {MOEQ_FMT_MXFP4, E, N, 64, 32, at<void>(2 * kFar), nullptr, at<uint8_t>(6 * kFar)};
  EXPECT(moeq_grouped_mm_mxfp4(&xq, &wq, off, y, nullptr), MOEQ_OK);
  EXPECT(moeq_grouped_mm_mxfp4(&xq, &wq, off, at<uint16_t>(kFar + M * 32), nullptr), MOEQ_OK);
  EXPECT(moeq_grouped_mm_mxfp4(&xq, &wq, off, at<uint16_t>(kFar + M * 32 - 16), nullptr), MOEQ_EINVAL);
  EXPECT(launches, 9);
  moeq_qweight none = {MOEQ_FMT_MXFP4, 1, 0, 64, 32, nullptr, nullptr, nullptr};
  EXPECT(moeq_grouped_mm_mxfp4(&none, &wq, nullptr, nullptr, nullptr), MOEQ_OK);
  EXPECT(moeq_grouped_mm_mxfp4(nullptr, &wq, off, y, nullptr), MOEQ_EINVAL);
  EXPECT(moeq_grouped_mm_mxfp4(&xq, nullptr, off, y, nullptr), MOEQ_EINVAL);
  wq.num_experts = INT_MAX;
  EXPECT(moeq_grouped_mm_mxfp4(&xq, &wq, off, y, nullptr), MOEQ_ESHAPE);
  xq.rows = INT_MAX;
  EXPECT(moeq_grouped_mm_mxfp4(&xq, &wq, off, y, nullptr), MOEQ_ESHAPE);
  EXPECT(launches, 9);

  // Segments: every expert's rows fit the segments that the workspace has
  // room for, whatever the sizes.
  for (int32_t m : {0, 1, 511, 512, 513, 100000, 1 << 20, (1 << 28) - 1, 1 << 28})
    for (int32_t n : {8, 64, 72, 4096, 1 << 20})
      for (int32_t k : {8, 64, 72, 4096, 1 << 20}) {
        const int32_t seg = moeq::grad_weight_segment(m, n, k);
        EXPECT(seg >= 512 && seg % 64 == 0, 1);
        // the worst split: as many experts as can have just more than one segment
        const int64_t experts = m / (seg + 1);
        EXPECT(moeq::grad_weight_slots(m, seg) >= (experts > 0 ? (m - experts * (seg + 1)) / seg + 2 * experts : 0), 1);
      }
  EXPECT(moeq_grouped_mm_grad_weight_workspace_bytes(1 << 28, 1024, 1 << 15, 1 << 14) % 16, 0);
}

static void clipping() {
  launches = 0;
  float* norm = at<float>(kFar);
  void* ws = at<void>(2 * kFar);
  EXPECT(moeq_clip_grad_norm_workspace_bytes(-1), 0);
  EXPECT(moeq_clip_grad_norm_workspace_bytes(INT_MIN), 0);
  EXPECT(moeq_clip_grad_norm_workspace_bytes(INT_MAX) > moeq_clip_grad_norm_workspace_bytes(INT_MAX - 96), 1);
  EXPECT(moeq_clip_grad_norm_workspace_bytes(0) >= 16, 1);
  // tensors in a row, in place and into other buffers, in an order of their own
  std::vector<moeq_grad> g;
  uintptr_t src = 3 * kFar, dst = 4 * kFar;
  for (int i = 0; i < 300; ++i) {
    const int64_t n = i % 7 == 3 ? 0 : (i * 37) % 900 + 1;
    const int32_t dtype = i % 2 ? MOEQ_DTYPE_FP32 : MOEQ_DTYPE_BF16;
    g.push_back({n ? at<void>(src) : nullptr, n ? at<void>(i % 3 ? dst : src) : nullptr, n, dtype});
    src += (uintptr_t)((n * 4 + 3) / 4 * 4);
    dst += (uintptr_t)((n * 4 + 3) / 4 * 4);
  }
  for (size_t i = 0; i < g.size(); ++i) std::swap(g[i], g[(i * 7919) % g.size()]);
  const size_t need = moeq_clip_grad_norm_workspace_bytes((int32_t)g.size());
  auto clip = [&](double max_norm = 1.0) {
    return moeq_clip_grad_norm(g.data(), (int32_t)g.size(), max_norm, norm, ws, need, nullptr);
  };
  EXPECT(clip(), MOEQ_OK);
  EXPECT(clip(0.0), MOEQ_OK);
  EXPECT(clip(__builtin_inf()), MOEQ_OK);
  EXPECT(launches, 3);
  EXPECT(clip(-1.0), MOEQ_EINVAL);
  EXPECT(clip(__builtin_nan("")), MOEQ_EINVAL);
  for (size_t i = 0; i < g.size(); i += 13) {
    if (g[i].numel == 0) continue;
    const moeq_grad keep = g[i];
    g[i].numel = int64_t(1) << 38;
    EXPECT(clip(), MOEQ_EINVAL);
    g[i] = keep; g[i].numel = INT64_MIN;
    EXPECT(clip(), MOEQ_EINVAL);
    g[i] = keep; g[i].dst = g[(i + 1) % g.size()].numel ? const_cast<void*>(g[(i + 1) % g.size()].src) : at<void>(src - 4);
    if (g[(i + 1) % g.size()].numel) EXPECT(clip(), MOEQ_EINVAL);
    g[i] = keep; g[i].dst = norm;
    EXPECT(clip(), MOEQ_EINVAL);
    g[i] = keep; g[i].dtype = 0;
    EXPECT(clip(), MOEQ_EFORMAT);
    g[i] = keep;
  }
  EXPECT(clip(), MOEQ_OK);
  EXPECT(launches, 4);
  EXPECT(moeq_clip_grad_norm(nullptr, 0, 1.0, norm, ws, need, nullptr), MOEQ_OK);
  EXPECT(moeq_clip_grad_norm(nullptr, 1, 1.0, norm, ws, need, nullptr), MOEQ_EINVAL);

  // The launches' tables hold every tensor that is not empty, once, in order,
  // and their chunks cover it.
  std::vector<int> seen;
  for (int32_t from = 0; from < (int32_t)g.size();) {
    moeq::Table t;
    const int32_t next = moeq::fill(t, g.data(), (int32_t)g.size(), from);
    EXPECT(next > from, 1);
    EXPECT(t.count <= moeq::kTable, 1);
    int32_t i = from;
    int64_t chunks = 0;
    for (int k = 0; k < t.count; ++k, ++i) {
      while (g[i].numel == 0) ++i;
      seen.push_back(i);
      EXPECT(t.e[k].src == g[i].src && t.e[k].dst == g[i].dst && t.e[k].n == g[i].numel, 1);
      EXPECT(t.e[k].first, chunks);
      const bool fp32 = (t.fp32[k >> 5] >> (k & 31)) & 1u;
      EXPECT(fp32, g[i].dtype == MOEQ_DTYPE_FP32);
      chunks += (g[i].numel + moeq::chunk_of(fp32) - 1) / moeq::chunk_of(fp32);
    }
    EXPECT(t.chunks, chunks);
    from = next;
  }
  size_t live = 0;
  for (const moeq_grad& x : g) live += x.numel > 0;
  EXPECT(seen.size(), live);
}

int main() {
  rows_of_an_expert();
  mxfp4_format();
  products();
  clipping();
  if (failures) fprintf(stderr, "%d check(s) failed\n", failures);
  else printf("grouped driver: all checks passed\n");
  return failures ? 1 : 0;
}
