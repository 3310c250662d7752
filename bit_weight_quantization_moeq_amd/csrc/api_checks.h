// Checks that the C entry points share.  All run on the host before the first
// HIP call, so that a rejected call has no side effect.
#pragma once

#include <initializer_list>

#include "grouped.h"

namespace moeq {
namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

moeq_status device_status(hipError_t e) { return e == hipSuccess ? MOEQ_OK : MOEQ_EDEVICE; }

constexpr int32_t kMaxDim = 1 << 20;     // N and K of a grouped product
constexpr int64_t kMaxExpertBytes = int64_t(1) << 31;
constexpr int32_t kMaxRows = 1 << 28;    // M of a grouped product

[[maybe_unused]] moeq_status check_grouped(int32_t M, int32_t E, int32_t N, int32_t K) {
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
[[maybe_unused]] Span bf16(const uint16_t* p, int64_t rows, int64_t cols) { return {p, rows * cols * 2}; }
[[maybe_unused]] Span ints(const int32_t* offsets, int32_t E) { return {offsets, (E + int64_t(1)) * 4}; }

}  // namespace
}  // namespace moeq
