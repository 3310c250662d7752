// Drives the host code of the grouped products, the MXFP4 format and the
// gradient clipping (no GPU, no kernel launch), built with AddressSanitizer
// and UndefinedBehaviorSanitizer on the host code.  Exits non-zero on the
// first result that differs from the documented one.
#include <stdio.h>

#include <climits>
#include <cstdint>

#include "grouped.h"

static int failures = 0;
#define EXPECT(call, want)                                                                          \
  do {                                                                                              \
    const long long got_ = (long long)(call), want_ = (long long)(want);                            \
    if (got_ != want_) {                                                                            \
      fprintf(stderr, "%s:%d: %s -> %lld, expected %lld\n", __FILE__, __LINE__, #call, got_, want_); \
      ++failures;                                                                                   \
    }                                                                                               \
  } while (0)

// Whatever two offsets hold, an expert's rows lie in [0, M).
static void rows_of_an_expert() {
  const int32_t at[] = {INT_MIN, INT_MIN + 1, -5, -1, 0, 1, 7, 8, 9, 1 << 28, INT_MAX - 1, INT_MAX};
  for (const int32_t M : {0, 1, 8, 1 << 28})
    for (const int32_t from : at)
      for (const int32_t to : at) {
        const int64_t lo = from < 0 ? 0 : from < M ? from : M, hi = to < 0 ? 0 : to < M ? to : M;
        const moeq::RowRange r = moeq::row_range(from, to, M);
        EXPECT(r.lo, lo);
        EXPECT(r.n, hi > lo ? hi - lo : 0);
      }
}

int main() {
  rows_of_an_expert();
  if (failures) fprintf(stderr, "%d check(s) failed\n", failures);
  else printf("grouped driver: all checks passed\n");
  return failures ? 1 : 0;
}
