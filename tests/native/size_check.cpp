// Host-side check of the size rules that choose between cached and streaming
// accesses (past_caches), at sizes whose byte counts pass 64 bits.  Built with
// the host sanitizers by tests/test_host_sanitizers.py and run on the CPU.
#include <stdint.h>
#include <stdio.h>

#include "launch.h"

namespace {

int failures = 0;

void check(int64_t rows, int64_t per, int64_t cols, int size, bool want) {
  if (fp8fg::past_caches(rows, per, cols, size) == want) return;
  printf("FAIL past_caches(%lld, %lld, %lld, %d)\n", (long long)rows, (long long)per, (long long)cols, size);
  ++failures;
}

}  // namespace

int main() {
  const int64_t limit = fp8fg::kStreamBytes, big = 0x7FFFFFFF;
  for (int size : {2, 4}) {
    check(0, 8, 4096, size, false);
    check(1, 1, 8, size, false);
    check(limit / 8 / 256 / size, 8, 256, size, false);
    check(limit / 8 / 256 / size + 1, 8, 256, size, true);
    for (int64_t rows : {(int64_t)1 << 24, big})
      for (int64_t per : {(int64_t)1 << 20, fp8fg::kCombineMaxK})
        for (int64_t cols : {(int64_t)8, (int64_t)1 << 28}) check(rows, per, cols, size, true);
  }
  // the kernels' steps over the places end without passing int32
  if (fp8fg::kCombineMaxK + 15 > big) {
    printf("FAIL kCombineMaxK\n");
    ++failures;
  }
  printf("%d failures\n", failures);
  return failures == 0 ? 0 : 1;
}
