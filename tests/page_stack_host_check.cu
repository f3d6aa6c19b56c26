// Host-side check of the free stack's test (page_stack.cuh) against 64-bit arithmetic.
// Built and run by tests/test_page_stack_host.py; prints "ok <cases>" or the first failures.
#include <climits>
#include <cstdio>

#include "page_stack.cuh"

int main() {
  const int n0s[] = {INT_MIN, INT_MIN + 1, -1, 0, 1, 2, 63, 64, 65, 1 << 20, INT_MAX - 64, INT_MAX - 1, INT_MAX};
  const int backs[] = {0, 1, 2, 63, 64, 65, 1 << 20, INT_MAX - 1, INT_MAX};
  const int pages[] = {1, 2, 64, 65, 1 << 20, INT_MAX - 1, INT_MAX};
  int cases = 0, fails = 0;
  for (int n0 : n0s)
    for (int back : backs)
      for (int p : pages) {
        ++cases;
        const bool want = n0 >= 0 && (long long)n0 + back <= p;
        if (specv::page_stack_holds(n0, back, p) != want && fails++ < 5) std::printf("%d %d %d\n", n0, back, p);
      }
  if (fails) return 1;
  std::printf("ok %d\n", cases);
  return 0;
}
