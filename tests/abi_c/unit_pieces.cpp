// The units of a row and their pieces, for every row length up to 70 and the lengths around some larger multiples: adding
// kernels write each element exactly once, and nothing outside the row.
#include <cstdio>
#include <vector>

#include "gc_internal.h"

static int check(uint32_t n, uint32_t unit, uint32_t ve) {
  std::vector<int> written(n, 0), held(n, 0);
  int outside = 0;
  for (uint32_t u = 0; u < (n + unit - 1) / unit; ++u)
    for (uint32_t off = 0; off < unit; off += ve) {
      const uint32_t s = gci::unit_start(n, unit, u) + off, here = gci::unit_held(n, unit, off, ve);
      for (uint32_t e = 0; e < here; ++e) {
        if (s + e >= n) {
          ++outside;
          continue;
        }
        ++held[s + e];
        if (e >= gci::unit_shared(n, unit, u, off, ve)) ++written[s + e];
      }
    }
  int bad = outside;
  for (uint32_t i = 0; i < n; ++i) bad += written[i] != 1 || held[i] < 1;
  if (bad) std::printf("row of %u, unit %u in pieces of %u: %d wrong\n", n, unit, ve, bad);
  return bad != 0;
}

int main() {
  std::vector<uint32_t> rows;
  for (uint32_t n = 1; n <= 70; ++n) rows.push_back(n);
  for (uint32_t m : {1000u, 4096u, 20000u})
    for (uint32_t n = m - 9; n <= m + 9; ++n) rows.push_back(n);
  int failures = 0;
  for (uint32_t n : rows) failures += check(n, 4, 4) + check(n, 8, 8) + check(n, 8, 4);
  std::printf("%d failures\n", failures);
  return failures != 0;
}
