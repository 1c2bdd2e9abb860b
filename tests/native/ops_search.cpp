// The search by which a wave finds a row's positions among the sorted tokens,
// run on the CPU with 64 lanes in turn: two searches at once over arrays of
// every length up to a few hundred and some long ones.  A lane looks only at
// indexes of the array, also where one search has ended before the other.
#include <stdint.h>
#include <stdio.h>

#include <algorithm>
#include <random>
#include <vector>

#include "zero_ops.h"

using zk::ops::LowerBound;

int main() {
  std::mt19937_64 rng(5);
  int fail = 0;
  long checks = 0;
  auto expect = [&](bool c, const char* what, long long a, long long b) {
    ++checks;
    if (!c && fail++ < 20) fprintf(stderr, "FAIL: %s (%lld, %lld)\n", what, a, b);
  };
  for (int trial = 0; trial < 3000; ++trial) {
    const int64_t n = trial < 600 ? trial : 1 + (int64_t)(rng() % (trial % 50 ? 5000 : 300000));
    const int32_t rows = 1 + (int32_t)(rng() % (trial % 3 ? 100 : 100000));
    std::vector<int32_t> sorted(n);
    for (auto& v : sorted) v = (int32_t)(rng() % rows);
    std::sort(sorted.begin(), sorted.end());
    const int64_t key[2] = {trial % 4 ? (int64_t)(rng() % (rows + 1)) : 0, trial % 5 ? (int64_t)(rng() % (rows + 2)) : rows};
    LowerBound s[2] = {{0, n}, {0, n}};
    int rounds = 0;
    while (s[0].open() || s[1].open()) {
      if (++rounds > 64) break;
      for (int k = 0; k < 2; ++k) {
        int below = 0;
        for (int lane = 0; lane < 64; ++lane) {
          const int64_t i = s[k].probe(lane);
          if (i >= s[k].hi) continue;
          expect(i >= s[k].lo && i >= 0 && i < n, "an index outside the search", i, s[k].lo);
          if (i >= 0 && i < n) below += sorted[i] < key[k];
        }
        s[k].narrow(below);
      }
    }
    for (int k = 0; k < 2; ++k)
      expect(s[k].lo == std::lower_bound(sorted.begin(), sorted.end(), key[k]) - sorted.begin(), "wrong place", s[k].lo, key[k]);
  }
  // One that has ended, wherever it did.
  for (const int64_t at : {int64_t(0), int64_t(1), int64_t(5000)}) {
    LowerBound s{at, at};
    for (int lane = 0; lane < 64; ++lane) expect(s.probe(lane) >= s.hi, "an ended search looks at an index", s.probe(lane), at);
    s.narrow(0);
    expect(s.lo == at && s.hi == at, "an ended search moves", s.lo, at);
  }
  printf("%ld checks, %d failures\n", checks, fail);
  return fail != 0;
}
