// Walks through the parts of random ranges of rows as the weight gradient by
// expert counts them, and compares with what its grid and workspace hold.
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "act_bounds.hpp"

int main() {
  std::mt19937_64 rng(7);
  long checked = 0;
  for (int turn = 0; turn < 200000; ++turn) {
    const int64_t rows = 1 + (int64_t)(rng() % (turn % 3 == 0 ? 200 : turn % 3 == 1 ? 5000 : 200000));
    const int ranges = 1 + (int)(rng() % (turn % 2 ? 9 : 200));
    const int64_t most = 1 + (int64_t)(rng() % (turn % 5 ? 40 : 4));
    std::vector<int64_t> at(ranges + 1);
    for (auto& v : at) v = (int64_t)(rng() % (uint64_t)(rows + 1));
    if (turn % 7 == 0)
      for (auto& v : at) v = v / 64 * 64 + 1 <= rows ? v / 64 * 64 + 1 : rows;
    // ascending, from 0 to rows or inside
    for (size_t i = 1; i < at.size(); ++i)
      for (size_t j = i; j > 0 && at[j - 1] > at[j]; --j) std::swap(at[j - 1], at[j]);
    if (turn % 4) at.front() = 0, at.back() = rows;
    int64_t steps = 0, split = 0, parts = 0, units = 0;
    for (int e = 0; e < ranges; ++e) {
      const int64_t n = (at[e + 1] - at[e] + 63) / 64;
      const int64_t s = n > most ? (n + most - 1) / most : 1;
      steps += n;
      split += s > 1;
      parts += s > 1 ? s : 0;
      units += s;
    }
    const gq::UnitBounds b(rows, ranges, most);
    if (steps > b.steps || split > b.split || parts > b.parts || units > b.units) {
      std::printf("rows %ld ranges %d most %ld: %ld %ld %ld %ld over %ld %ld %ld %ld\n", (long)rows,
                  ranges, (long)most, (long)steps, (long)split, (long)parts, (long)units,
                  (long)b.steps, (long)b.split, (long)b.parts, (long)b.units);
      return 1;
    }
    ++checked;
  }
  std::printf("ok %ld\n", checked);
  return 0;
}
