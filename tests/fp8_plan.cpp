// With arguments rows, k_tiles, out, experts (any number of times four): prints the
// product's plan for each.  Without: walks random tables through random plans, and
// says what does not hold.
#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "fp8_plan.hpp"

static int walk() {
  std::mt19937_64 rng(5);
  auto upto = [&](int64_t n) { return 1 + (int64_t)(rng() % (uint64_t)n); };
  long two = 0, split = 0, both = 0;
  for (int turn = 0; turn < 200000; ++turn) {
    const int64_t rows = upto(turn % 3 == 0 ? 300 : turn % 3 == 1 ? 3000 : 40000);
    const int64_t out = upto(turn % 2 ? 300 : 9000);
    const int k_tiles = (int)upto(turn % 4 ? 140 : 12);
    const int experts = turn % 5 == 0 ? 1 : (int)upto(turn % 5 < 3 ? 8 : 1024);
    const gq::LinearPlan p = gq::plan_linear(rows, k_tiles, out, experts);
    const char* wrong = nullptr;
    if (p.splits < 1 || p.per < 1 || (int64_t)p.splits * p.per < k_tiles ||
        (int64_t)(p.splits - 1) * p.per >= k_tiles)
      wrong = "splits";
    if (p.tile == 0) {
      if (p.splits != 1 || p.teams != 1) wrong = "few tokens";
    } else {
      // tiles of a table, ascending within the rows
      std::vector<int64_t> at(experts + 1);
      for (auto& v : at) v = (int64_t)(rng() % (uint64_t)(rows + 1));
      std::sort(at.begin(), at.end());
      if (turn % 4) at.front() = 0, at.back() = rows;
      int64_t tiles = 0;
      for (int e = 0; e < experts; ++e) tiles += (at[e + 1] - at[e] + p.tile - 1) / p.tile;
      tiles *= (out + p.tile - 1) / p.tile * p.splits;
      const int64_t slots = p.tile == 64 && p.teams == 1 ? 2 * gq::kCus : gq::kCus;
      if (p.grid < 1 || p.grid > slots || (p.grid < slots && p.grid < tiles)) wrong = "grid";
      // two teams take one tile and leave
      if (p.teams == 2 && (p.tile != 64 || tiles > p.grid)) wrong = "teams";
      // where any table's tiles are alone on their CUs, two teams take them
      const int64_t most =
          gq::ragged_tiles(rows, experts, p.tile) * ((out + p.tile - 1) / p.tile) * p.splits;
      if (p.tile == 64 && (p.teams == 2) != (most <= gq::kCus)) wrong = "which kernel";
      two += p.teams == 2;
      split += p.splits > 1;
      both += p.teams == 2 && p.splits > 1;
    }
    if (wrong) {
      std::printf("%s: rows %ld k_tiles %d out %ld experts %d: tile %d teams %d splits %d per %d "
                  "grid %ld\n", wrong, (long)rows, k_tiles, (long)out, experts, p.tile, p.teams,
                  p.splits, p.per, (long)p.grid);
      return 1;
    }
  }
  std::printf("ok %ld %ld %ld\n", two, split, both);
  return 0;
}

int main(int argc, char** argv) {
  if (argc < 5) return walk();
  for (int i = 1; i + 3 < argc; i += 4) {
    const gq::LinearPlan p = gq::plan_linear(std::atol(argv[i]), std::atoi(argv[i + 1]),
                                             std::atol(argv[i + 2]), std::atoi(argv[i + 3]));
    std::printf("%d %d %d %d %ld\n", p.tile, p.teams, p.splits, p.per, (long)p.grid);
  }
  return 0;
}
