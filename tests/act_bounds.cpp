// Walks the loads that k_act_wgrad makes of dy through registers
// (csrc/act_wgrad.hip, load_dy) over small matrices and prints the first that
// leaves its matrix.  The rule that picks the unchecked loads is the library's.
#include <algorithm>
#include <cstdio>
#include <cstdlib>

#include "act_bounds.hpp"

// The furthest value past the matrix's last one that any load of dy touches
// (<= 0: none).  bo: the tile's columns, bk: tokens of a step.
static int64_t past_the_end(int64_t rows, int64_t out, int64_t ld, int bo, int bk,
                            int64_t t0, int64_t per, int64_t free_rows) {
  const int lpr = bo / 8, threads = 512, pieces = bk * bo / 8 / threads;
  const int64_t end = (rows - 1) * ld + out;
  const int64_t t1 = std::min(t0 + per, rows);
  const int steps = (int)((t1 - t0 + bk - 1) / bk);
  int64_t worst = -end;
  for (int64_t o0 = 0; o0 < out; o0 += bo)
    for (int st = 0; st <= steps + 1; ++st)          // two steps ahead
      for (int tid = 0; tid < threads; ++tid)
        for (int i = 0; i < pieces; ++i) {
          const int64_t row = t0 + (int64_t)st * bk + tid / lpr + i * (threads / lpr);
          int64_t last;                               // the last value read, from dy
          if (t0 + (int64_t)(st + 1) * bk <= free_rows) {
            last = row * ld + o0 + std::min<int64_t>(tid % lpr * 8, out - 1 - o0) + 7;
          } else {
            const int64_t valid = row < t1 ? out - o0 - tid % lpr * 8 : 0;
            if (valid <= 0) continue;
            last = row * ld + o0 + tid % lpr * 8 + std::min<int64_t>(valid, 8) - 1;
          }
          worst = std::max(worst, last + 1 - end);
        }
  return worst;
}

int main() {
  int bad = 0;
  const int tiles[3][2] = {{256, 32}, {128, 64}, {128, 32}};
  for (auto& t : tiles)
    for (int64_t out : {1, 2, 3, 4, 5, 6, 7, 8, 9, 15, 129})
      for (int64_t pad : {0, 1, 5})
        for (int64_t rows = 1; rows <= 140; ++rows)
          for (int64_t per : {(int64_t)64, (int64_t)192}) {
            const int64_t ld = out + pad;
            const int64_t free_rows = gq::rows_with_room(rows, ld, 7);
            for (int64_t t0 = 0; t0 < rows; t0 += per) {
              const int64_t w = past_the_end(rows, out, ld, t[0], t[1], t0, per, free_rows);
              if (w > 0 && bad++ < 5)
                std::printf("tile %d, step %d: rows %lld, out %lld, ld %lld, from token %lld: "
                            "%lld values past the end\n", t[0], t[1], (long long)rows,
                            (long long)out, (long long)ld, (long long)t0, (long long)w);
            }
          }
  // no row is left out without need
  for (int64_t ld = 1; ld <= 20; ++ld)
    for (int64_t past = 0; past <= 20; ++past) {
      const int64_t r = gq::rows_with_room(100, ld, past);
      if (!((100 - r) * ld >= past && (99 - r) * ld < past) && bad++ < 5)
        std::printf("rows_with_room(100, %lld, %lld) = %lld\n", (long long)ld,
                    (long long)past, (long long)r);
    }
  std::printf("%d bad\n", bad);
  return bad != 0;
}
