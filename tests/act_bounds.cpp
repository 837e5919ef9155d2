// Walks index arithmetic of the 8-bit activation kernels on the host; prints
// what is wrong.  The bounds and layouts are the library's (act_bounds.hpp).
//   loads   the loads that k_act_wgrad makes of dy through registers
//           (csrc/act_wgrad.hip, load_dy) stay inside their matrix
//   cover   packing and unpacking (csrc/act_pack.hip) reach every chunk of every
//           row once, in launches that the device takes
#include <algorithm>
#include <cstdio>
#include <cstring>
#include <vector>

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

static int loads() {
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
  return bad;
}

// The launches of `rows` rows: how often each chunk is reached.
static bool covers(int64_t rows, int64_t chunks, int at_once, int64_t most) {
  const gq::Cover c(chunks, at_once, most);
  const int tpr = 1 << c.tlog, per = gq::kCoverThreads >> c.tlog;
  std::vector<int> seen(rows * chunks);
  if (c.rows < 1) return false;
  for (int64_t r = 0; r < rows; r += c.rows) {
    const int64_t n = std::min(rows - r, c.rows), blocks = c.blocks(n);
    if (blocks < 1 || blocks > most) return false;
    for (int64_t b = 0; b < blocks; ++b)
      for (int64_t u = b * at_once; u < (b + 1) * at_once; ++u)
        for (int t = 0; t < gq::kCoverThreads; ++t) {
          const int64_t row = u / c.turns * per + t / tpr, ch = u % c.turns * tpr + t % tpr;
          if (row < n && ch < chunks) ++seen[(r + row) * chunks + ch];
        }
  }
  return std::all_of(seen.begin(), seen.end(), [](int v) { return v == 1; });
}

static int cover() {
  int bad = 0;
  for (int64_t rows : {1, 3, 64, 65, 500})
    for (int64_t chunks : {1, 2, 5, 64, 200, 256, 257, 600})
      for (int at_once : {1, 2})
        for (int64_t most : {3, 7, 1000})
          if (!covers(rows, chunks, at_once, most) && bad++ < 5)
            std::printf("cover: %lld rows of %lld chunks, %d units, %lld workgroups\n",
                        (long long)rows, (long long)chunks, at_once, (long long)most);
  // the largest matrices of every width and group: all taken, in 257 launches at
  // most (2^38 rows of one column, 64 of them per workgroup)
  for (int64_t cols = 1; cols <= 1 << 20; cols = cols < 300 ? cols + 1 : cols * 3 / 2)
    for (int group = 32; group <= 1024; group *= 2) {
      const int64_t rows = (int64_t(1) << 38) / cols, pitch = (cols + 15) / 16 * 16;
      const int G = gq::group_lanes(group, pitch);
      const int64_t whole = ((cols + 7) / 8 + G - 1) / G * G;
      const bool pack = group <= 512;       // longer groups: a walk by stride
      const gq::Cover c = pack ? gq::Cover(whole, 1) : gq::Cover((cols + 7) / 8, 2);
      const int64_t first = std::min(rows, c.rows), n = (rows + c.rows - 1) / c.rows;
      // a group lies in one row's lanes, and all of the pitch is written
      const bool fits = !pack || (G >= 4 && G <= 64 && (G & (G - 1)) == 0 && G <= 1 << c.tlog &&
                                  (G == group / 8 || G >= pitch / 8) && whole * 8 >= pitch);
      if ((c.blocks(first) > gq::kCoverBlocks || !fits || n > 257) && bad++ < 5)
        std::printf("cover: %lld x %lld, group %d: %lld launches of %lld workgroups\n",
                    (long long)rows, (long long)cols, group, (long long)n,
                    (long long)c.blocks(first));
    }
  return bad;
}

int main(int argc, char** argv) {
  const int bad = argc > 1 && !std::strcmp(argv[1], "cover") ? cover() : loads();
  std::printf("%d bad\n", bad);
  return bad != 0;
}
