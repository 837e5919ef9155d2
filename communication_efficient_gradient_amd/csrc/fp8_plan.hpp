// fp8_plan.hpp — which kernel the 8-bit floating point product takes, in plain
// C++: the launcher asks it, and host tests.
#pragma once

#include <stdint.h>

#include "act_bounds.hpp"

namespace gq {

// Which of the two: a workgroup of k_fp8_linear_few reads the codes of its tokens (up to
// 32) from L2 for 16 or 32 outputs, the tiled kernel once for 64.  That is
// little beside the weight up to 4 tokens; from there on what one CU reads so
// decides, which is compared below.  Measured (us here / there, bf16, tokens x
// out x cols; what is compared behind it):
//    1 x 16384 x 8192 22.3 / 22.6          4 x 4096 x 4096  6.7 / 11.9
//   64 x 4096 x 4096 10.8 / 12.1 (32)     16 x 8192 x 8192 17.9 / 16.6 (32)
//   17 x 8192 x 8192 20.0 / 16.7 (34)      8 x 20000 x 8192 32.8 / 31.8 (40)
//   12 x 16384 x 8192 29.8 / 23.0 (48)    32 x 4608 x 8192 25.5 / 14.2 (64)
// Several experts: 32 tokens over 16 x 1024 x 2048 7.5 / 9.6, 64 over 8 x 2048 x
// 2048 8.6 / 8.9, 64 over 64 x 1024 x 1024 15.0 / 17.7, 128 over 32 x 2048 x
// 2048 31.1 / 22.4.
inline bool few_tokens(int64_t rows, int64_t out, int experts) {
  if (rows <= 4 || rows > 64) return rows <= 4;
  if (experts > 1) return true;
  const int64_t groups = rows <= 32 ? (out + 15) / 16 : 2 * ((out + 31) / 32);
  return (groups + kCus - 1) / kCus * (rows < 32 ? rows : 32) <= 32;
}

struct LinearPlan {
  int tile;         // rows and columns of a tile; 0: the kernel for few tokens
  int teams;        // of waves that share one
  int splits, per;  // of the sum, and 128-byte k-tiles of one
  int64_t grid;     // workgroups
};

// Tile, teams and splits by an estimate of the time in microseconds: rounds of
// workgroups, a k-tile each, what a tile costs besides, and the parts' way through
// memory and back.  How the tokens are spread over several experts is not known
// here: the estimate takes them to be spread evenly, the grid holds any table's
// tiles.  Two teams take one tile each, so any table's tiles have to be within the
// chip's CUs, splits included.  Measured (bf16, whole call): 1024 x 4096 x 4096 26
// us with 128-tiles, 37 with 64, 48 with 256; 256 x 4096 x 4096 12.7 with 64; 100 x
// 1024 x 8192 20.3 whole, 14.0 in 8; 512 x 2048 x 8192 21.5 whole, 28.6 in 2; 1111
// over 3 x 100 x 16000 17.3 in 6 by two teams, 18.6 to 20.7 in 7, which are too many
// for them.
inline LinearPlan plan_linear(int64_t rows, int k_tiles, int64_t out, int experts) {
  LinearPlan best = {0, 1, 1, k_tiles, 0};
  if (few_tokens(rows, out, experts)) return best;
  double least = 1e30;
  const int64_t each = (rows + experts - 1) / experts;
  const int64_t used = (rows + each - 1) / each;
  for (int tile = 64; tile <= 256; tile *= 2) {
    const int64_t columns = (out + tile - 1) / tile;
    const int64_t tiles = used * ((each + tile - 1) / tile) * columns;
    for (int s = 1; s <= 8 && (s == 1 || k_tiles / s >= 8); ++s) {
      const int per = (k_tiles + s - 1) / s, splits = (k_tiles + per - 1) / per;
      const int64_t most = ragged_tiles(rows, experts, tile) * columns * splits;
      const int teams = tile == 64 && most <= kCus ? 2 : 1;
      const int64_t slots = tile == 64 && teams == 1 ? 2 * kCus : kCus;   // the chip's
      const double rounds = (double)((tiles * splits + slots - 1) / slots);
      double t;
      if (tile == 256) t = rounds * (per * 1.6 + 12.0);
      else if (tile == 128) t = rounds * (per * 0.6 + 5.0);
      else if (teams == 2) t = per * 0.24 + 4.0;
      else t = rounds * (per * 0.44 + 4.0);
      if (splits > 1) t += 6.0 + 8.0 * (double)(splits * rows) * (double)out / 2.4e6;
      if (t < least) {
        least = t;
        best = {tile, teams, splits, per, most < slots ? most : slots};
      }
    }
  }
  return best;
}

}  // namespace gq
