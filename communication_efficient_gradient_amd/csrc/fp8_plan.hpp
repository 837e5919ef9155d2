// fp8_plan.hpp — which kernel the 8-bit floating point product takes, in plain
// C++: the launcher asks it, and host tests.
#pragma once

#include <stdint.h>

#include "act_bounds.hpp"

namespace gq {

// Which of the two: a workgroup of k_fp8_linear_few reads the codes of its tokens (up
// to 32) from L2 for 16 or 32 outputs, the tiled kernel once for 64.  That is
// little beside the weight up to 4 tokens; from there on what one CU reads so
// decides, in rows, which is compared below: of one weight by whole rounds of
// workgroups, of several experts, whose workgroups end at different times, all in
// all.  Measured (us here / there, bf16, tokens x out x cols; what is compared
// behind it):
//    1 x 16384 x 8192 22.3 / 22.6          4 x 4096 x 4096  6.7 / 11.9
//   64 x 4096 x 4096 10.8 / 12.1 (32)     16 x 8192 x 8192 17.9 / 16.6 (32)
//   17 x 8192 x 8192 20.0 / 16.7 (34)      8 x 20000 x 8192 32.8 / 31.8 (40)
//   12 x 16384 x 8192 29.8 / 23.0 (48)    32 x 4608 x 8192 25.5 / 14.2 (64)
// Several experts, tokens over experts x out x cols, even loads / uneven ones:
//   64 over 2 x 2048 x 2048  6.7 8.4 / 8.9 8.9 (32)
//   24 over 3 x 5120 x 5120  19.3 19.6 / 16.3 16.4 (30)
//   64 over 16 x 2050 x 4100 25.8 26.9 / 34.6 34.3 (32)
//   60 over 6 x 3000 x 1500  7.8 8.1 / 10.8 10.7 (44)
//   48 over 4 x 4096 x 4096  17.7 19.6 / 14.8 14.8 (48)
//   24 over 3 x 12000 x 1200 11.8 11.8 / 14.9 14.8 (70)
//   64 over 2 x 4096 x 4096  18.8 21.1 / 13.0 13.1 (64)
//   32 over 2 x 8192 x 8192  34.4 42.8 / 23.2 23.5 (64)
//   64 over 64 x 4096 x 1024 78.9 50.1 / 50.6 30.7 (64)
//   64 over 2 x 8192 x 8192  64.3 72.8 / 23.4 24.4 (128)
// (1068 such pairs: 46 is 1.2 % over the faster one of each in the mean, 27 % at
// most beyond the limit and 49 % below it; the kernel for few tokens always 4.7 %
// and up to 199 %.)
inline bool few_tokens(int64_t rows, int64_t out, int experts) {
  if (rows <= 4 || rows > 64) return rows <= 4;
  const int64_t groups = (out + 15) / 16;
  if (experts > 1) return groups * rows <= 46 * kCus;
  return ((rows <= 32 ? groups : 2 * ((out + 31) / 32)) + kCus - 1) / kCus *
             (rows < 32 ? rows : 32) <= 32;
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
