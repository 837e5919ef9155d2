// act_bounds.hpp — index bounds of the 8-bit activation kernels, in plain C++:
// what the launchers and kernels use is what the host tests walk through.
#pragma once

#include <stdint.h>

namespace gq {

constexpr int kCus = 256;  // compute units

// Of a matrix of `rows` rows with stride `ld`, how many (from the first on) let
// `past` more values be read behind their last column without leaving the
// matrix: those values lie in the following rows, ceil(past / ld) of them.  None
// where there are no rows: then the stride may be anything, 0 too.
constexpr int64_t rows_with_room(int64_t rows, int64_t ld, int64_t past) {
  return rows > 0 ? rows - (past + ld - 1) / ld : 0;
}

// The smallest p with 2^p >= v.
constexpr int log2_up(int64_t v) {
  int p = 0;
  while ((int64_t(1) << p) < v) ++p;
  return p;
}

// Threads of a workgroup that packs or unpacks, and the most such workgroups
// of a launch, which holds fewer than 2^32 threads.
constexpr int kCoverThreads = 256;
constexpr int64_t kCoverBlocks = (int64_t(1) << 32) / kCoverThreads - 1;

// How rows of `chunks` chunks are laid over workgroups.  2^tlog threads share a
// row and take its chunks in `turns`; a unit is one turn of kCoverThreads /
// 2^tlog rows, a workgroup takes `at_once` units.  `rows`: what one launch of
// at most `most` workgroups covers.
struct Cover {
  int tlog, turns, at_once;
  int64_t rows;

  constexpr Cover(int64_t chunks, int at_once, int64_t most = kCoverBlocks)
      : tlog(log2_up(chunks < kCoverThreads ? chunks : kCoverThreads)),
        turns((int)((chunks + (1 << tlog) - 1) >> tlog)),
        at_once(at_once),
        rows(most * at_once / turns * (kCoverThreads >> tlog)) {}

  constexpr int64_t blocks(int64_t n) const {
    const int64_t per = kCoverThreads >> tlog;
    return ((n + per - 1) / per * turns + at_once - 1) / at_once;
  }
};

// Lanes that share a step where a group is `group` columns, 32 .. 512: of a row
// that is shorter than its one group, those that hold it (4 at least).
constexpr int group_lanes(int group, int64_t pitch) {
  const int row = 1 << log2_up(pitch / 8 > 4 ? pitch / 8 : 4);
  return group / 8 < row ? group / 8 : row;
}

// Tiles of `tile` rows that ranges one after the other within `rows` rows have at
// most: each range with rows in it may end inside one.
constexpr int64_t ragged_tiles(int64_t rows, int64_t ranges, int64_t tile) {
  const int64_t some = ranges < rows ? ranges : rows;
  return (rows + some * (tile - 1)) / tile;
}

// Rows of several ranges are summed in steps of 64, a range of more than `most`
// steps in parts of up to `most`.  What a grid and a workspace have to hold for
// any ranges that lie one after the other within `rows` rows.
struct UnitBounds {
  int64_t steps;    // of all ranges: each may end inside one
  int64_t split;    // ranges that have parts
  int64_t parts;
  int64_t units;    // parts, and ranges without

  static constexpr int64_t steps_of(int64_t rows, int64_t ranges) {
    return rows / 64 + (ranges < rows ? ranges : rows);
  }

  // a range of n > most steps has at most n / most + 1 parts
  constexpr UnitBounds(int64_t rows, int64_t ranges, int64_t most)
      : steps(steps_of(rows, ranges)),
        split(steps / (most + 1) < ranges ? steps / (most + 1) : ranges),
        parts(split > 0 ? steps / most + split : 0),
        units(ranges + parts) {}
};

}  // namespace gq
