// act_bounds.hpp — index bounds of the 8-bit activation kernels, in plain C++:
// what the launchers and kernels use is what the host tests walk through.
#pragma once

#include <stdint.h>

namespace gq {

// Of a matrix of `rows` rows with stride `ld`, how many (from the first on) let
// `past` more values be read behind their last column without leaving the
// matrix: those values lie in the following rows, ceil(past / ld) of them.
constexpr int64_t rows_with_room(int64_t rows, int64_t ld, int64_t past) {
  return rows - (past + ld - 1) / ld;
}

}  // namespace gq
