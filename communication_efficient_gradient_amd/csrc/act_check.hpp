// act_check.hpp — the argument checks that the C entry points of the operators
// of a training step share.  Host only.
#pragma once

#include <cmath>
#include <cstdint>

#include "act.hpp"
#include "gq.h"

namespace {

constexpr int64_t kMaxElements = int64_t(1) << 38;
constexpr int64_t kMaxCols = int64_t(1) << 20;
constexpr int64_t kMaxLinearCols = 131071;  // 2^7 * 2^7 * cols < 2^31
constexpr int64_t kMaxTiles = int64_t(1) << 24;  // of 64 x 64 results

bool aligned(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

int64_t dtype_bytes(int dtype) { return dtype == GQ_F32 ? 4 : 2; }

int check_act(const gq_act* a, gq::ActDims* A) {
  if (a == nullptr) return GQ_EINVAL;
  if (a->rows < 0 || a->cols < 1 || a->cols > kMaxCols) return GQ_EINVAL;
  if (a->rows > kMaxElements / a->cols) return GQ_EINVAL;
  if (a->dtype != GQ_F32 && a->dtype != GQ_BF16 && a->dtype != GQ_F16)
    return GQ_EUNSUPPORTED;
  const int g = a->group;
  if (g != 0 && (g < 32 || g > 32768 || (g & (g - 1)) != 0)) return GQ_EINVAL;
  A->rows = a->rows;
  A->cols = a->cols;
  A->pitch = (a->cols + 15) / 16 * 16;
  A->dtype = a->dtype;
  A->whole_row = g == 0;
  A->group = g == 0 ? (int)A->pitch : g;
  A->groups = g == 0 ? 1 : (int)((a->cols + g - 1) / g);
  return GQ_OK;
}

int check_out(const gq::ActDims& A, int64_t out) {
  if (out < 1 || out > kMaxCols) return GQ_EINVAL;
  if (A.rows > kMaxElements / out || out > kMaxElements / A.cols) return GQ_EINVAL;
  return GQ_OK;
}

// One step per row, sums that 32 bits hold, tiles that one launch numbers.
int check_linear(const gq::ActDims& A, int64_t out) {
  if (!A.whole_row || A.cols > kMaxLinearCols) return GQ_EUNSUPPORTED;
  if ((A.rows + 63) / 64 > kMaxTiles / ((out + 63) / 64)) return GQ_EUNSUPPORTED;
  return GQ_OK;
}

// A range of device memory a call reads or writes.
struct Range {
  const void* p;
  int64_t bytes;
};

bool overlap(const Range& a, const Range& b) {
  if (!a.p || !b.p || a.bytes == 0 || b.bytes == 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x < y + (uintptr_t)b.bytes && y < x + (uintptr_t)a.bytes;
}

// Whether a written range meets any other range of the call.
template <int NW, int NR>
bool any_overlap(const Range (&w)[NW], const Range (&r)[NR]) {
  for (int i = 0; i < NW; ++i) {
    for (int j = i + 1; j < NW; ++j)
      if (overlap(w[i], w[j])) return true;
    for (int j = 0; j < NR; ++j)
      if (overlap(w[i], r[j])) return true;
  }
  return false;
}

// A strided matrix of the activations' type; false if it cannot be one.
bool matrix(const gq::ActDims& A, const void* p, int64_t cols, int64_t ld, Range* r) {
  const int64_t e = dtype_bytes(A.dtype);
  *r = {p, 0};
  if (A.rows == 0) return true;
  if (p == nullptr || !aligned(p, (uintptr_t)e) || ld < cols) return false;
  if (ld > (kMaxElements * 4) / A.rows) return false;
  r->bytes = ((A.rows - 1) * ld + cols) * e;
  return true;
}

bool same(const Range& a, int64_t lda, const Range& b, int64_t ldb) {
  return a.p == b.p && lda == ldb;
}

// An 8-bit form: both of its buffers, or none of them where that is allowed.
bool form(const gq::ActDims& A, const int8_t* codes, const float* steps, Range* c, Range* s) {
  *c = {codes, A.rows * A.pitch};
  *s = {steps, A.rows * A.groups * 4};
  if (A.rows == 0) return true;
  return codes && steps && aligned(codes, 16) && aligned(steps, 4);
}

bool vec(const float* p) { return p && aligned(p, 4); }
bool vec_or_null(const float* p) { return aligned(p, 4); }

bool space(const void* ws, int64_t have, int64_t need) {
  if (need == 0) return true;
  return ws && aligned(ws, 16) && have >= need;
}

int launch_status(int hip_rc) { return hip_rc == 0 ? GQ_OK : GQ_ELAUNCH; }

}  // namespace
