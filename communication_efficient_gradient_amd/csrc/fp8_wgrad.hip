// fp8_wgrad.hip — weight and bias gradients of a linear layer whose input is
// kept in 8-bit floating point, of one weight or of one per expert (the tile
// and its exactness: wgrad_tile.hpp):
//   dw[e, o, c] <- beta dw[e, o, c] + sum_{t of e} dy[t, o] x^[t, c]
//   db[e, o]    <- beta db[e, o]    + sum_{t of e} dy[t, o]
//
// The sum runs over tokens, whose steps differ, so the 8-bit matrix
// instructions cannot scale it: codes are decoded to 16 bits on their way into
// LDS (exact).  bf16, 16384 tokens: one weight of 4096 x 4096 430 to 460 us, 1.2
// PFLOP/s; eight of 2048 x 2048 with 2048 tokens each 155 us (167 on inputs from HBM,
// fp16 171, fp32, three products, 363), with 84 to 6400 160, 0.86 PFLOP/s: of a
// tile's 32 steps of 1.7 us and 17 us besides, its 256 KB of results and the next
// one's first copies are what nothing runs beside: a workgroup takes one tile and
// most of a CU's LDS, so the next one starts when it has left.
#include <cmath>

#include "fp8.hpp"
#include "wgrad_tile.hpp"

namespace gq {
namespace {

struct Fp8Form {
  static __device__ __forceinline__ void decode8(uint2 w, float step, float (&f)[8]) {
    fp8_decode8(w, step, f);
  }
};

struct ExpertArgs {
  int experts;
  const int64_t* offsets;
  int most;       // steps of 64 tokens that one workgroup takes
  int share;      // tiles of an XCD of each unit; 0: tiles go round the XCDs
  int high;       // of a block of tiles that an XCD takes
  int64_t parts;  // that the workspace holds: enough for ascending tables
};

// A unit is what the tiles' workgroups take of the sum: an expert's tokens, or
// a part of them where they are more than `most` steps.  Loads of experts
// differ, so units are taken by length, those over half of `most` first, then
// those over a quarter, then the rest, and no expert keeps a few workgroups
// busy when the others are done (16384 tokens over 8 experts x 2048 x 2048 in the
// table's order, whole: 326 us).
struct Unit {
  int expert, split, splits;
  int part;       // the first of the expert's parts in the workspace
};

// Each lane looks at a run of experts; the tokens' table is small and the same
// for all waves.  `u`: the unit's number, or the split expert's (JOIN).
template <bool JOIN>
__device__ __forceinline__ bool find_unit(const ExpertArgs& x, int64_t rows, int u, Unit* r) {
  const int lane = (int)threadIdx.x & 63, each = (x.experts + 63) / 64;
  const int lo = min(lane * each, x.experts), hi = min(lo + each, x.experts);
  auto splits_of = [&](int e, int* kind) {
    const Tokens t = tokens_of(x.offsets, e, rows);
    const int steps = (int)((t.hi - t.lo + 63) / 64);
    const int s = max(1, (steps + x.most - 1) / x.most);
    const int len = (steps + s - 1) / s;
    *kind = JOIN ? (s > 1 ? 0 : 1) : 2 * len > x.most ? 0 : 4 * len > x.most ? 1 : 2;
    return s;
  };
  int count[3] = {}, parts = 0;     // of this lane's experts
  for (int e = lo; e < hi; ++e) {
    int kind;
    const int s = splits_of(e, &kind);
#pragma unroll
    for (int k = 0; k < 3; ++k) count[k] += kind == k ? (JOIN ? 1 : s) : 0;
    parts += s > 1 ? s : 0;
  }
  auto up_to = [&](int v) {         // of the lanes up to this one
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int w = __shfl_up(v, d);
      if (lane >= d) v += w;
    }
    return v;
  };
  const int part0 = up_to(parts) - parts;
  int kind = -1, first = 0, base = 0;   // the unit's kind, and this lane's first of it
#pragma unroll
  for (int k = 0; k < (JOIN ? 1 : 3); ++k) {
    const int end = up_to(count[k]), total = __builtin_amdgcn_readlane(end, 63);
    if (kind < 0 && u < base + total) {
      kind = k;
      first = base + end - count[k];
    }
    base += total;
  }
  if (kind < 0) return false;
  const int mine = kind == 0 ? count[0] : kind == 1 ? count[1] : count[2];
  const uint64_t found = __ballot(u >= first && u < first + mine);
  Unit f = {0, 0, 1, part0};
  if (u >= first && u < first + mine) {
    int left = u - first;
    for (int e = lo; e < hi; ++e) {
      int k;
      const int s = splits_of(e, &k), n = JOIN ? 1 : s;
      f.expert = e;
      f.splits = s;
      f.split = left;
      if (k == kind && left < n) break;
      if (k == kind) left -= n;
      f.part += s > 1 ? s : 0;
    }
  }
  const int at = (int)__builtin_ctzll(found);
  r->expert = __builtin_amdgcn_readlane(f.expert, at);
  r->split = __builtin_amdgcn_readlane(f.split, at);
  r->splits = __builtin_amdgcn_readlane(f.splits, at);
  r->part = __builtin_amdgcn_readlane(f.part, at);
  return true;
}

// As k_act_wgrad, a tile of a unit.
template <typename T, bool COPY, int BO, int BC, int WO, int WC, int BK>
__global__ __launch_bounds__((BO / WO) * (BC / WC) * 64, 2) void k_fp8_wgrad(WgradArgs a,
                                                                            ExpertArgs x) {
  __shared__ __attribute__((aligned(16))) char lds[wgrad_lds<T, BO, BC, BK>];
  const int tiles = a.otiles * a.ctiles;
  int u, t;
  if (x.share) {
    const int q = (int)blockIdx.x / 8;
    u = q / x.share;
    t = (int)blockIdx.x % 8 * x.share + q - u * x.share;
    if (t >= tiles) return;
  } else {
    u = (int)blockIdx.x / tiles;
    t = (int)blockIdx.x - u * tiles;
  }
  Unit unit;
  if (!find_unit<false>(x, a.rows, u, &unit)) return;
  // columns of `high` tiles, so that those of an XCD are a block of them
  const int top = t / (x.high * a.ctiles) * x.high, h = min(x.high, a.otiles - top);
  const int in = t - top * a.ctiles, ot = top + in % h, ct = in / h;
  const Tokens r = tokens_of(x.offsets, unit.expert, a.rows);
  const int64_t per = ((r.hi - r.lo + 63) / 64 + unit.splits - 1) / unit.splits * 64;
  const int64_t t0 = min(r.lo + unit.split * per, r.hi), t1 = min(t0 + per, r.hi);
  const bool part = unit.splits > 1;
  const int64_t weight = (int64_t)a.out * a.cols, at = unit.part + unit.split;
  if (part && at >= x.parts) return;
  float* dw = part ? a.ws_w + at * quads(weight) : a.dw + unit.expert * weight;
  float* db = a.db;
  if (db) db = part ? a.ws_b + at * quads(a.out) : db + (int64_t)unit.expert * a.out;
  // a chunk of dy runs out of its row only where that stays before the
  // expert's end too
  a.free_rows = min(a.free_rows, r.hi);
  wgrad_tile<T, Fp8Form, COPY, COPY, BO, BC, WO, WC, BK>(a, lds, ot, ct, t0, t1, r.hi, dw, part,
                                                         db, part);
}

// Adds the parts of the experts that have some, in order; blockIdx.y counts
// those experts.
__global__ __launch_bounds__(256) void k_fp8_wgrad_join(WgradArgs a, ExpertArgs x) {
  Unit unit;
  if (!find_unit<true>(x, a.rows, (int)blockIdx.y, &unit)) return;
  if (unit.part + unit.splits > x.parts) return;
  const int64_t n = (int64_t)a.out * a.cols;
  const int64_t qw = quads(n) / 4, total = qw + (a.db ? quads(a.out) / 4 : 0);
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * 256) {
    const bool w = i < qw;
    const int64_t e = (w ? i : i - qw) * 4, len = w ? n : a.out, stride = quads(len);
    const float* q = (w ? a.ws_w : a.ws_b) + unit.part * stride + e;
    f32x4 s = *(const f32x4*)q;
    int k = 1;
    for (; k + 8 <= unit.splits; k += 8) {
      f32x4 v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = *(const f32x4*)(q + (k + j) * stride);
#pragma unroll
      for (int j = 0; j < 8; ++j) s += v[j];
    }
    for (; k < unit.splits; ++k) s += *(const f32x4*)(q + k * stride);
    float* o = (w ? a.dw : a.db) + unit.expert * len + e;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (e + j < len) o[j] = a.beta == 0.f ? s[j] : fmaf(a.beta, o[j], s[j]);
  }
}

struct Plan {
  int tile, otiles, ctiles;
  int most;                   // steps of a unit
  int64_t units, parts, split_experts;   // at most
};

// Tile and length of the units by an estimate of the time in microseconds: the
// longest of what the busiest CU and one workgroup of the largest unit take, a
// step of 64 tokens each, what a tile costs besides, and the parts' way through
// memory and back.  How the tokens are spread over several experts is not known
// here: the largest is taken to have three times its share, a CU 1.3 times.
// Parts are only written where an expert has more than a unit, else they cost
// the empty launch that would join them: units may end at a CU's share even if
// none is expected to (16384 tokens over 8 x 2048 x 2048, loads as drawn for six
// batches: 187 us with units of 86 steps, 237 with any; 2048 tokens 69 / 65 / 61
// us with 16 / 32 / any).
Plan plan_wgrad(const ActDims& A, int64_t out, int experts) {
  const int64_t rows = A.rows > 0 ? A.rows : 1;
  const int64_t some = experts < rows ? experts : rows;   // that have tokens
  const int64_t steps = UnitBounds::steps_of(rows, experts);
  auto share = [&](double times) {
    return times < (double)some ? times * (double)steps / (double)some : (double)steps;
  };
  const double big_step = A.dtype == GQ_F32 ? 5.0 : 1.9;
  const double small_step = A.dtype == GQ_F32 ? 3.4 : 1.45;
  Plan best = {};
  double least = 1e30;
  auto consider = [&](int tile, int64_t ot, int64_t ct, int64_t most, double t) {
    if (t >= least) return;
    least = t;
    best = {tile, (int)ot, (int)ct, (int)most, 0, 0, 0};
  };
  for (int tile = 128; tile <= 256; tile *= 2) {
    const int64_t ot = (out + tile - 1) / tile, ct = (A.cols + tile - 1) / tile;
    const double slots = tile == 256 ? kCus : 2 * kCus, tiles = (double)(ot * ct);
    const double load = (double)steps * tiles / slots;
    // of `units` units, the longest `unit` steps, and `parts` parts
    auto time = [&](double load, double unit, double units, double parts) {
      double step = tile == 256 ? big_step : small_step;
      if (tile == 128 && tiles * units <= kCus) step *= 0.7;  // alone on its CU
      const double t = (load > unit ? load : unit) * step +
                       std::ceil(tiles * units / slots) * (tile == 256 ? 8.0 : 5.0);
      return parts == 0. ? t : t + 8.0 + 8.0 * parts * (double)out * (double)A.cols / 6.5e6;
    };
    if (some == 1) {
      for (int64_t s = 1; s <= 32 && (s == 1 || steps / s >= 4); ++s) {
        const int64_t most = (steps + s - 1) / s;
        consider(tile, ot, ct, most,
                 time(load, (double)most, (double)s, s > 1 ? (double)s : 0.));
      }
      continue;
    }
    const double cu = 1.3 * load, large = share(3.), one = share(1.);
    auto several = [&](int64_t most) {
      const double m = (double)most;
      const double parts = one > m     ? (double)some * std::ceil(one / m)
                           : large > m ? std::ceil(large / m) : 0.;
      const double units = one > m ? parts : (double)some + parts;
      consider(tile, ot, ct, most,
               time(cu, large < m ? large : m, units, parts) + (most < steps ? 4.0 : 0.));
    };
    for (int64_t s = 1; s <= 32 && (s == 1 || steps / s >= 4); ++s)
      several((steps + s - 1) / s);
    const double m = std::ceil(cu);
    if (m > 32.)
      consider(tile, ot, ct, (int64_t)m, 4.0 + time(cu, large < m ? large : m, (double)some, 0.));
  }
  const UnitBounds u(rows, experts, best.most);
  best.split_experts = u.split;
  best.parts = u.parts;
  best.units = u.units;
  return best;
}

// BIG, SMALL: tokens of a step for 256- and 128-tiles.
template <typename T, bool COPY, int BIG, int SMALL>
void wgrad_t(const WgradArgs& a, const ExpertArgs& x, const Plan& p, hipStream_t st) {
  const int64_t g = x.share ? p.units * 8 * x.share : p.units * p.otiles * p.ctiles;
  if (p.tile == 256)
    k_fp8_wgrad<T, COPY, 256, 256, 128, 64, BIG><<<(unsigned)g, 512, 0, st>>>(a, x);
  else k_fp8_wgrad<T, COPY, 128, 128, 64, 32, SMALL><<<(unsigned)g, 512, 0, st>>>(a, x);
}

}  // namespace

int64_t fp8_wgrad_workspace(const ActDims& A, int64_t out, int experts) {
  const Plan p = plan_wgrad(A, out, experts);
  return 4 * p.parts * (quads(out * A.cols) + quads(out));
}

int launch_fp8_wgrad(const ActDims& A, int64_t out, int experts, const int64_t* offsets,
                     const void* dy, int64_t lddy, const uint8_t* codes, const float* steps,
                     float beta, float* dw, float* db, void* ws, hipStream_t st) {
  const Plan p = plan_wgrad(A, out, experts);
  float* w = (float*)ws;
  WgradArgs a = {A.rows,   (int)out, (int)A.cols, (int)A.pitch, A.groups, 7,
                 dy,       lddy,     rows_with_room(A.rows, lddy, 7),
                 (const int8_t*)codes, steps, beta, dw, db,
                 w,        w + p.parts * quads(out * A.cols),
                 1,        p.otiles, p.ctiles,    1,            0};
  // What an XCD reads through its L2 is the dy of its tiles' rows and the codes
  // of their columns: a block twice as wide as high has as many bytes of both
  // in 16 bits (16384 tokens over 8 x 2048 x 2048, an XCD's 8 tiles of a unit 8 x 1 /
  // 2 x 4: 582 / 279 MB fetched, 164 / 159 us; 8192 over 1024 x 1024 42 / 39 us).
  const int tiles = p.otiles * p.ctiles, share = tiles >= 32 ? div_up(tiles, 8) : 0;
  int high = 1;
  while (high < 8 && 8 * high * high <= share) high *= 2;
  const ExpertArgs x = {experts, offsets, p.most, share, high, p.parts};
  // copies move 16 bytes of a row at 16-byte addresses, to the row's last one
  const bool copy = A.dtype != GQ_F32 && ((uintptr_t)dy & 15) == 0 && lddy % 8 == 0 &&
                    lddy < (1 << 23) && out % 8 == 0;
  // the bias's columns over the tiles of a row, 32 to a tile at least
  if (copy)
    while (a.turns * 2 <= p.ctiles && a.turns * 2 <= p.tile / 32) a.turns *= 2;
  if (A.dtype == GQ_F32) wgrad_t<float, false, 32, 32>(a, x, p, st);
  else if (A.dtype == GQ_F16 && copy) wgrad_t<_Float16, true, 64, 64>(a, x, p, st);
  else if (A.dtype == GQ_F16) wgrad_t<_Float16, false, 32, 64>(a, x, p, st);
  else if (copy) wgrad_t<__bf16, true, 64, 64>(a, x, p, st);
  else wgrad_t<__bf16, false, 32, 64>(a, x, p, st);
  int rc = (int)hipGetLastError();
  if (rc == 0 && p.parts > 0) {
    const int64_t b = (quads(out * A.cols) / 4 + quads(out) / 4 + 255) / 256;
    const dim3 g((unsigned)(b < 4096 ? b : 4096), (unsigned)p.split_experts);
    k_fp8_wgrad_join<<<g, 256, 0, st>>>(a, x);
    rc = (int)hipGetLastError();
  }
  return rc;
}

}  // namespace gq
