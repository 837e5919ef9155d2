// fp8_wgrad.hip — weight and bias gradients of a linear layer whose input is
// kept in 8-bit floating point, of one weight or of one per expert (the tile
// and its exactness: wgrad_tile.hpp):
//   dw[e, o, c] <- beta dw[e, o, c] + sum_{t of e} dy[t, o] x^[t, c]
//   db[e, o]    <- beta db[e, o]    + sum_{t of e} dy[t, o]
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
};

// As k_act_wgrad; the tokens of each expert are split by themselves.
template <typename T, bool COPY, int BO, int BC, int WO, int WC, int BK>
__global__ __launch_bounds__((BO / WO) * (BC / WC) * 64, 2) void k_fp8_wgrad(WgradArgs a,
                                                                            ExpertArgs x) {
  __shared__ __attribute__((aligned(16))) char lds[wgrad_lds<T, BO, BC, BK>];
  Tile tile;
  if (!TileWalk(a.otiles, a.ctiles, a.splits * x.experts).take(&tile)) return;
  const int e = tile.split / a.splits, split = tile.split - e * a.splits;
  const Tokens r = tokens_of(x.offsets, e, a.rows);
  const int64_t per = (r.hi - r.lo + (int64_t)64 * a.splits - 1) / ((int64_t)64 * a.splits) * 64;
  const int64_t t0 = min(r.lo + split * per, r.hi), t1 = min(t0 + per, r.hi);
  const bool w_part = a.splits > 1, b_part = a.splits * a.turns > 1;
  const int64_t weight = (int64_t)a.out * a.cols;
  float* dw = (w_part ? a.ws_w + split * quads(weight * x.experts) : a.dw) + e * weight;
  float* db = a.db;
  if (db) {
    if (b_part)
      db = a.ws_b + ((int64_t)split * a.turns + tile.j) * quads((int64_t)a.out * x.experts);
    db += (int64_t)e * a.out;
  }
  // a chunk of dy runs out of its row only where that stays before the
  // expert's end too
  a.free_rows = min(a.free_rows, r.hi);
  wgrad_tile<T, Fp8Form, COPY, BO, BC, WO, WC, BK>(a, lds, tile.i, tile.j, t0, t1, r.hi, dw,
                                                   w_part, db, b_part);
}

struct Plan {
  int tile, splits, otiles, ctiles, turns;
};

Plan plan_wgrad(const ActDims& A, int64_t out, int experts) {
  // as if the tokens were spread evenly over the experts
  const int64_t each = (A.rows + experts - 1) / experts;
  const int64_t steps = each > 0 ? (each + 63) / 64 : 1;
  const double big_step = A.dtype == GQ_F32 ? 5.0 : 1.9;
  const double small_step = A.dtype == GQ_F32 ? 3.4 : 1.45;
  Plan best = {};
  double least = 1e30;
  for (int tile = 128; tile <= 256; tile *= 2) {
    const int64_t ot = (out + tile - 1) / tile, ct = (A.cols + tile - 1) / tile;
    for (int64_t s = 1; s <= 32 && (s == 1 || s * 2 <= steps); ++s) {
      const int64_t per = (steps + s - 1) / s;
      const int64_t groups = ot * ct * s * experts, slots = tile == 256 ? kCus : 2 * kCus;
      double step = tile == 256 ? big_step : small_step;
      if (tile == 128 && groups <= kCus) step *= 0.7;  // alone on its CU
      double t = (double)((groups + slots - 1) / slots) *
                 ((double)per * step + (tile == 256 ? 8.0 : 5.0));
      if (s > 1) t += 4.0 + 8.0 * (double)(s * out * experts) * (double)A.cols / 6.5e6;
      if (t < least) {
        least = t;
        best = {tile, (int)s, (int)ot, (int)ct, (int)ct};
      }
    }
  }
  if (best.splits == 1 && steps <= 32) best.turns = 1;
  return best;
}

// BIG, SMALL: tokens of a step for 256- and 128-tiles.
template <typename T, bool COPY, int BIG, int SMALL>
void wgrad_t(const WgradArgs& a, const ExpertArgs& x, int tile, hipStream_t st) {
  const unsigned g = (unsigned)(a.otiles * a.ctiles * a.splits * x.experts);
  if (tile == 256) k_fp8_wgrad<T, COPY, 256, 256, 128, 64, BIG><<<g, 512, 0, st>>>(a, x);
  else k_fp8_wgrad<T, COPY, 128, 128, 64, 32, SMALL><<<g, 512, 0, st>>>(a, x);
}

}  // namespace

int64_t fp8_wgrad_workspace(const ActDims& A, int64_t out, int experts) {
  const Plan p = plan_wgrad(A, out, experts);
  const int64_t w = p.splits > 1 ? p.splits * quads(out * A.cols * experts) : 0;
  const int64_t b =
      p.splits * p.turns > 1 ? (int64_t)p.splits * p.turns * quads(out * experts) : 0;
  return 4 * (w + b);
}

int launch_fp8_wgrad(const ActDims& A, int64_t out, int experts, const int64_t* offsets,
                     const void* dy, int64_t lddy, const uint8_t* codes, const float* steps,
                     float beta, float* dw, float* db, void* ws, hipStream_t st) {
  const Plan p = plan_wgrad(A, out, experts);
  float* w = (float*)ws;
  const int64_t wn = p.splits > 1 ? p.splits * quads(out * A.cols * experts) : 0;
  WgradArgs a = {A.rows, (int)out, (int)A.cols, (int)A.pitch, A.groups, 7,
                 dy,     lddy,     rows_with_room(A.rows, lddy, 7),
                 (const int8_t*)codes, steps, beta, dw, db,
                 w,      w + wn,   p.splits, p.otiles, p.ctiles, p.turns, 0,
                 out * A.cols * experts, out * experts};
  const ExpertArgs x = {experts, offsets};
  // copies move 16 bytes of a row at 16-byte addresses, to the row's last one
  const bool copy = A.dtype != GQ_F32 && ((uintptr_t)dy & 15) == 0 && lddy % 8 == 0 &&
                    lddy < (1 << 23) && out % 8 == 0;
  if (A.dtype == GQ_F32) wgrad_t<float, false, 32, 32>(a, x, p.tile, st);
  else if (A.dtype == GQ_F16 && copy) wgrad_t<_Float16, true, 64, 64>(a, x, p.tile, st);
  else if (A.dtype == GQ_F16) wgrad_t<_Float16, false, 32, 64>(a, x, p.tile, st);
  else if (copy) wgrad_t<__bf16, true, 64, 64>(a, x, p.tile, st);
  else wgrad_t<__bf16, false, 32, 64>(a, x, p.tile, st);
  int rc = (int)hipGetLastError();
  if (rc == 0 && (p.splits > 1 || (db && p.splits * p.turns > 1))) {
    const int64_t n = (p.splits > 1 ? quads(out * A.cols * experts) : 0) + quads(out * experts);
    const int64_t b = (n / 4 + 255) / 256;
    k_act_wgrad_join<<<(unsigned)(b < 4096 ? b : 4096), 256, 0, st>>>(a);
    rc = (int)hipGetLastError();
  }
  return rc;
}

}  // namespace gq
