// act_wgrad.hip — weight and bias gradient of a linear layer whose input is
// kept in 8-bit integers (the tile and its exactness: wgrad_tile.hpp).
#include "wgrad_tile.hpp"

namespace gq {
namespace {

struct Int8Form {
  static __device__ __forceinline__ void decode8(uint2 w, float step, float (&f)[8]) {
    gq::decode8(w, step, f);
  }
};

template <typename T, bool COPY, int BO, int BC, int WO, int WC, int BK>
__global__ __launch_bounds__((BO / WO) * (BC / WC) * 64, 2) void k_act_wgrad(WgradArgs a) {
  __shared__ __attribute__((aligned(16))) char lds[wgrad_lds<T, BO, BC, BK>];
  Tile tile;
  if (!TileWalk(a.otiles, a.ctiles, a.splits).take(&tile)) return;
  const int64_t t0 = (int64_t)tile.split * a.per;
  const int64_t t1 = min(t0 + a.per, a.rows);
  const bool w_part = a.splits > 1, b_part = a.splits * a.turns > 1;
  float* dw = w_part ? a.ws_w + tile.split * quads((int64_t)a.out * a.cols) : a.dw;
  float* db = a.db;
  if (db && b_part) db = a.ws_b + ((int64_t)tile.split * a.turns + tile.j) * quads(a.out);
  wgrad_tile<T, Int8Form, COPY, false, BO, BC, WO, WC, BK>(a, lds, tile.i, tile.j, t0, t1,
                                                           a.rows, dw, w_part, db, b_part);
}

// Adds the parts of dw (splits of them) and db (splits * turns), in order:
// four neighbouring results per thread, the loads of eight parts at a time
// (whole quads: parts are padded to them and a quad never straddles dw's end).
__global__ __launch_bounds__(256) void k_act_wgrad_join(WgradArgs a) {
  const int64_t n = a.splits > 1 ? (int64_t)a.out * a.cols : 0;
  const int64_t qw = (n + 3) / 4, total = qw + (a.db ? (a.out + 3) / 4 : 0);
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * 256) {
    const bool w = i < qw;
    const int64_t e = (w ? i : i - qw) * 4, len = w ? n : a.out;
    const float* q = (w ? a.ws_w : a.ws_b) + e;
    const int64_t stride = quads(len);
    const int parts = w ? a.splits : a.splits * a.turns;
    f32x4 s = *(const f32x4*)q;
    int k = 1;
    for (; k + 8 <= parts; k += 8) {
      f32x4 v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = *(const f32x4*)(q + (k + u) * stride);
#pragma unroll
      for (int u = 0; u < 8; ++u) s += v[u];
    }
    for (; k < parts; ++k) s += *(const f32x4*)(q + k * stride);
    float* o = (w ? a.dw : a.db) + e;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (e + j < len) o[j] = a.beta == 0.f ? s[j] : fmaf(a.beta, o[j], s[j]);
  }
}

struct Plan {
  int tile, splits, otiles, ctiles, turns;
  int64_t per;
};

// The tile's side and the number of splits by an estimate of the time in
// microseconds: rounds of workgroups (one 256 x 256 tile or two 128 x 128
// tiles per CU), a step of 64 tokens each, what a tile costs besides, and the
// parts' way through memory and back.  Measured (bf16, whole call): 16384 x
// 2048 x 2048 tokens x out x cols 140 us with 256-tiles and 4 splits, 170 with
// 128-tiles and 2; 8192 x 1024 x 1024 41.4 us with 256 and 13, 38.1 with 128 and
// 8; 512 x 1024 x 4096 22.6 and 12.6 us unsplit; 8192 x 256 x 256 25.3 and 17.5 us
// with 32 splits.
Plan plan_wgrad(const ActDims& A, int64_t out) {
  const int64_t steps = (A.rows + 63) / 64;
  const double big_step = A.dtype == GQ_F32 ? 5.0 : 1.9;
  const double small_step = A.dtype == GQ_F32 ? 3.4 : 1.45;
  Plan best = {};
  double least = 1e30;
  for (int tile = 128; tile <= 256; tile *= 2) {
    const int64_t ot = (out + tile - 1) / tile, ct = (A.cols + tile - 1) / tile;
    for (int64_t s = 1; s <= 32 && (s == 1 || s * 2 <= steps); ++s) {
      const int64_t per = s == 1 ? (steps > 0 ? steps : 1) : (steps + s - 1) / s;
      const int64_t groups = ot * ct * s, slots = tile == 256 ? kCus : 2 * kCus;
      double step = tile == 256 ? big_step : small_step;
      if (tile == 128 && groups <= kCus) step *= 0.7;  // alone on its CU
      double t = (double)((groups + slots - 1) / slots) *
                 ((double)per * step + (tile == 256 ? 8.0 : 5.0));
      if (s > 1) t += 4.0 + 8.0 * (double)(s * out) * (double)A.cols / 6.5e6;
      if (t < least) {
        least = t;
        best = {tile, (int)(((steps > 0 ? steps : 1) + per - 1) / per), (int)ot, (int)ct,
                (int)ct, per * 64};
      }
    }
  }
  // Shared out, the bias's sums need a second launch to join them (4 to 5 us);
  // of up to 32 steps one tile takes all.  bf16: 1024 x 2048 x 2048 18.2 us so,
  // 21.9 shared out, 2048 x 4096 x 2048 45.0 and 49.9, 4096 x 4096 x 4096 127 and
  // 128, 16384 x 4096 x 4096 475 and 457.
  if (best.splits == 1 && steps <= 32) best.turns = 1;
  return best;
}

// BIG, SMALL: tokens of a step for 256- and 128-tiles.
template <typename T, bool COPY, int BIG, int SMALL>
void wgrad_t(const WgradArgs& a, int tile, hipStream_t st) {
  const unsigned g = (unsigned)(a.otiles * a.ctiles * a.splits);
  if (tile == 256) k_act_wgrad<T, COPY, 256, 256, 128, 64, BIG><<<g, 512, 0, st>>>(a);
  else k_act_wgrad<T, COPY, 128, 128, 64, 32, SMALL><<<g, 512, 0, st>>>(a);
}

}  // namespace

int64_t act_wgrad_workspace(const ActDims& A, int64_t out) {
  const Plan p = plan_wgrad(A, out);
  const int64_t w = p.splits > 1 ? p.splits * quads(out * A.cols) : 0;
  const int64_t b = p.splits * p.turns > 1 ? (int64_t)p.splits * p.turns * quads(out) : 0;
  return 4 * (w + b);
}

int launch_act_wgrad(const ActDims& A, int64_t out, const void* dy, int64_t lddy,
                     const int8_t* codes, const float* steps, float beta,
                     float* dw, float* db, void* ws, hipStream_t st) {
  const Plan p = plan_wgrad(A, out);
  int glog = 31;
  if (!A.whole_row)
    for (glog = 0; (1 << glog) < A.group;) ++glog;
  float* w = (float*)ws;
  const int64_t wn = p.splits > 1 ? p.splits * quads(out * A.cols) : 0;
  const WgradArgs a = {A.rows, (int)out, (int)A.cols, (int)A.pitch, A.groups, glog,
                       dy,     lddy,     rows_with_room(A.rows, lddy, 7),
                       codes,  steps,    beta,        dw,           db,
                       w,      w + wn,   p.splits,    p.otiles,     p.ctiles,
                       p.turns, p.per};
  // copies move 16 bytes of a row at 16-byte addresses, to the row's last one
  const bool copy = A.dtype != GQ_F32 && ((uintptr_t)dy & 15) == 0 && lddy % 8 == 0 &&
                    lddy < (1 << 23) &&
                    out % 8 == 0;
  // Through registers 64-token steps of 256-tiles spill (16384 x 4095 x 4096
  // bf16: 973 us, 547 with 32); fp32's three terms fill LDS with 32.
  if (A.dtype == GQ_F32) wgrad_t<float, false, 32, 32>(a, p.tile, st);
  else if (A.dtype == GQ_F16 && copy) wgrad_t<_Float16, true, 64, 64>(a, p.tile, st);
  else if (A.dtype == GQ_F16) wgrad_t<_Float16, false, 32, 64>(a, p.tile, st);
  else if (copy) wgrad_t<__bf16, true, 64, 64>(a, p.tile, st);
  else wgrad_t<__bf16, false, 32, 64>(a, p.tile, st);
  int rc = (int)hipGetLastError();
  if (rc == 0 && (p.splits > 1 || (db && p.splits * p.turns > 1))) {
    const int64_t n = (p.splits > 1 ? quads(out * A.cols) : 0) + quads(out);
    const int64_t b = (n / 4 + 255) / 256;
    k_act_wgrad_join<<<(unsigned)(b < 4096 ? b : 4096), 256, 0, st>>>(a);
    rc = (int)hipGetLastError();
  }
  return rc;
}

}  // namespace gq
