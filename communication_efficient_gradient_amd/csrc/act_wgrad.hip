// act_wgrad.hip — weight and bias gradient of a linear layer whose input is
// kept in 8 bits:
//   dw[o, c] <- beta dw[o, c] + sum_t dy[t, o] x^[t, c]
//   db[o]    <- beta db[o]    + sum_t dy[t, o]
//
// The sum runs over tokens, the slow axis of both operands, so tiles [t][col]
// go to LDS as they lie in memory and come out through the transposing LDS
// read (each lane gets consecutive tokens of one column, the operand layout
// of the matrix instructions).  Every product is exact, only the fp32
// accumulation rounds:
//   bf16  x^ = code * step is exact in bf16, dy is used as it is
//   fp16  x^ is exact in fp16: steps are at most 2^9, and one below 2^-24 comes
//         with values that are multiples of 2^-24 and kept as they are
//   fp32  dy is split into three bf16 terms (24 significant bits) whose sum is
//         the value itself, one matrix product each with x^ in bf16; below
//         2^-110 the third term is cut at bf16's last place, 2^-133
#include <type_traits>

#include "act.hpp"
#include "act_bounds.hpp"

namespace gq {
namespace {

#define GQ_LDS __attribute__((address_space(3)))
typedef GQ_LDS char* LdsPtr;

template <typename T>
constexpr int kPlanes = 1;
template <>
inline constexpr int kPlanes<float> = 3;

struct WgradArgs {
  int64_t rows;
  int out, cols, pitch, groups, glog;
  const void* dy;
  int64_t lddy;
  int64_t free_rows;   // rows of dy that a chunk may run out of
  const int8_t* codes;
  const float* steps;
  float beta;
  float *dw, *db;      // results
  float *ws_w, *ws_b;  // parts: [split][out * cols], [split][turns][out], in quads
  int splits, otiles, ctiles;
  int turns;           // tiles of a row that share the bias's sums
  int64_t per;         // tokens of a split, a multiple of 64
};

// Length of a part in the workspace: whole quads of floats.
__host__ __device__ inline int64_t quads(int64_t n) { return (n + 3) / 4 * 4; }

// Byte offset of 32-byte chunk `ch` (16 columns) of token row t in a tile of W
// columns.  One transposing read takes two neighbouring chunks of rows 0..3
// and 8..11 (or 4..7 and 12..15); the exclusive or spreads those over all
// banks.
template <int W>
__device__ __forceinline__ int place(int t, int ch) {
  return t * (W * 2) + ((ch ^ ((t & 3) << 1 | (t >> 3 & 1))) << 5);
}

// Where a lane's part of a 32-column, 16-token operand lies: column lane % 32,
// tokens 8 (lane / 32) + 0..3 of a tile that starts at chunk `ch` (even); the
// next four tokens lie 4 rows further at the same place of their row.
template <int W>
__device__ __forceinline__ int operand_place(int ch, int lane) {
  const int t = lane / 32 * 8 + lane % 16 / 4;
  return place<W>(t, ch + lane / 16 % 2) + lane % 4 * 8;
}

template <int W>
__device__ __forceinline__ s16x8 operand(LdsPtr p) {
  const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((GQ_LDS s16x4*)p);
  const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((GQ_LDS s16x4*)(p + 4 * W * 2));
  return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

template <typename T>
__device__ __forceinline__ f32x16 product(s16x8 a, s16x8 b, f32x16 c) {
  if constexpr (std::is_same_v<T, _Float16>) {
    typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  } else {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  }
}

// Eight values x^ in the products' type (exact in it, see above).
template <typename T>
__device__ __forceinline__ u32x4 packed(const float (&f)[8]) {
  if constexpr (std::is_same_v<T, _Float16>) {
    u32x4 r;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      r[j] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(f[2 * j], f[2 * j + 1]));
    return r;
  } else {
    return __builtin_bit_cast(u32x4, narrow<__bf16>(f));
  }
}

// A tile of BO output features by BC columns per workgroup, WO by WC of it per
// wave, in steps of BK tokens.  While a step's products run, dy of the next
// step is copied to LDS (COPY: straight from memory, which needs 16-byte
// rows; otherwise through registers, split into the type's bf16 terms) and
// its codes, loaded one step earlier, are decoded into LDS.  A step of 256 x
// 256 moves 260 KB through LDS and keeps the matrix cores busy for 2048 cycles:
// the two share the time.  16384 x 4096 x 4096 (tokens x out x cols): 455 us in
// a loop in bf16 and 468 in fp16, 1.2 PFLOP/s, median 525 (504 to 625) under the
// profiler, matrix cores 60 % busy; fp32 326 us for 4096 x 4096 x 4096.
template <typename T, bool COPY, int BO, int BC, int WO, int WC, int BK>
__global__ __launch_bounds__((BO / WO) * (BC / WC) * 64, 2) void k_act_wgrad(WgradArgs a) {
  constexpr int P = kPlanes<T>;
  static_assert(!COPY || P == 1, "");
  constexpr int WAVES = (BO / WO) * (BC / WC), TH = WAVES * 64;
  constexpr int OT = WO / 32, CT = WC / 32, KK = BK / 16;
  constexpr int ABUF = P * BK * BO * 2, BBUF = BK * BC * 2, BUF = ABUF + BBUF;
  __shared__ __attribute__((aligned(16))) char lds[2 * BUF];
  const int tid = (int)threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wo = wave % (BO / WO) * WO, wc = wave / (BO / WO) * WC;
  Tile tile;
  if (!TileWalk(a.otiles, a.ctiles, a.splits).take(&tile)) return;
  const int ot = tile.i, ct = tile.j;
  const int o0 = ot * BO, c0 = ct * BC;
  const int64_t t0 = (int64_t)tile.split * a.per;
  const int64_t t1 = min(t0 + a.per, a.rows);
  const int steps = (int)((t1 - t0 + BK - 1) / BK);

  // ---- dy.  Rows past the last lie behind the range and read as zeros;
  // columns past the last hold anything, and what they give is not stored.
  const char* dy = (const char*)((const T*)a.dy + o0);
  const int64_t row_bytes = a.lddy * (int64_t)sizeof(T);
  const int64_t dy_end = ((a.rows - 1) * a.lddy + a.out - o0) * (int64_t)sizeof(T);
  // copies: a wave instruction fills two rows of 256 columns, or four of 128
  constexpr int AI = BK * BO * 2 / 1024 / WAVES, LPR = BO / 8;  // lanes per row
  int oa[AI];  // a lane's place in the tile, without the step's first row
#pragma unroll
  for (int i = 0; i < AI; ++i) {
    const int t = (wave * AI + i) * (64 / LPR) + lane / LPR, p = lane % LPR;
    // the 16 bytes that belong at place p of row t
    const int ch = (p / 2) ^ ((t & 3) << 1 | (t >> 3 & 1));
    oa[i] = t * (int)row_bytes + ch * 32 + p % 2 * 16;
  }
  const char* dy_at = dy + t0 * row_bytes;  // of the step that is copied next
  int64_t dy_left = dy_end - t0 * row_bytes;
  auto copy_dy = [&](LdsPtr to) {
    const BufferRange r = range_of(dy_at, dy_left);
#pragma unroll
    for (int i = 0; i < AI; ++i)
      copy16_to_lds(r, oa[i], 0, to + (wave * AI + i) * 1024);
    dy_at += BK * row_bytes;
    dy_left -= BK * row_bytes;
  };
  // through registers: pieces of eight columns, BO / 8 per row
  constexpr int AP = COPY ? 1 : BK * BO / 8 / TH;
  Raw8<T> ra[AP];
  // A short last chunk may run on into the rows that follow (up to seven values
  // behind the row's last one: seven rows where a row is one value), and
  // columns past the last hold anything; only the steps that reach a row
  // without that much behind it take care to stay inside theirs.
  const int odd = min(tid % LPR * 8, a.out - 1 - o0);
  auto load_dy = [&](int st) {
    const int64_t first = t0 + (int64_t)st * BK + tid / LPR;
    const T* r = (const T*)dy + first * a.lddy;
    if (t0 + (int64_t)(st + 1) * BK <= a.free_rows) {
#pragma unroll
      for (int i = 0; i < AP; ++i)
        __builtin_memcpy(&ra[i], r + i * (TH / LPR) * a.lddy + odd, sizeof(ra[i]));
    } else {
#pragma unroll
      for (int i = 0; i < AP; ++i) {
        const bool live = first + i * (TH / LPR) < t1;
        ra[i] = load8(r + i * (TH / LPR) * a.lddy + tid % LPR * 8,
                      live ? a.out - o0 - tid % LPR * 8 : 0);
      }
    }
  };
  float bsum[8] = {};
  auto write_dy = [&](LdsPtr to, bool sum, int i) {
    const int q = i * TH + tid, t = q / LPR, p = q % LPR;
    float v[8];
    if (P > 1 || sum) widen(ra[i], v);
    if (sum) {
#pragma unroll
      for (int j = 0; j < 8; ++j) bsum[j] += v[j];
    }
    if constexpr (P == 1)
      *(GQ_LDS u32x4*)(to + place<BO>(t, p / 2) + p % 2 * 16) =
          __builtin_bit_cast(u32x4, ra[i]);
#pragma unroll
    for (int k = 0; k < (P > 1 ? P : 0); ++k) {
      u32x4 h;
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        // the first eight significant bits, exactly; the rest stays in v
        const uint32_t x = __float_as_uint(v[j]), y = __float_as_uint(v[j + 1]);
        h[j / 2] = __builtin_amdgcn_perm(y, x, 0x07060302u);
        if (k + 1 < P) {
          v[j] -= __uint_as_float(x & 0xffff0000u);
          v[j + 1] -= __uint_as_float(y & 0xffff0000u);
        }
      }
      *(GQ_LDS u32x4*)(to + k * (BK * BO * 2) + place<BO>(t, p / 2) + p % 2 * 16) = h;
    }
  };

  // ---- codes: pieces of eight columns, BC / 8 per row
  constexpr int BP = BK * BC / 8 / TH, PPR = BC / 8;
  uint2 rc[BP];
  float rs[BP];
  const int pc = c0 + tid % PPR * 8;  // TH is a multiple of PPR
  const int grp = min(pc >> a.glog, a.groups - 1);
  // past the last row everything reads as zero
  const int tc = tid / PPR;  // token of piece 0; TH / PPR tokens between pieces
  const int ocode = tc * a.pitch + pc, ostep = (tc * a.groups + grp) * 4;
  const int8_t* c_at = a.codes + t0 * a.pitch;  // of the step loaded next
  const float* s_at = a.steps + t0 * a.groups;
  int64_t rows_left = a.rows - t0;
  BufferRange rng_c, rng_s;
  auto next_codes = [&] {
    rng_c = range_of(c_at, rows_left * a.pitch);
    rng_s = range_of(s_at, rows_left * a.groups * 4);
    c_at += (int64_t)BK * a.pitch;
    s_at += (int64_t)BK * a.groups;
    rows_left -= BK;
  };
  auto load_codes = [&](int i) {
    const auto w = __builtin_amdgcn_raw_buffer_load_b64(rng_c, ocode,
                                                        i * (TH / PPR) * a.pitch, 0);
    rc[i] = make_uint2(w[0], w[1]);
    rs[i] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(
        rng_s, ostep, i * (TH / PPR) * a.groups * 4, 0));
  };
  auto write_codes = [&](LdsPtr to, int i) {
    const int t = (i * TH + tid) / PPR, p = tid % PPR;
    float f[8];
    decode8(rc[i], rs[i], f);
    *(GQ_LDS u32x4*)(to + place<BC>(t, p / 2) + p % 2 * 16) =
        packed<T>(f);
  };

  // The bias's sums are shared out over the tiles of a row: tile ct < turns
  // takes the steps st with st % turns == ct.
  const bool bias = a.db != nullptr && ct < a.turns;
  auto sum_dy = [&](LdsPtr from) {
    constexpr int N = BK * BO / 8 / TH;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int q = i * TH + tid, t = q / LPR, p = q % LPR;
      const u32x4 u = *(GQ_LDS u32x4*)(from + place<BO>(t, p / 2) + p % 2 * 16);
      float v[8];
      widen(__builtin_bit_cast(Raw8<std::conditional_t<sizeof(T) == 2, T, __bf16>>, u), v);
#pragma unroll
      for (int j = 0; j < 8; ++j) bsum[j] += v[j];
    }
  };

  f32x16 acc[OT][CT];
#pragma unroll
  for (int i = 0; i < OT; ++i)
#pragma unroll
    for (int j = 0; j < CT; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

  int pa[OT], pb[CT];
#pragma unroll
  for (int i = 0; i < OT; ++i) pa[i] = operand_place<BO>((wo + i * 32) / 16, lane);
#pragma unroll
  for (int j = 0; j < CT; ++j) pb[j] = operand_place<BC>((wc + j * 32) / 16, lane);
  s16x8 fa[2][OT], fb[2][CT];
  // operands of sub-step k (a 16-token block and a plane of dy)
  auto read_a = [&](int to, LdsPtr from, int k) {
    const LdsPtr q = from + k % P * (BK * BO * 2) + k / P * (16 * BO * 2);
#pragma unroll
    for (int i = 0; i < OT; ++i) fa[to][i] = operand<BO>(q + pa[i]);
  };
  auto read_b = [&](int to, LdsPtr from, int kk) {
    const LdsPtr q = from + kk * (16 * BC * 2);
#pragma unroll
    for (int j = 0; j < CT; ++j) fb[to][j] = operand<BC>(q + pb[j]);
  };

  int turn = 0;  // st % turns
  // Step st from (now_a, now_b), with step st + 1 prepared in (next_a, next_b)
  // and the codes of step st + 2 loaded.  All four are restrict: reads and
  // writes here do not wait for the copies on their way to next_a.  The barrier
  // does: the compiler counts the copies as writes to LDS and waits before it
  // for all but the loads of codes, which are younger (a test follows this in
  // the assembly).  Past the last step zeros are prepared.
  auto step = [&](int st, LdsPtr __restrict__ now_a, LdsPtr __restrict__ now_b,
                  LdsPtr __restrict__ next_a, LdsPtr __restrict__ next_b) {
    turn = turn + 1 == a.turns ? 0 : turn + 1;
    const bool sum = bias && turn == ct && st + 1 < steps;
    if constexpr (COPY) copy_dy(next_a);
    next_codes();
#pragma unroll
    for (int k = 0; k < KK * P; ++k) {
      const int kk = k / P, p = k % P;
      if (k + 1 < KK * P) {
        if (p == P - 1) read_b((kk + 1) & 1, now_b, kk + 1);
        read_a((k + 1) & 1, now_a, k + 1);
      } else {
        __syncthreads();  // the next step is in LDS, this one is read
        if (COPY && sum) sum_dy(next_a);
        read_b(0, next_b, 0);
        read_a(0, next_a, 0);
      }
      // the pieces are decoded in the first two sub-steps, which leaves the
      // loads that follow them the rest of the step
      if (k < 2) {
        if constexpr (!COPY) {
#pragma unroll
          for (int i = k * AP / 2; i < (k + 1) * AP / 2; ++i) {
            write_dy(next_a, sum, i);
          }
        }
#pragma unroll
        for (int i = k * BP / 2; i < (k + 1) * BP / 2; ++i) {
          write_codes(next_b, i);
          load_codes(i);
        }
      }
      if (!COPY && k == (KK * P > 2 ? 2 : 1)) load_dy(st + 2);
#pragma unroll
      for (int i = 0; i < OT; ++i)
#pragma unroll
        for (int j = 0; j < CT; ++j)
          acc[i][j] = product<T>(fa[k & 1][i], fb[kk & 1][j], acc[i][j]);
      // reads and decoding between products
#pragma unroll
      for (int g = 0; g < OT * CT; ++g) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
        if (COPY && k < 2) __builtin_amdgcn_sched_group_barrier(0x002, 8, 0);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  const LdsPtr a0 = (LdsPtr)lds, b0 = a0 + ABUF, a1 = a0 + BUF, b1 = a1 + ABUF;
  if (steps > 0) {
    if constexpr (COPY) copy_dy(a0);
    next_codes();
#pragma unroll
    for (int i = 0; i < BP; ++i) load_codes(i);
    next_codes();
    if constexpr (!COPY) {
      load_dy(0);
#pragma unroll
      for (int i = 0; i < AP; ++i) write_dy(a0, bias && ct == 0, i);
      load_dy(1);
    }
#pragma unroll
    for (int i = 0; i < BP; ++i) {
      write_codes(b0, i);
      load_codes(i);
    }
    __syncthreads();
    if (COPY && bias && ct == 0) sum_dy(a0);
    read_a(0, a0, 0);
    read_b(0, b0, 0);
  }
  int st = 0;
  for (; st + 1 < steps; st += 2) {
    step(st, a0, b0, a1, b1);
    step(st + 1, a1, b1, a0, b0);
  }
  if (st < steps) step(st, a0, b0, a1, b1);
  // a lane holds one column of sixteen output features per 32 x 32 tile, so a
  // store instruction writes two whole 128-byte lines
  const bool parts = a.splits > 1;
  float* dw = parts ? a.ws_w + tile.split * quads((int64_t)a.out * a.cols) : a.dw;
  const float beta = parts ? 0.f : a.beta;
#pragma unroll
  for (int j = 0; j < CT; ++j) {
    const int c = c0 + wc + j * 32 + lane % 32;
    if (c >= a.cols) continue;
#pragma unroll
    for (int i = 0; i < OT; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int o = o0 + wo + i * 32 + r / 4 * 8 + lane / 32 * 4 + r % 4;
        if (o >= a.out) continue;
        float* q = dw + (int64_t)o * a.cols + c;
        *q = beta == 0.f ? acc[i][j][r] : fmaf(beta, *q, acc[i][j][r]);
      }
  }
  if (bias) {
    // threads of one piece of columns hold sums of different rows
    __syncthreads();
    float* sh = reinterpret_cast<float*>(lds);  // [TH / LPR][BO]
#pragma unroll
    for (int j = 0; j < 8; ++j) sh[tid / LPR * BO + tid % LPR * 8 + j] = bsum[j];
    __syncthreads();
    const bool one = a.splits == 1 && a.turns == 1;
    for (int o = tid; o < BO && o0 + o < a.out; o += TH) {
      float s = 0.f;
#pragma unroll
      for (int t = 0; t < TH / LPR; ++t) s += sh[t * BO + o];
      if (one) {
        float* q = a.db + o0 + o;
        *q = a.beta == 0.f ? s : fmaf(a.beta, *q, s);
      } else {
        a.ws_b[((int64_t)tile.split * a.turns + ct) * quads(a.out) + o0 + o] = s;
      }
    }
  }
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
