// wgrad_tile.hpp — a tile of the weight gradient of a linear layer whose input is
// kept in an 8-bit form:
//   dw[o, c] <- beta dw[o, c] + sum_t dy[t, o] x^[t, c]
//   db[o]    <- beta db[o]    + sum_t dy[t, o]
//
// The sum runs over tokens, the slow axis of both operands, so tiles [t][col]
// go to LDS as they lie in memory and come out through the transposing LDS
// read (each lane gets consecutive tokens of one column, the operand layout
// of the matrix instructions).  Every product is exact, only the fp32
// accumulation rounds:
//   bf16  x^ = code * step is exact in bf16, dy is used as it is
//   fp16  x^ is exact in fp16: a form of fp16 values has steps up to 2^9 (int8)
//         or 2^7 (e4m3), and one whose smallest codes lie below 2^-24 comes with
//         values that are multiples of 2^-24 and kept as they are; a form that
//         came from elsewhere is rounded to fp16 as unpacking rounds it
//   fp32  dy is split into three bf16 terms (24 significant bits) whose sum is
//         the value itself, one matrix product each with x^ in bf16; below
//         2^-110 the third term is cut at bf16's last place, 2^-133
#pragma once

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

// Bytes of LDS that a tile takes: two steps of dy (in each of its terms) and x^.
template <typename T, int BO, int BC, int BK>
constexpr int wgrad_lds = 2 * (kPlanes<T> * BK * BO * 2 + BK * BC * 2);

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

// Eight values x^ in the products' type: rounded to it as gq_*_unpack rounds them
// (exact for forms of its values, see above).
template <typename T>
__device__ __forceinline__ u32x4 packed(const float (&f)[8]) {
  return __builtin_bit_cast(
      u32x4, narrow<std::conditional_t<std::is_same_v<T, float>, __bf16, T>>(f));
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
// The sum runs over the tokens t0 .. t1 - 1; tokens from `end` on (t1 or
// further) read as zeros.  dw, db: of the tile's weight, or its part of them
// (db NULL: no bias; `parts`: a part, which beta does not concern).
template <typename T, typename Form, bool COPY, bool COLS, int BO, int BC, int WO, int WC, int BK>
__device__ __forceinline__ void wgrad_tile(const WgradArgs& a, char* lds, int ot, int ct,
                                           int64_t t0, int64_t t1, int64_t end, float* dw,
                                           bool w_part, float* db, bool b_part) {
  constexpr int P = kPlanes<T>;
  static_assert(COPY ? P == 1 : !COLS, "");
  constexpr int WAVES = (BO / WO) * (BC / WC), TH = WAVES * 64;
  constexpr int OT = WO / 32, CT = WC / 32, KK = BK / 16;
  constexpr int ABUF = P * BK * BO * 2, BBUF = BK * BC * 2, BUF = ABUF + BBUF;
  const int tid = (int)threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wo = wave % (BO / WO) * WO, wc = wave / (BO / WO) * WC;
  const int o0 = ot * BO, c0 = ct * BC;
  const int steps = (int)((t1 - t0 + BK - 1) / BK);

  // ---- dy.  Rows past the last lie behind the range and read as zeros;
  // columns past the last hold anything, and what they give is not stored.
  const char* dy = (const char*)((const T*)a.dy + o0);
  const int64_t row_bytes = a.lddy * (int64_t)sizeof(T);
  const int64_t dy_end = ((end - 1) * a.lddy + a.out - o0) * (int64_t)sizeof(T);
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
  int64_t rows_left = end - t0;
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
    Form::decode8(rc[i], rs[i], f);
    *(GQ_LDS u32x4*)(to + place<BC>(t, p / 2) + p % 2 * 16) =
        packed<T>(f);
  };

  // The bias's sums are shared out over the tiles of a row.  Tile ct < turns
  // takes the steps st with st % turns == ct, which gives parts, or (COLS, turns
  // a power of two) 1 / turns of the columns: `ppt` pieces of eight of each row.
  const bool bias = db != nullptr && ct < a.turns;
  const int ppt = COLS ? LPR / a.turns : LPR;
  auto add_piece = [&](LdsPtr from, int t, int p) {
    const u32x4 u = *(GQ_LDS u32x4*)(from + place<BO>(t, p / 2) + p % 2 * 16);
    float v[8];
    widen(__builtin_bit_cast(Raw8<std::conditional_t<sizeof(T) == 2, T, __bf16>>, u), v);
#pragma unroll
    for (int j = 0; j < 8; ++j) bsum[j] += v[j];
  };
  auto sum_dy = [&](LdsPtr from) {
    if constexpr (COLS) {
      // a thread's pieces lie in the same columns: TH is a multiple of ppt
      for (int q = tid; q < BK * ppt; q += TH)
        add_piece(from, q / ppt, ct * ppt + tid % ppt);
      return;
    }
    constexpr int N = BK * BO / 8 / TH;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int q = i * TH + tid;
      add_piece(from, q / LPR, q % LPR);
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
    const bool sum = !COLS && bias && turn == ct && st + 1 < steps;
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
      // in the middle of the step: right behind the barrier nothing hides it
      if (COLS && k == 0 && bias) sum_dy(now_a);
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
    if (COPY && !COLS && bias && ct == 0) sum_dy(a0);
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
  const float beta = w_part ? 0.f : a.beta;
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
    const int width = ppt * 8;
    __syncthreads();
    float* sh = reinterpret_cast<float*>(lds);  // [TH / ppt][width]
#pragma unroll
    for (int j = 0; j < 8; ++j) sh[tid / ppt * width + tid % ppt * 8 + j] = bsum[j];
    __syncthreads();
    if constexpr (COLS) {
      // 8 groups to a thread first, then those TH / width sums
      float s = 0.f;
#pragma unroll
      for (int g = 0; g < 8; ++g) s += sh[(tid / width * 8 + g) * width + tid % width];
      __syncthreads();
      sh[tid] = s;
      __syncthreads();
      const int o = o0 + ct * width + tid;
      if (tid < width && o < a.out) {
        s = 0.f;
        for (int g = 0; g < TH / width; ++g) s += sh[g * width + tid];
        float* q = db + o;
        *q = b_part || a.beta == 0.f ? s : fmaf(a.beta, *q, s);
      }
      return;
    }
    for (int o = tid; o < BO && o0 + o < a.out; o += TH) {
      float s = 0.f;
#pragma unroll
      for (int t = 0; t < TH / LPR; ++t) s += sh[t * BO + o];
      float* q = db + o0 + o;
      *q = b_part || a.beta == 0.f ? s : fmaf(a.beta, *q, s);
    }
  }
}

}  // namespace
}  // namespace gq
