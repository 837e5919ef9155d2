// fp8_linear.hip — the product of a linear layer from 8-bit floating point
// forms, of one weight or of one per expert:
//   y[t, o] = sum_c x^[t, c] w^[e(t), o, c] + b[e(t), o]
//
// Both operands are rows of e4m3 codes along the summed axis, 16-byte aligned
// and zero-padded, 32 consecutive ones per lane straight from LDS into the
// scaled matrix instruction, which multiplies by both steps' powers of two
// itself (fp8.hpp): one accumulator runs over all blocks of 128.
//
// The 8-bit matrix instructions (scaled or not) add eight products at a time,
// aligned at the largest and cut at 2^-13 of it, and only these sums in 24 bits
// (measured).  Eight cuts are up to 2^-10 of the eight's magnitudes, so a result may
// be off by 2^-10 of the sum of all magnitudes: a quarter of what bf16 rounds by at
// most, twice what fp16 does, and any share of a result whose terms cancel.  Measured
// over 16384 columns of codes of all sizes, in the 2-norm: of one sign fp16 1.7e-4 of
// the results (rounding alone 1.6e-4), bf16 1.3e-3 (1.3e-3); where all but 1.7 in 1000
// of the magnitudes cancel fp16 1.3e-3, bf16 2.1e-3, fp32 7e-6.  Callers for whom
// that is too much take fp32 results: there codes are decoded to bf16 (exact, with
// their step) between LDS and the matrix instruction, whose products are exact and
// summed in fp32, at half the rate.
//
// 8192 x 8192 x 4096 (tokens x out x cols): bf16 219 to 230 us in a loop, 2.4 to
// 2.5 PFLOP/s (the library's product of the same codes with one scale for all:
// 180 us), on inputs from HBM 240 to 244, fp32 405 to 420 and 435; 16384 x 2048 x
// 2048 64 us, over 32 experts of 512 tokens 68, from HBM 81 to 85 (fp32 133), of
// uneven loads 103 (168); with transposed forms the same within 5 %.  One token
// through 4096 x 4096 6.5 us, 2.6 TB/s of weight, through 16384 x 8192 22.5 us, 5.9
// TB/s.  Matrix cores are busy 57 % of 460k cycles at 2.1 GHz.  What is waited for are the copies to LDS: without any 178 us, all from
// the same lines in L2 219 of 228, without the reads from LDS no less.
#include <type_traits>

#include "fp8.hpp"
#include "fp8_plan.hpp"

namespace gq {
namespace {

typedef __attribute__((address_space(3))) uint8_t* LdsPtr;

// Up to 16 bytes of a row of y, of which `valid` values exist.
template <typename T>
__device__ __forceinline__ void store_piece(T* y, const u32x4& w, int valid) {
  constexpr int E = 16 / (int)sizeof(T);
  if (valid >= E) {
    __builtin_memcpy(y, &w, 16);
  } else {
    T o[E];
    __builtin_memcpy(o, &w, 16);
#pragma unroll
    for (int j = 0; j < E; ++j)
      if (j < valid) y[j] = o[j];
  }
}

struct LinearArgs {
  int64_t rows;
  int out, pitch, groups, experts;
  const int64_t* offsets;
  const uint8_t *codes, *w_codes;
  const float *steps, *w_steps, *bias;
  void* y;
  int64_t ldy;
  float* ws;
  int splits, per;  // per: 128-byte k-tiles of a split
  int ntiles;
};

// The experts' rows, tile by tile.  Boundaries are clamped to the matrix and
// made ascending, so that whatever the table holds there are at most rows / BM
// + experts tiles of rows, each within the matrix.
struct Experts {
  int bound[kMaxExperts + 1];   // first row of each, and the last one's end
  int first[kMaxExperts + 1];   // its first tile of rows
};

template <int BM>
__device__ __forceinline__ void read_experts(const LinearArgs& a, Experts& x) {
  if (threadIdx.x < 64) {
    const int lane = (int)threadIdx.x, n = a.experts + 1;
    const int each = (n + 63) / 64, lo = lane * each;
    int most = 0;
    for (int i = lo; i < min(lo + each, n); ++i) {
      const int64_t v = a.offsets ? a.offsets[i] : i * a.rows;
      most = max(most, (int)min(max(v, (int64_t)0), a.rows));
      x.bound[i] = most;
    }
    int before = most;          // largest of the lanes up to this one
    for (int d = 1; d < 64; d *= 2) {
      const int v = __shfl_up(before, d);
      if (lane >= d) before = max(before, v);
    }
    before = __shfl_up(before, 1);
    if (lane == 0) before = 0;
    for (int i = lo; i < min(lo + each, n); ++i) x.bound[i] = max(x.bound[i], before);
    // the lanes read each other's
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "workgroup");
    int tiles = 0;
    for (int i = lo; i < min(lo + each, a.experts); ++i) {
      x.first[i] = tiles;
      tiles += (x.bound[i + 1] - x.bound[i] + BM - 1) / BM;
    }
    int sum = tiles;
    for (int d = 1; d < 64; d *= 2) {
      const int v = __shfl_up(sum, d);
      if (lane >= d) sum += v;
    }
    for (int i = lo; i < min(lo + each, a.experts); ++i) x.first[i] += sum - tiles;
    if (lane == 63) x.first[a.experts] = sum;
  }
  __syncthreads();
}

struct ExpertTile {
  int row, end;       // rows of the expert from the tile's first on
  int j, split, expert;
};

// TileWalk over the experts' tiles of rows by ntiles tiles of columns.
struct ExpertWalk {
  const Experts& x;
  int ntiles, tiles, next, end, stride, e;

  __device__ __forceinline__ ExpertWalk(const Experts& x, int experts, int ntiles, int splits)
      : x(x), ntiles(ntiles), e(0) {
    tiles = __builtin_amdgcn_readfirstlane(x.first[experts]) * ntiles;
    const int total = tiles * splits, xcd = (int)blockIdx.x % 8;
    const int per = total / 8, more = total % 8, first = xcd * per + min(xcd, more);
    next = first + (int)blockIdx.x / 8;
    end = first + per + (xcd < more ? 1 : 0);
    stride = ((int)gridDim.x + 7) / 8;
  }

  template <int BM>
  __device__ __forceinline__ bool take(ExpertTile* t) {
    if (next >= end) return false;
    t->split = next / tiles;
    const int in = next - t->split * tiles;
    int a = __builtin_amdgcn_readfirstlane(x.first[e]);
    if (in < a * ntiles) {      // the next split
      e = 0;
      a = 0;
    }
    int b = __builtin_amdgcn_readfirstlane(x.first[e + 1]);
    while (in >= b * ntiles) {
      ++e;
      a = b;
      b = __builtin_amdgcn_readfirstlane(x.first[e + 1]);
    }
    const int k = in - a * ntiles, first = k / (8 * ntiles) * 8, h = min(8, b - a - first);
    const int r = k - first * ntiles;
    t->expert = e;
    t->row = __builtin_amdgcn_readfirstlane(x.bound[e]) + (first + r % h) * BM;
    t->end = __builtin_amdgcn_readfirstlane(x.bound[e + 1]);
    t->j = r / h;
    next += stride;
    return true;
  }
};

__device__ __forceinline__ i32x8 join16(i32x4 a, i32x4 b) {
  return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

// Among N neighbouring lanes (2 or 4): lane a's u[k] <- lane k's u[a].
template <int N>
__device__ __forceinline__ void transpose_lanes(u32x4 (&u)[N]) {
  const int lane = (int)threadIdx.x;
#pragma unroll
  for (int d = 1; d < N; d *= 2)
#pragma unroll
    for (int k = 0; k < N; ++k) {
      if (k & d) continue;
      const bool hi = (lane & d) != 0;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint32_t x = u[k][w], y = u[k | d][w];
        const uint32_t r = xshfl(hi ? x : y, d);
        u[k][w] = hi ? r : x;
        u[k | d][w] = hi ? y : r;
      }
    }
}

// Four consecutive results of a lane as the words of their type.
template <typename T>
__device__ __forceinline__ void words_of(const f32x4& v, uint32_t* w) {
  T o[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) o[r] = (T)v[r];
  __builtin_memcpy(w, o, sizeof(o));
}

// Eight codes times their step in bf16.
__device__ __forceinline__ bf16x8 bf16_of(int lo, int hi, float step) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)lo, step, false);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)lo, step, true);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)hi, step, false);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)hi, step, true);
  return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// c + a b over the 64 columns (32 x 32 results) or 128 (16 x 16) that the
// lanes hold 32 consecutive ones of; sa, sb: the steps' bits.
template <bool EXACT>
__device__ __forceinline__ f32x16 product(i32x8 a, i32x8 b, f32x16 c, uint32_t sa, uint32_t sb) {
  if constexpr (!EXACT) {
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 0, 0, 0, (int)(sa >> 23), 0,
                                                           (int)(sb >> 23));
  } else {
#pragma unroll
    for (int k = 0; k < 8; k += 2)
      c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
          bf16_of(a[k], a[k + 1], __uint_as_float(sa)),
          bf16_of(b[k], b[k + 1], __uint_as_float(sb)), c, 0, 0, 0);
    return c;
  }
}

template <bool EXACT>
__device__ __forceinline__ f32x4 product(i32x8 a, i32x8 b, f32x4 c, uint32_t sa, uint32_t sb) {
  if constexpr (!EXACT) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, (int)(sa >> 23), 0,
                                                            (int)(sb >> 23));
  } else {
#pragma unroll
    for (int k = 0; k < 8; k += 2)
      c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
          bf16_of(a[k], a[k + 1], __uint_as_float(sa)),
          bf16_of(b[k], b[k + 1], __uint_as_float(sb)), c, 0, 0, 0);
    return c;
  }
}

// Tiles of BM tokens by BN outputs, WM by WN of one per wave, in k-tiles of
// 128 codes, which is one step.  An LDS row is 128 bytes in eight 16-byte
// chunks, chunk j of row r at place j ^ (r / 2 % 8): sixteen lanes that read
// one chunk of sixteen rows then touch every bank once.  NS k-tiles share LDS:
// one is multiplied while NS - 1 are on their way.  (Four halves of 64 codes
// instead of two k-tiles, half a k-tile further ahead: 239 us instead of 219 for
// 8192 x 8192 x 4096.)  Steps come for four k-tiles at once, since each row's lie
// in a line of their own.  Workgroups stay and walk the tiles, and the copies run
// on into the next tile while the present one's last products run and its results
// leave.
//
// A small tile alone on its CU is a chain of waits (a k-tile of 64 x 64 takes 790
// cycles, of which its products are 128; with eight k-tiles on their way instead
// of four 18.9 us instead of 16.0 for 203 x 2050 x 4100 fp16).  TEAMS = 2: two
// teams of waves take every second k-tile each, in step, and add up in LDS (13.0
// us; four teams of two 12.9, but 256 x 2048 x 2048 9.0 and not 8.4).  Such a
// workgroup takes one tile only.
template <typename T, int BM, int BN, int WM, int WN, int NS, int TEAMS>
__global__ __launch_bounds__(TEAMS * (BM / WM) * (BN / WN) * 64, 2) void k_fp8_linear(
    LinearArgs a) {
  constexpr bool EXACT = std::is_same_v<T, float>;
  constexpr int BK = 128, CH = BK / 16, RPI = 64 / CH;
  constexpr int WAVES = (BM / WM) * (BN / WN);    // of a team
  static_assert(TEAMS == 1 || TEAMS == 2, "");
  constexpr int MT = WM / 32, NTL = WN / 32;
  constexpr int BUF = (BM + BN) * BK, ROUND = TEAMS * BUF;  // the teams' side by side
  // results leave in pieces of 16 bytes: a lane has UNITS of each 32 tokens
  constexpr int E = 16 / (int)sizeof(T), UNITS = WN / (2 * E), STORES = MT * UNITS;
  // steps of a tile's rows and of its (one or two) blocks of outputs; as many
  // slots as k-tiles, since each may be the first of another tile.  One slot
  // more for the bias, which is used when the copies are NS k-tiles ahead.
  constexpr int BLOCKS = (BN + kFp8Block - 1) / kFp8Block, SLOT = (BM + 2) * 16;
  static_assert(BM / 64 < WAVES - 1 && BLOCKS <= 2, "waves for the weight's steps and the bias");
  // One array: with several the compiler tells them apart, and waits for all
  // copies before it reads from one that they may go to.
  constexpr int STEPS = NS * ROUND, BIAS = STEPS + NS * SLOT, TABLE = BIAS + (NS + 1) * BN * 4;
  __shared__ __attribute__((aligned(16))) uint8_t lds[TABLE + sizeof(Experts)];
  Experts& experts = *reinterpret_cast<Experts*>(&lds[TABLE]);
  const int lane = (int)threadIdx.x & 63;
  const int id = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int team = TEAMS == 1 ? 0 : id / WAVES, wave = TEAMS == 1 ? id : id % WAVES;
  const int wm = wave % (BM / WM) * WM, wn = wave / (BM / WM) * WN;
  read_experts<BM>(a, experts);

  // copies: a wave instruction fills RPI rows of codes, each team of its own
  // k-tiles; every fourth k-tile one more of the first team brings the steps of
  // 64 rows, or of the weight (the wave past those), and every tile's first the
  // bias (the last wave).  Rows past the end lie behind the buffers' ranges and
  // read as zeros.
  constexpr int CM = BM / RPI / WAVES, CN = BN / RPI / WAVES;
  const int cl = lane % CH, rl = lane / CH;
  const bool row_steps = wave < BM / 64;
  const int step_at = (row_steps ? wave * 64 + lane : lane) * a.groups * 4;
  const int step_to = row_steps ? wave * 1024 : BM * 16;
  BufferRange bm, bn, bs;         // bs: of the steps, or the bias
  auto ranges_of = [&](const ExpertTile& t) {
    const int n = t.j * BN, rows = min(t.end - t.row, BM);
    // of this tile's rows only: shorter than kPastEnd whatever the matrix
    bm = range_of(a.codes + (int64_t)t.row * a.pitch, (int64_t)rows * a.pitch);
    bn = range_of(a.w_codes + ((int64_t)t.expert * a.out + n) * a.pitch,
                  (int64_t)min(a.out - n, BN) * a.pitch);
    const int blocks = div_up(a.out, kFp8Block), block = n / kFp8Block;
    bs = wave == WAVES - 1
             ? range_of(a.bias + (int64_t)t.expert * a.out + n,
                        a.bias ? (int64_t)min(a.out - n, BN) * 4 : 0)
         : row_steps
             ? range_of(a.steps + (int64_t)t.row * a.groups, (int64_t)rows * a.groups * 4)
             : range_of(a.w_steps + ((int64_t)t.expert * blocks + block) * a.groups,
                        (int64_t)min(blocks - block, BLOCKS) * a.groups * 4);
  };
  const int k_tiles = a.groups;
  // what is copied next: k-tile ck + team (up to cend) of the walk's last tile,
  // into cat
  ExpertWalk copies(experts, a.experts, a.ntiles, a.splits);
  ExpertTile ctile;
  bool copying = copies.take<BM>(&ctile);
  int ck = 0, cend = 0, cat = team * BUF, csteps = 0, csat = 0, cbias = 0;
  bool cfirst = true;
  auto enter = [&] {
    ranges_of(ctile);
    cfirst = true;
    csteps = ck = ctile.split * a.per;
    cend = min(ck + a.per, k_tiles);
  };
  auto copy_next = [&] {
    if (!copying) return;
    const int k0 = (ck + team) * BK;
    // chunks past the pitch (in the last, short k-tile; the second team has one
    // past the last of an odd number) are zeros too
    const int left = (a.pitch - k0) / 16;
#pragma unroll
    for (int i = 0; i < CM; ++i) {
      const int r = (wave * CM + i) * RPI + rl, c = cl ^ (r / 2 % CH);
      copy16_to_lds(bm, c < left ? r * a.pitch + c * 16 : kPastEnd, k0,
                    (LdsPtr)&lds[cat + (wave * CM + i) * 1024]);
    }
#pragma unroll
    for (int i = 0; i < CN; ++i) {
      const int r = (wave * CN + i) * RPI + rl, c = cl ^ (r / 2 % CH);
      copy16_to_lds(bn, c < left ? r * a.pitch + c * 16 : kPastEnd, k0,
                    (LdsPtr)&lds[cat + BM * BK + (wave * CN + i) * 1024]);
    }
    if (team == 0 && ck == csteps) {
      // what lies past a row's last step is not used
      if (row_steps || (wave == BM / 64 && lane < BLOCKS))
        copy16_to_lds(bs, step_at, ck * 4, (LdsPtr)&lds[STEPS + csat + step_to]);
      if (wave == WAVES - 1 && cfirst) {
        if (lane < BN / 4) copy16_to_lds(bs, lane * 16, 0, (LdsPtr)&lds[BIAS + cbias]);
        cbias = cbias == NS * BN * 4 ? 0 : cbias + BN * 4;
        cfirst = false;
      }
      csteps += 4;
      csat = csat + SLOT == NS * SLOT ? 0 : csat + SLOT;
    }
    cat = cat + ROUND >= NS * ROUND ? team * BUF : cat + ROUND;
    ck += TEAMS;
    if (ck >= cend) {
      copying = TEAMS == 1 && copies.take<BM>(&ctile);
      if (copying) enter();
    }
  };
  // Waits until this wave's reads are done and its copies but those of the
  // LEFT youngest k-tiles have arrived, then for the other waves.  Copies and
  // stores are done with in order.  `stored`: behind those copies there are the
  // STORES of a whole tile's results, which need not have left; anything else in
  // flight (steps, other results) only makes the wait longer.  Once there is
  // nothing left to copy the youngest are fewer, so all are waited for.
  auto meet = [&](auto left, bool all, bool stored) {
    constexpr int LEFT = decltype(left)::value;
    if (all) {
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    } else if (stored) {
      asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(LEFT * (CM + CN) + STORES) : "memory");
    } else {
      asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(LEFT * (CM + CN)) : "memory");
    }
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };

  // Fragments: 32 rows by 64 codes.  Those of the next half k-tile are read
  // between the present one's products, a token's as soon as its last product
  // is on its way and into the same registers (the scheduling barriers: all at
  // once they would need 32 more than there are).
  const int fr = lane % 32;
  int place[2][2];
#pragma unroll
  for (int kk = 0; kk < 2; ++kk)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      place[kk][h] = fr * BK + (((kk * 4 + lane / 32 * 2 + h) ^ (fr / 2 % CH)) << 4);
  auto half = [&](int at, int row, int kk, int h) {
    return *reinterpret_cast<const i32x4*>(&lds[at + row * BK + place[kk][h]]);
  };
  i32x4 fm[MT][2], fn[2][NTL][2];
  uint32_t em[2][MT], en[2];      // the steps, of this k-tile and the next
  auto read_m = [&](int j, int at, int kk) {
#pragma unroll
    for (int h = 0; h < 2; ++h) fm[j][h] = half(at, wm + j * 32, kk, h);
  };
  // the j-th of MT parts of the weight's
  auto read_n = [&](int j, int to, int at, int kk) {
#pragma unroll
    for (int i = j * 2 * NTL / MT; i < (j + 1) * 2 * NTL / MT; ++i)
      fn[to][i / 2][i % 2] = half(at + BM * BK, wn + i / 2 * 32, kk, i % 2);
  };
  int sat = 0;                    // where the steps of the next k-tile lie
  auto read_steps = [&](int to) {
#pragma unroll
    for (int j = 0; j < MT; ++j)
      em[to][j] = *reinterpret_cast<const uint32_t*>(&lds[STEPS + sat + team * 4 + (wm + j * 32 + fr) * 16]);
    en[to] = *reinterpret_cast<const uint32_t*>(
        &lds[STEPS + sat + team * 4 + (BM + (BN > kFp8Block ? wn / kFp8Block : 0)) * 16]);
  };
  // on to the next k-tile's, `k` of them behind the tile's first
  auto next_steps = [&](int k) {
    if (k & 3) sat += 4 * TEAMS;
    else sat = sat / SLOT + 1 == NS ? 0 : (sat / SLOT + 1) * SLOT;
  };

  ExpertWalk walk(experts, a.experts, a.ntiles, a.splits);
  ExpertTile tile;
  if (!walk.take<BM>(&tile)) return;
  enter();
#pragma unroll
  for (int i = 0; i < NS; ++i) copy_next();
  meet(std::integral_constant<int, NS - 1>{}, !copying, false);
  int at = team * BUF, bias = 0;           // places of the k-tile and of the tile's bias
  bool stored = false;
  read_steps(0);
#pragma unroll
  for (int j = 0; j < MT; ++j) {
    read_m(j, at, 0);
    read_n(j, 0, at, 0);
  }
  for (;;) {
    const int n0 = tile.j * BN;
    const int first = tile.split * a.per, last = min(first + a.per, k_tiles);
    f32x16 acc[NTL][MT];
#pragma unroll
    for (int i = 0; i < NTL; ++i)
#pragma unroll
      for (int j = 0; j < MT; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
    for (int kt = first; kt < last; kt += TEAMS) {
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        if (kk == 1) {
          // keeps the first half's products before the barrier: the compiler
          // would move them behind the copies' branches, to the others
#pragma unroll
          for (int i = 0; i < NTL; ++i)
#pragma unroll
            for (int j = 0; j < MT; ++j) asm volatile("" : "+v"(acc[i][j]));
          // the next k-tile is in LDS and this one is read: its place is free
          meet(std::integral_constant<int, NS - 2>{}, !copying, stored);
          stored = false;
          copy_next();
          at = at + ROUND >= NS * ROUND ? team * BUF : at + ROUND;
          next_steps(kt + TEAMS >= last ? 0 : kt + TEAMS - first);
          read_steps(1);
        }
#pragma unroll
        for (int j = 0; j < MT; ++j) {
#pragma unroll
          for (int i = 0; i < NTL; ++i)
            // (of a k-tile past the last the steps are other rows')
            if (TEAMS == 1 || kt + team < last)
              acc[i][j] = product<EXACT>(join16(fn[kk][i][0], fn[kk][i][1]),
                                       join16(fm[j][0], fm[j][1]), acc[i][j], en[0], em[0][j]);
          read_m(j, at, 1 - kk);
          read_n(j, 1 - kk, at, 1 - kk);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
#pragma unroll
      for (int j = 0; j < MT; ++j) em[0][j] = em[1][j];
      en[0] = en[1];
    }
    if constexpr (TEAMS == 2) {
      // no copies are on their way, and behind this barrier no reads
      __syncthreads();
      f32x4* sums = reinterpret_cast<f32x4*>(&lds[0]) + wave * (NTL * MT * 4 * 64) + lane;
#pragma unroll
      for (int i = 0; i < NTL * MT * 4; ++i) {
        const f32x16& c = acc[i / 4 / MT][i / 4 % MT];
        const int q = i % 4 * 4;
        if (team == 1) sums[i * 64] = f32x4{c[q], c[q + 1], c[q + 2], c[q + 3]};
      }
      __syncthreads();
      if (team == 1) return;
#pragma unroll
      for (int i = 0; i < NTL * MT * 4; ++i) {
        const f32x4 v = sums[i * 64];
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[i / 4 / MT][i / 4 % MT][i % 4 * 4 + r] += v[r];
      }
    }
    // A lane holds, of one token per 32 x 32 tile, four consecutive outputs in
    // each of the tile's four quarters, the lane 32 further the next four.  In 16
    // bits the two first swap halves, so that each has eight consecutive outputs
    // of every second quarter.  Then neighbouring lanes, which have neighbouring
    // tokens, exchange their 16-byte pieces: each store writes whole lines (128
    // bytes of a row; 64 where the wave's part is 32 outputs of 16 bits).
    if (a.splits == 1) {
      constexpr int G = UNITS < 4 ? UNITS : 4;    // lanes that exchange
      const int half = lane / 32, nb = lane % G;
      stored = tile.row + BM <= tile.end && n0 + BN <= a.out;
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        u32x4 u[UNITS / G][G];
#pragma unroll
        for (int i = 0; i < NTL; ++i)
#pragma unroll
          for (int q = 0; q < 4; q += sizeof(T) == 2 ? 2 : 1) {
            auto result = [&](int q) {
              const int n = wn + i * 32 + q * 8 + half * 4;
              const f32x4 b = *reinterpret_cast<const f32x4*>(&lds[BIAS + bias + n * 4]);
              f32x4 v;
#pragma unroll
              for (int r = 0; r < 4; ++r) v[r] = acc[i][j][q * 4 + r] + b[r];
              return v;
            };
            u32x4 w;
            if constexpr (sizeof(T) == 2) {
              uint32_t x[2], y[2];
              words_of<T>(result(q), x);
              words_of<T>(result(q + 1), y);
#pragma unroll
              for (int r = 0; r < 2; ++r) {
                const auto z = __builtin_amdgcn_permlane32_swap(x[r], y[r], false, false);
                w[r] = z[0];
                w[2 + r] = z[1];
              }
            } else {
              w = __builtin_bit_cast(u32x4, result(q));
            }
            const int k = sizeof(T) == 2 ? i * 2 + q / 2 : i * 4 + q;
            u[k / G][k % G] = w;
          }
#pragma unroll
        for (int g = 0; g < UNITS / G; ++g) {
          transpose_lanes(u[g]);
          // piece nb of the group, of token k of the neighbours
          const int n = n0 + wn + (g * G + nb) * (2 * E) + half * E;
#pragma unroll
          for (int k = 0; k < G; ++k) {
            const int m = tile.row + wm + j * 32 + fr - nb + k;
            if (m < tile.end) store_piece((T*)a.y + m * a.ldy + n, u[g][k], a.out - n);
          }
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        const int m = tile.row + wm + j * 32 + fr;
        if (m >= tile.end) continue;
#pragma unroll
        for (int i = 0; i < NTL; ++i)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int n = n0 + wn + i * 32 + q * 8 + lane / 32 * 4;
            float* p = a.ws + ((int64_t)tile.split * a.rows + m) * a.out + n;
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (n + r < a.out) p[r] = acc[i][j][q * 4 + r];
          }
      }
    }
    if (TEAMS > 1 || !walk.take<BM>(&tile)) return;
    bias = bias == NS * BN * 4 ? 0 : bias + BN * 4;
  }
}

// The splits' sums, added in order, of the rows that belong to an expert.
template <typename T>
__global__ __launch_bounds__(256) void k_fp8_linear_join(LinearArgs a) {
  const int64_t total = a.rows * a.out;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * 256) {
    const int64_t m = i / a.out;
    const int n = (int)(i - m * a.out);
    int e = 0;
    if (a.offsets) {
      int hi = a.experts;       // offsets[e] <= m < offsets[hi], or none
      if (m < a.offsets[0] || m >= a.offsets[hi]) continue;
      while (hi - e > 1) {
        const int mid = (e + hi) / 2;
        if (a.offsets[mid] <= m) e = mid;
        else hi = mid;
      }
    }
    float s = a.ws[i];
    for (int k = 1; k < a.splits; ++k) s += a.ws[k * total + i];
    if (a.bias) s += a.bias[(int64_t)e * a.out + n];
    ((T*)a.y)[m * a.ldy + n] = (T)s;
  }
}

// Few tokens.  A workgroup takes 16 * MT tokens of an expert by 16 * NT outputs;
// its eight waves take turns of four k-tiles along the sum and add up in LDS.
// Operands come straight from memory and L2 in the products' layout, 32 codes of
// one row per lane, 16 rows by 128 codes per instruction: nothing waits for a
// barrier until the sums are joined.
constexpr int kFewWaves = 8;

template <typename T, int MT, int NT>
__global__ __launch_bounds__(kFewWaves * 64) void k_fp8_linear_few(LinearArgs a) {
  constexpr bool EXACT = std::is_same_v<T, float>;
  constexpr int U = 4, HALF = kFewWaves / 2, E = MT * NT * 256;
  __shared__ __attribute__((aligned(16))) float sums[HALF][E];
  const int lane = (int)threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int n0 = (int)blockIdx.x * (16 * NT), expert = (int)blockIdx.y;
  const Tokens t = tokens_of(a.offsets, expert, a.rows);
  const int blocks = div_up(a.out, kFp8Block);
  const BufferRange w = range_of(a.w_codes + ((int64_t)expert * a.out + n0) * a.pitch,
                                 (int64_t)min(a.out - n0, 16 * NT) * a.pitch);
  // 16 * NT outputs lie in one block
  const BufferRange sw =
      range_of(a.w_steps + ((int64_t)expert * blocks + n0 / kFp8Block) * a.groups,
               (int64_t)a.groups * 4);
  const float* bias = a.bias ? a.bias + (int64_t)expert * a.out : nullptr;
  const int row = lane % 16 * a.pitch, col = lane / 16 * 32;
  const int64_t m0 = t.lo + (int64_t)blockIdx.z * (16 * MT);
  if (m0 >= t.hi) return;
  const int64_t rows = min(t.hi - m0, (int64_t)(16 * MT));
  const BufferRange x = range_of(a.codes + m0 * a.pitch, rows * a.pitch);
  const BufferRange sx = range_of(a.steps + m0 * a.groups, rows * a.groups * 4);
  f32x4 acc[NT][MT];
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int i = 0; i < MT; ++i) acc[j][i] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int k = wave * U; k < a.groups; k += kFewWaves * U) {
    i32x8 fw[U][NT], fx[U][MT];
    u32x4 ew, ex[MT];
    auto load = [&](const BufferRange& r, int c, int at) {
      // past the pitch lies the next row: those chunks are zeros
      const i32x4 lo = __builtin_bit_cast(
          i32x4, __builtin_amdgcn_raw_buffer_load_b128(r, c < a.pitch ? at + c : kPastEnd, 0, 0));
      const i32x4 hi = __builtin_bit_cast(
          i32x4, __builtin_amdgcn_raw_buffer_load_b128(
                     r, c + 16 < a.pitch ? at + c + 16 : kPastEnd, 0, 0));
      return join16(lo, hi);
    };
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = (k + u) * 128 + col;
#pragma unroll
      for (int j = 0; j < NT; ++j) fw[u][j] = load(w, c, row + j * 16 * a.pitch);
#pragma unroll
      for (int i = 0; i < MT; ++i) fx[u][i] = load(x, c, row + i * 16 * a.pitch);
    }
    ew = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(sw, k * 4, 0, 0));
#pragma unroll
    for (int i = 0; i < MT; ++i)
      ex[i] = __builtin_bit_cast(
          u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                     sx, ((lane % 16 + i * 16) * a.groups + k) * 4, 0, 0));
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (k + u >= a.groups) break;   // there lie other rows' steps
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < MT; ++i)
          acc[j][i] = product<EXACT>(fw[u][j], fx[u][i], acc[j][i], ew[u], ex[i][u]);
    }
  }
  // a lane holds four consecutive outputs of token lane % 16; kept as
  // [token][output], 16 * NT outputs to a token
  auto at = [&](int j, int i) {
    return (i * 16 + lane % 16) * (16 * NT) + j * 16 + lane / 16 * 4;
  };
  if (wave >= HALF) {
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < MT; ++i)
        *reinterpret_cast<f32x4*>(&sums[wave - HALF][at(j, i)]) = acc[j][i];
  }
  __syncthreads();
  if (wave < HALF) {
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        f32x4* p = reinterpret_cast<f32x4*>(&sums[wave][at(j, i)]);
        *p += acc[j][i];
      }
  }
  __syncthreads();
  for (int e = (int)threadIdx.x * 4; e < E; e += kFewWaves * 64 * 4) {
    const int64_t m = m0 + e / (16 * NT);
    const int n = n0 + e % (16 * NT);
    if (m >= t.hi || n >= a.out) continue;
    f32x4 s = *reinterpret_cast<const f32x4*>(&sums[0][e]);
#pragma unroll
    for (int v = 1; v < HALF; ++v) s += *reinterpret_cast<const f32x4*>(&sums[v][e]);
    T o[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) o[r] = (T)(s[r] + (bias ? bias[min(n + r, a.out - 1)] : 0.f));
    T* y = (T*)a.y + m * a.ldy + n;
    if (n + 4 <= a.out) {
      __builtin_memcpy(y, o, sizeof(o));
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (n + r < a.out) y[r] = o[r];
    }
  }
}

template <typename T, int MT, int NT>
void few(const LinearArgs& a, hipStream_t st) {
  const dim3 g(div_up(a.out, 16 * NT), a.experts, div_up(a.rows, 16 * MT));
  k_fp8_linear_few<T, MT, NT><<<g, kFewWaves * 64, 0, st>>>(a);
}

template <typename T>
int linear_t(const LinearPlan& p, LinearArgs a, hipStream_t st) {
  if (p.tile == 0) {
    if (a.experts > 1 || a.rows <= 16) few<T, 1, 1>(a, st);
    else if (a.rows <= 32) few<T, 2, 1>(a, st);
    else few<T, 2, 2>(a, st);
    return (int)hipGetLastError();
  }
  const unsigned g = (unsigned)p.grid;
  if (p.tile == 256) k_fp8_linear<T, 256, 256, 128, 64, 2, 1><<<g, 512, 0, st>>>(a);
  else if (p.tile == 128) k_fp8_linear<T, 128, 128, 64, 32, 4, 1><<<g, 512, 0, st>>>(a);
  else if (p.teams == 2) k_fp8_linear<T, 64, 64, 32, 32, 4, 2><<<g, 512, 0, st>>>(a);
  else k_fp8_linear<T, 64, 64, 32, 32, 4, 1><<<g, 256, 0, st>>>(a);
  int rc = (int)hipGetLastError();
  if (rc == 0 && a.splits > 1) {
    const int64_t b = (a.rows * a.out + 255) / 256;
    k_fp8_linear_join<T><<<(unsigned)(b < 4096 ? b : 4096), 256, 0, st>>>(a);
    rc = (int)hipGetLastError();
  }
  return rc;
}

}  // namespace

int64_t fp8_linear_workspace(const ActDims& A, int64_t out, int experts) {
  if (A.rows == 0) return 0;
  const LinearPlan p = plan_linear(A.rows, A.groups, out, experts);
  return p.splits > 1 ? 4 * p.splits * A.rows * out : 0;
}

int launch_fp8_linear(const ActDims& A, int64_t out, int experts, const int64_t* offsets,
                      const uint8_t* codes, const float* steps, const uint8_t* w_codes,
                      const float* w_steps, const float* bias, void* y, int64_t ldy, void* ws,
                      hipStream_t st) {
  if (A.rows == 0) return 0;
  const LinearPlan p = plan_linear(A.rows, A.groups, out, experts);
  const LinearArgs a = {A.rows, (int)out, (int)A.pitch, A.groups, experts, offsets,
                        codes,  w_codes,  steps,        w_steps,  bias,    y,
                        ldy,    (float*)ws, p.splits,   p.per,
                        p.tile ? div_up(out, p.tile) : 0};
  switch (A.dtype) {
    case GQ_F32: return linear_t<float>(p, a, st);
    case GQ_BF16: return linear_t<__bf16>(p, a, st);
    default: return linear_t<_Float16>(p, a, st);
  }
}

}  // namespace gq
