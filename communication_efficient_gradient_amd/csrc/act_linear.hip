// act_linear.hip — the product of a linear layer in 8-bit integers:
//   y[t, o] = (sum_c q[t, c] w[o, c]) s[t] v[o] + b[o]
// with one step s per token and one v per output feature.  The integer sums
// are exact (int32, |code| <= 128, so up to 131071 columns), in any order.
//
// Both operands are rows of int8 along the summed axis, 16-byte aligned and
// zero-padded, which is the layout the matrix instructions take: 16 (32x32x32)
// consecutive codes per lane, straight from LDS.  8192 x 8192 x 4096 (tokens x
// out x cols): 233 us in a loop, 2.4 POP/s, median 272 (255 to 293) under the
// profiler; one token through 4096 x 4096: median 6.3 us (5.2 to 6.6), 2.7 TB/s
// of weight, and through 16384 x 8192 24 us, 5.6 TB/s.
#include "act.hpp"

namespace gq {
namespace {

typedef __attribute__((address_space(3))) int8_t* LdsPtr;

template <typename T>
struct Word16 {
  typedef T V __attribute__((ext_vector_type(16 / sizeof(T))));
};

// Up to 16 bytes of a row of y, of which `valid` values exist.
template <typename T, typename V>
__device__ __forceinline__ void store_piece(T* y, const V& w, int valid) {
  constexpr int E = 16 / (int)sizeof(T);
  if (valid >= E) {
    __builtin_memcpy(y, &w, 16);
  } else {
#pragma unroll
    for (int j = 0; j < E; ++j)
      if (j < valid) y[j] = w[j];
  }
}

struct LinearArgs {
  int64_t rows;
  int out, pitch;
  const int8_t *codes, *w_codes;
  const float *steps, *w_steps, *bias;
  void* y;
  int64_t ldy;
  int32_t* ws;
  int splits, per;  // per: 128-byte k-tiles of a split
  int mtiles, ntiles;
};

// Tiles of BM tokens by BN outputs, WM by WN of one per wave, in k-tiles of BK
// codes.  An LDS row is BK bytes in CH 16-byte chunks, chunk j of row r at
// place j ^ (r / (16 / CH) % CH): sixteen lanes that read one chunk of sixteen
// rows then touch every bank once.  NS k-tiles share LDS: one is multiplied
// while NS - 1 are on their way.  Workgroups stay and walk the tiles, and the
// copies run on into the next tile while the present one's last products run
// and its results leave.
template <typename T, int BM, int BN, int WM, int WN, int BK, int NS>
__global__ __launch_bounds__((BM / WM) * (BN / WN) * 64, 2) void k_act_linear(LinearArgs a) {
  constexpr int CH = BK / 16, KK = BK / 32, RPI = 64 / CH;
  constexpr int WAVES = (BM / WM) * (BN / WN);
  constexpr int MT = WM / 32, NTL = WN / 32;
  constexpr int BUF = (BM + BN) * BK;
  __shared__ __attribute__((aligned(16))) int8_t lds[NS * BUF];
  const int lane = (int)threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int wm = wave % (BM / WM) * WM, wn = wave / (BM / WM) * WN;

  // copies: a wave instruction fills RPI rows.  Rows past the end lie behind
  // the buffers' ranges and read as zeros.
  constexpr int CM = BM / RPI / WAVES, CN = BN / RPI / WAVES;
  const int cl = lane % CH, rl = lane / CH;
  BufferRange bm, bn;
  auto ranges_of = [&](const Tile& t) {
    const int64_t m = (int64_t)t.i * BM, n = (int64_t)t.j * BN;
    // of this tile's rows only: shorter than kPastEnd whatever the matrix
    bm = range_of(a.codes + m * a.pitch, min(a.rows - m, (int64_t)BM) * a.pitch);
    bn = range_of(a.w_codes + n * a.pitch, min(a.out - n, (int64_t)BN) * a.pitch);
  };
  const int k_tiles = div_up(a.pitch, BK);
  // what is copied next: k-tile ck (up to cend) of the walk's last tile, into cat
  TileWalk copies(a.mtiles, a.ntiles, a.splits);
  Tile ctile;
  bool copying = copies.take(&ctile);
  int ck = 0, cend = 0, cat = 0;
  auto enter = [&] {
    ranges_of(ctile);
    ck = ctile.split * a.per;
    cend = min(ck + a.per, k_tiles);
  };
  auto copy_next = [&] {
    if (!copying) return;
    const int k0 = ck * BK;
    // chunks past the pitch (in the last, short k-tile) are zeros too
    const int left = (a.pitch - k0) / 16;
#pragma unroll
    for (int i = 0; i < CM; ++i) {
      const int r = (wave * CM + i) * RPI + rl, c = cl ^ (r / (16 / CH) % CH);
      copy16_to_lds(bm, c < left ? r * a.pitch + c * 16 : kPastEnd, k0,
                    (LdsPtr)&lds[cat + (wave * CM + i) * 1024]);
    }
#pragma unroll
    for (int i = 0; i < CN; ++i) {
      const int r = (wave * CN + i) * RPI + rl, c = cl ^ (r / (16 / CH) % CH);
      copy16_to_lds(bn, c < left ? r * a.pitch + c * 16 : kPastEnd, k0,
                    (LdsPtr)&lds[cat + BM * BK + (wave * CN + i) * 1024]);
    }
    cat = cat + BUF == NS * BUF ? 0 : cat + BUF;
    if (++ck == cend) {
      copying = copies.take(&ctile);
      if (copying) enter();
    }
  };
  // Waits until this wave's reads are done and its copies but those of the NS -
  // 2 youngest k-tiles have arrived, then for the other waves.  Copies arrive
  // in order; anything else in flight (results on their way out) only makes
  // the wait longer.  Once there is nothing left to copy the youngest are
  // fewer, so all are waited for.
  auto meet = [&](bool all) {
    if (NS == 2 || all) {
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    } else {
      asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"((NS - 2) * (CM + CN)) : "memory");
    }
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };

  // The next k-step's fragments (32 rows by 32 codes) are read from LDS between
  // the present one's products (the scheduling groups); the next k-tile is on
  // its way into the other buffer.
  const int fr = lane % 32;
  int place[KK];
#pragma unroll
  for (int kk = 0; kk < KK; ++kk)
    place[kk] = fr * BK + (((kk * 2 + lane / 32) ^ (fr / (16 / CH) % CH)) << 4);
  i32x4 fm[2][MT], fn[2][NTL];
  auto read = [&](int to, int at, int kk) {
    const int8_t* p = &lds[at + place[kk]];
#pragma unroll
    for (int i = 0; i < NTL; ++i)
      fn[to][i] = *reinterpret_cast<const i32x4*>(p + (BM + wn + i * 32) * BK);
#pragma unroll
    for (int j = 0; j < MT; ++j)
      fm[to][j] = *reinterpret_cast<const i32x4*>(p + (wm + j * 32) * BK);
  };

  TileWalk walk(a.mtiles, a.ntiles, a.splits);
  Tile tile;
  if (!walk.take(&tile)) return;
  enter();
#pragma unroll
  for (int i = 0; i < NS - 1; ++i) copy_next();
  meet(!copying);
  read(0, 0, 0);
  int at = 0;
  for (;;) {
    const int64_t m0 = (int64_t)tile.i * BM;
    const int n0 = tile.j * BN;
    const int first = tile.split * a.per, last = min(first + a.per, k_tiles);
    i32x16 acc[NTL][MT];
#pragma unroll
    for (int i = 0; i < NTL; ++i)
#pragma unroll
      for (int j = 0; j < MT; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0;
    int was = at;
    for (int kt = first; kt < last; ++kt) {
      was = at;
      copy_next();
#pragma unroll
      for (int kk = 0; kk < KK; ++kk) {
        if (kk < KK - 1) {
          read((kk + 1) & 1, at, kk + 1);
        } else {
          meet(!copying);  // the next k-tile is in LDS, this one is read
          at = at + BUF == NS * BUF ? 0 : at + BUF;
          read(0, at, 0);
        }
#pragma unroll
        for (int j = 0; j < MT; ++j)
#pragma unroll
          for (int i = 0; i < NTL; ++i)
            acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fn[kk & 1][i], fm[kk & 1][j],
                                                             acc[i][j], 0, 0, 0);
#pragma unroll
        for (int g = 0; g < MT + NTL; ++g) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        }
        if (MT * NTL > MT + NTL)
          __builtin_amdgcn_sched_group_barrier(0x008, MT * NTL - MT - NTL, 0);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    // A lane holds, of one token per 32 x 32 tile, four consecutive outputs in
    // each of the tile's four quarters: eight bytes of bf16, at 32 rows of y.
    // The wave's results therefore go through its own part of the buffer that
    // the last k-tile left, TOK tokens at a time, and leave as whole 16-byte
    // pieces of WN-long rows (8192 x 8192 x 4096: 321 us with direct stores).
    if (a.splits == 1) {
      using V = typename Word16<T>::V;  // 16 bytes of results
      constexpr int E = 16 / (int)sizeof(T), ROW = WN / E;  // pieces per row
      constexpr int MINE = BUF / WAVES, FIT = MINE / (WN * (int)sizeof(T));
      constexpr int TOK = FIT < WM ? FIT : WM;
      static_assert(TOK % 32 == 0 && WM % TOK == 0, "");
      int8_t* mine = lds + was + wave * MINE;
      const int lo = lane / 32 * 4;
      const bool whole = n0 + BN <= a.out;
#pragma unroll
      for (int j0 = 0; j0 < MT; j0 += TOK / 32) {
        float s[TOK / 32];
#pragma unroll
        for (int jj = 0; jj < TOK / 32; ++jj)
          s[jj] = a.steps[min(m0 + wm + (j0 + jj) * 32 + fr, a.rows - 1)];
#pragma unroll
        for (int i = 0; i < NTL; ++i)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int n = i * 32 + q * 8 + lo;
            float v[4], b[4] = {0.f, 0.f, 0.f, 0.f};
            if (whole) {
              __builtin_memcpy(v, a.w_steps + n0 + wn + n, 16);
              if (a.bias) __builtin_memcpy(b, a.bias + n0 + wn + n, 16);
            } else {
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                const int o = min(n0 + wn + n + r, a.out - 1);
                v[r] = a.w_steps[o];
                if (a.bias) b[r] = a.bias[o];
              }
            }
#pragma unroll
            for (int jj = 0; jj < TOK / 32; ++jj) {
              const int row = jj * 32 + fr;
              T o[4];
#pragma unroll
              for (int r = 0; r < 4; ++r)
                o[r] = (T)((float)acc[i][j0 + jj][q * 4 + r] * s[jj] * v[r] + b[r]);
              // piece p of row `row` is kept at place p ^ (row % ROW)
              __builtin_memcpy(
                  mine + (row * ROW + ((n / E) ^ (row % ROW))) * 16 + n % E * (int)sizeof(T),
                  o, sizeof(o));
            }
          }
#pragma unroll
        for (int k = 0; k < TOK * ROW / 64; ++k) {
          const int row = (k * 64 + lane) / ROW, p = lane % ROW;
          const V w = *reinterpret_cast<const V*>(mine + (row * ROW + (p ^ (row % ROW))) * 16);
          const int64_t m = m0 + wm + j0 * 32 + row;
          const int n = n0 + wn + p * E;
          if (m < a.rows) store_piece((T*)a.y + m * a.ldy + n, w, a.out - n);
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        const int64_t m = m0 + wm + j * 32 + lane % 32;
        if (m >= a.rows) continue;
#pragma unroll
        for (int i = 0; i < NTL; ++i)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int n = n0 + wn + i * 32 + q * 8 + lane / 32 * 4;
            int32_t* p = a.ws + ((int64_t)tile.split * a.rows + m) * a.out + n;
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (n + r < a.out) p[r] = acc[i][j][q * 4 + r];
          }
      }
    }
    if (!walk.take(&tile)) return;
    // all waves are done with the buffer that is filled next
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  }
}

// The splits' integer sums, added and scaled.
template <typename T>
__global__ __launch_bounds__(256) void k_act_linear_join(LinearArgs a) {
  const int64_t total = a.rows * a.out;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * 256) {
    const int64_t m = i / a.out;
    const int n = (int)(i - m * a.out);
    int32_t acc = 0;
    for (int s = 0; s < a.splits; ++s) acc += a.ws[s * total + i];
    const float f = (float)acc * a.steps[m] * a.w_steps[n] + (a.bias ? a.bias[n] : 0.f);
    ((T*)a.y)[m * a.ldy + n] = (T)f;
  }
}

// Few tokens.  A workgroup takes 16 * MT tokens by 16 * NT outputs; its eight
// waves take turns of U * 64 codes along the sum and add up in LDS.  Operands
// come straight from memory (the weight once up to 32 tokens, which MT covers,
// twice above) and L2 in the products' layout, 16 codes of one row per lane, 16 rows by 64 codes
// per instruction: nothing waits for a barrier until the sums are joined, and
// U steps of loads per wave are in flight at once.
constexpr int kFewWaves = 8;

template <typename T, int MT, int NT, int U>
__global__ __launch_bounds__(kFewWaves * 64) void k_act_linear_few(LinearArgs a) {
  constexpr int HALF = kFewWaves / 2, E = MT * NT * 256;
  __shared__ __attribute__((aligned(16))) int32_t sums[HALF][E];
  const int lane = (int)threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int n0 = (int)blockIdx.x * (16 * NT);
  const int64_t m0 = (int64_t)blockIdx.y * (16 * MT);
  const BufferRange w = range_of(a.w_codes + (int64_t)n0 * a.pitch,
                                 (int64_t)min(a.out - n0, 16 * NT) * a.pitch);
  const BufferRange x = range_of(a.codes + m0 * a.pitch,
                                 min(a.rows - m0, (int64_t)(16 * MT)) * a.pitch);
  const int row = lane % 16 * a.pitch, col = lane / 16 * 16;
  i32x4 acc[NT][MT];
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int i = 0; i < MT; ++i) acc[j][i] = i32x4{0, 0, 0, 0};
  for (int k = wave * (U * 64); k < a.pitch; k += kFewWaves * U * 64) {
    i32x4 fw[U][NT], fx[U][MT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      // past the pitch lies the next row: those chunks are zeros
      const int c = k + u * 64 + col, at = c < a.pitch ? row + c : kPastEnd;
#pragma unroll
      for (int j = 0; j < NT; ++j)
        fw[u][j] = __builtin_bit_cast(
            i32x4, __builtin_amdgcn_raw_buffer_load_b128(w, at, j * 16 * a.pitch, 0));
#pragma unroll
      for (int i = 0; i < MT; ++i)
        fx[u][i] = __builtin_bit_cast(
            i32x4, __builtin_amdgcn_raw_buffer_load_b128(x, at + i * 16 * a.pitch, 0, 0));
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < MT; ++i)
          acc[j][i] =
              __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[u][j], fx[u][i], acc[j][i], 0, 0, 0);
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
        *reinterpret_cast<i32x4*>(&sums[wave - HALF][at(j, i)]) = acc[j][i];
  }
  __syncthreads();
  if (wave < HALF) {
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        i32x4* p = reinterpret_cast<i32x4*>(&sums[wave][at(j, i)]);
        *p += acc[j][i];
      }
  }
  __syncthreads();
  for (int e = (int)threadIdx.x * 4; e < E; e += kFewWaves * 64 * 4) {
    const int64_t m = m0 + e / (16 * NT);
    const int n = n0 + e % (16 * NT);
    if (m >= a.rows || n >= a.out) continue;
    i32x4 s = *reinterpret_cast<const i32x4*>(&sums[0][e]);
#pragma unroll
    for (int v = 1; v < HALF; ++v) s += *reinterpret_cast<const i32x4*>(&sums[v][e]);
    const float step = a.steps[m];
    T o[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int c = min(n + r, a.out - 1);
      o[r] = (T)((float)s[r] * step * a.w_steps[c] + (a.bias ? a.bias[c] : 0.f));
    }
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

// Which of the two: each workgroup above reads the codes of all its tokens (up
// to 32) from L2 for 16 or 32 outputs, the tiled kernel once for 64.  That is
// little beside the weight up to 4 tokens; from there on what one CU reads so
// decides.  Measured (us here / there, bf16, tokens x out x cols; the product
// compared below behind it):
//   16 x 8192 x 8192 17.5 / 21.5 (32)    17 x 8192 x 8192  18.9 / 21.7 (34)
//   64 x 4096 x 4096 10.3 / 12.7 (32)     8 x 20000 x 8192 40.1 / 36.3 (40)
//   16 x 9216 x 8192 24.2 / 21.8 (48)    12 x 16384 x 8192 30.1 / 23.2 (48)
//   32 x 4608 x 8192 23.8 / 21.5 (64)    64 x 16384 x 8192 79.8 / 25.7 (128)
//    4 x 50000 x 4096 42.8 / 47.4         1 x 16384 x 8192 24.1 / 22.8
// Past 64 tokens the tiled kernel: 65 x 4096 x 4096 15.0 / 12.8.
bool few_tokens(const ActDims& A, int64_t out) {
  if (A.rows <= 4 || A.rows > 64) return A.rows <= 4;
  const int groups = A.rows <= 32 ? div_up(out, 16) : 2 * div_up(out, 32);
  return div_up(groups, kCus) * (A.rows < 32 ? A.rows : 32) < 48;
}

template <typename T, int MT, int NT, int U>
void few(const LinearArgs& a, hipStream_t st) {
  const dim3 g(div_up(a.out, 16 * NT), div_up(a.rows, 16 * MT));
  k_act_linear_few<T, MT, NT, U><<<g, kFewWaves * 64, 0, st>>>(a);
}

struct Plan {
  int splits, per;  // of the sum, and 128-byte k-tiles of one
  int tile;         // rows and columns of a tile
};

// The tile's side and the number of splits by an estimate of the time in
// microseconds: rounds of tiles over the chip, their k-tiles, what a tile costs
// besides, and the splits' sums through memory.  Measured (tokens x out x
// cols): 4096 x 4096 x 4096 62 us with 256-tiles, 82 with 128; 1024 x 4096 x
// 4096 25 us with 128-tiles, 34 with 64, 43 with 256; 512 x 4096 x 4096 17.1 us
// with 64, 18.8 with 128; splits only pay for long sums on few tiles (8192 x 512
// x 8192: 42 us unsplit, 73 with two; 512 x 512 x 32768: 73 unsplit, 44 with two,
// 25 with as many as are taken).
Plan plan_linear(const ActDims& A, int64_t out) {
  const int kt = div_up(A.pitch, 128);
  Plan best = {1, kt, 0};
  if (few_tokens(A, out)) return best;
  double least = 1e30;
  for (int tile = 64; tile <= 256; tile *= 2) {
    const int64_t tiles = ((A.rows + tile - 1) / tile) * ((out + tile - 1) / tile);
    // up to 64 tokens unsplit: their products need no workspace
    for (int s = 1; s <= 8 && (s == 1 || (A.rows > 64 && kt / s >= 8)); ++s) {
      const int per = div_up(kt, s);
      const int64_t groups = tiles * s;
      const double rounds = (double)((groups + kCus - 1) / kCus);
      double t;
      if (tile == 256) t = rounds * (per * 1.6 + 12.0);
      else if (tile == 128) t = rounds * (per * 0.6 + 5.0);
      else if (groups <= kCus) t = per * 0.33 + 4.0;
      else t = (double)((groups + 2 * kCus - 1) / (2 * kCus)) * (per * 0.44 + 4.0);
      if (s > 1) t += 10.0 + 8.0 * (double)(s * A.rows) * (double)out / 2.4e6;
      if (t < least) {
        least = t;
        best = {div_up(kt, per), per, tile};
      }
    }
  }
  return best;
}

template <typename T>
int linear_t(const ActDims& A, LinearArgs a, int tile, hipStream_t st) {
  if (few_tokens(A, a.out)) {
    if (A.rows <= 16) few<T, 1, 1, 8>(a, st);
    else if (A.rows <= 32) few<T, 2, 1, 4>(a, st);
    else few<T, 2, 2, 4>(a, st);
    return (int)hipGetLastError();
  }
  a.mtiles = div_up(A.rows, tile);
  a.ntiles = div_up(a.out, tile);
  const int64_t tiles = (int64_t)a.mtiles * a.ntiles * a.splits;
  const int64_t most = tile == 64 ? 2 * kCus : kCus;  // what the chip holds
  const unsigned g = (unsigned)(tiles < most ? tiles : most);
  if (tile == 256) k_act_linear<T, 256, 256, 128, 64, 128, 2><<<g, 512, 0, st>>>(a);
  else if (tile == 128) k_act_linear<T, 128, 128, 64, 32, 128, 4><<<g, 512, 0, st>>>(a);
  else k_act_linear<T, 64, 64, 32, 32, 128, 4><<<g, 256, 0, st>>>(a);
  int rc = (int)hipGetLastError();
  if (rc == 0 && a.splits > 1) {
    const int64_t b = (A.rows * a.out + 255) / 256;
    k_act_linear_join<T><<<(unsigned)(b < 4096 ? b : 4096), 256, 0, st>>>(a);
    rc = (int)hipGetLastError();
  }
  return rc;
}

}  // namespace

int64_t act_linear_workspace(const ActDims& A, int64_t out) {
  if (A.rows == 0) return 0;
  const Plan p = plan_linear(A, out);
  return p.splits > 1 ? 4 * p.splits * A.rows * out : 0;
}

int launch_act_linear(const ActDims& A, int64_t out, const int8_t* codes,
                      const float* steps, const int8_t* w_codes,
                      const float* w_steps, const float* bias, void* y,
                      int64_t ldy, void* ws, hipStream_t st) {
  if (A.rows == 0) return 0;
  const Plan p = plan_linear(A, out);
  const LinearArgs a = {A.rows,  (int)out, (int)A.pitch, codes, w_codes,  steps,   w_steps,
                        bias,    y,        ldy,          (int32_t*)ws, p.splits, p.per, 0, 0};
  switch (A.dtype) {
    case GQ_F32: return linear_t<float>(A, a, p.tile, st);
    case GQ_BF16: return linear_t<__bf16>(A, a, p.tile, st);
    default: return linear_t<_Float16>(A, a, p.tile, st);
  }
}

}  // namespace gq
