// act_pack.hip — activations to and from their 8-bit form (act.hpp).
//
// Both directions are one pass over HBM: pack reads e bytes and writes 1
// (+ 4/group) per value, unpack the reverse.  A thread owns eight consecutive
// columns (16 bytes of bf16), so a wave's access is contiguous; a group of up
// to 512 columns lies in 4..64 neighbouring lanes and needs only lane
// exchanges, a longer one goes through LDS.  16384 x 4096 bf16 with a step per
// 128 columns: pack 44 us, 4.6 TB/s (a large copy's rate is 5.1; its input
// comes from HBM), unpack 30 us, 6.8 TB/s (its codes from the last-level
// cache; 38 without); 8192 x 4096 with a step per row: 24 us.  Groups over
// 16384 columns are read twice: 1024 x 40000 with a step per row 36 us, 24 with
// one per 128 columns.
#include "act.hpp"
#include "act_bounds.hpp"

namespace gq {
namespace {

constexpr int kBlock = kCoverThreads;

// A unit is what a workgroup takes at once: kBlock / tpr rows by tpr chunks
// (tpr a power of two, `turns` units side by side cover the rows).  Each
// workgroup takes one to pack and two consecutive ones to unpack, all loads
// first (16384 x 4096 bf16, one / two / four units: pack 44.5 / 48 / 53 us,
// unpack 32 / 30 / 30; 16 x 1024: 2.6 / 2.6 / 3.3 and 2.5 / 2.3 / 2.4).
constexpr int kPackUnits = 1, kUnpackUnits = 2;

struct Unit {
  int64_t rows0;  // row group
  int turn;
};

template <int UNITS>
__device__ __forceinline__ Unit first_unit(int turns) {
  const int64_t u = (int64_t)blockIdx.x * UNITS;
  Unit r;
  // 32-bit division where it is enough: one per workgroup
  r.rows0 = u >> 32 ? u / turns : (uint32_t)u / (uint32_t)turns;
  r.turn = (int)(u - r.rows0 * turns);
  return r;
}

__device__ __forceinline__ void next_unit(Unit* u, int turns) {
  if (++u->turn == turns) {
    u->turn = 0;
    ++u->rows0;
  }
}

// Groups of G * 8 columns, G = 4..64 lanes.
template <typename T, int END>
__global__ __launch_bounds__(kBlock) void k_act_pack_lanes(
    int64_t rows, int cols, int pitch, int groups, int Glog, int turns, int tlog,
    const T* __restrict__ x, int64_t ldx, int8_t* __restrict__ codes,
    float* __restrict__ steps) {
  const int tpr = 1 << tlog, per = kBlock >> tlog, G = 1 << Glog;
  const int lane = (int)threadIdx.x & (tpr - 1), in = (int)threadIdx.x >> tlog;
  constexpr int UNITS = kPackUnits;
  Raw8<T> raw[UNITS];
  Unit u = first_unit<UNITS>(turns), v = u;
#pragma unroll
  for (int i = 0; i < UNITS; ++i, next_unit(&u, turns)) {
    const int64_t row = u.rows0 * per + in;
    const int c = (u.turn * tpr + lane) * 8;
    raw[i] = load_chunk<END>(x + row * ldx, c, row < rows ? cols : 0);
  }
#pragma unroll
  for (int i = 0; i < UNITS; ++i, next_unit(&v, turns)) {
    const int64_t row = v.rows0 * per + in;
    const int c = v.turn * tpr + lane;
    float f[8];
    settle<END>(raw[i], c * 8, row < rows ? cols : 0);
    widen(raw[i], f);
    const Step s = step_of<T>(lanes_max(max_abs_bits(f), G));
    if (row < rows) {
      if (c * 8 < pitch)
        *reinterpret_cast<uint2*>(codes + row * pitch + c * 8) = codes8(f, s);
      const int grp = c >> Glog;
      if ((c & (G - 1)) == 0 && grp < groups) steps[row * groups + grp] = s.step;
    }
  }
}

// The largest value over a workgroup's NT threads (in all of them).
template <int NT>
__device__ __forceinline__ uint32_t block_max(uint32_t m, uint32_t* red) {
  m = lanes_max(m, 64);
  if constexpr (NT > 64) {
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NT / 64; ++i) m = max(m, red[i]);
  }
  return m;
}

// One group (a whole row, or 1024 columns and more) per NT threads: R chunks
// of each thread stay in registers; R = 0 reads the group twice.
template <typename T, int NT, int R, int END>
__global__ __launch_bounds__(NT < 256 ? 256 : NT) void k_act_pack_seg(
    int64_t rows, int cols, int pitch, int groups, int group,
    const T* __restrict__ x, int64_t ldx, int8_t* __restrict__ codes,
    float* __restrict__ steps) {
  __shared__ uint32_t red[16];
  constexpr int BT = NT < 256 ? 256 : NT;
  constexpr int PER = BT / NT;
  const int lane = (int)threadIdx.x % NT;
  const int64_t total = rows * groups, stride = (int64_t)gridDim.x * PER;
  int64_t at = (int64_t)blockIdx.x * PER + threadIdx.x / NT;
  Raw8<T> raw[R > 0 ? R : 1];
  auto fetch = [&](int64_t s) {
    const int64_t row = groups == 1 ? s : s / groups;
    const int lo = (int)(s - row * groups) * group, n = min(group, cols - lo);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int c = (lane + i * NT) * 8;
      raw[i] = load_chunk<END>(x + row * ldx, lo + c, s < total ? lo + n : 0);
    }
  };
  if constexpr (R > 0) fetch(at);
  for (; at < total; at += stride) {
    const int64_t row = groups == 1 ? at : at / groups;
    const int grp = (int)(at - row * groups);
    const int lo = grp * group;
    const int n = min(group, cols - lo);  // columns of this group
    // codes up to the pitch belong to the row's last group
    const int cn = grp == groups - 1 ? pitch - lo : n;
    int8_t* cr = codes + row * pitch + lo;
    uint32_t m = 0;
    if constexpr (R > 0) {
      float f[R][8];
#pragma unroll
      for (int i = 0; i < R; ++i) {
        settle<END>(raw[i], lo + (lane + i * NT) * 8, lo + n);
        widen(raw[i], f[i]);
        m = max(m, max_abs_bits(f[i]));
      }
      fetch(at + stride);
      const Step s = step_of<T>(block_max<NT>(m, red));
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const int c = (lane + i * NT) * 8;
        if (c < cn) *reinterpret_cast<uint2*>(cr + c) = codes8(f[i], s);
      }
      if (lane == 0) steps[at] = s.step;
    } else {
      const T* xr = x + row * ldx + lo;
      float f[8];
      for (int c = lane * 8; c < n; c += NT * 8) {
        widen(load8(xr + c, n - c), f);
        m = max(m, max_abs_bits(f));
      }
      const Step s = step_of<T>(block_max<NT>(m, red));
      for (int c = lane * 8; c < cn; c += NT * 8) {
        widen(load8(xr + c, n - c), f);
        *reinterpret_cast<uint2*>(cr + c) = codes8(f, s);
      }
      if (lane == 0) steps[at] = s.step;
    }
  }
}

template <typename T, int END>
__global__ __launch_bounds__(kBlock) void k_act_unpack(
    int64_t rows, int cols, int pitch, int groups, int glog, int turns, int tlog,
    const int8_t* __restrict__ codes, const float* __restrict__ steps,
    T* __restrict__ x, int64_t ldx) {
  const int tpr = 1 << tlog, per = kBlock >> tlog;
  const int lane = (int)threadIdx.x & (tpr - 1), in = (int)threadIdx.x >> tlog;
  constexpr int UNITS = kUnpackUnits;
  uint2 w[UNITS];
  float s[UNITS];
  Unit u = first_unit<UNITS>(turns), v = u;
#pragma unroll
  for (int i = 0; i < UNITS; ++i, next_unit(&u, turns)) {
    const int64_t row = u.rows0 * per + in;
    const int c = (u.turn * tpr + lane) * 8;
    w[i] = make_uint2(0, 0);
    s[i] = 0.f;
    if (row < rows && c < cols) {
      w[i] = *reinterpret_cast<const uint2*>(codes + row * pitch + c);
      s[i] = steps[row * groups + (c >> glog)];
    }
  }
#pragma unroll
  for (int i = 0; i < UNITS; ++i, next_unit(&v, turns)) {
    const int64_t row = v.rows0 * per + in;
    const int c = (v.turn * tpr + lane) * 8;
    float f[8];
    decode8(w[i], s[i], f);
    store_chunk<END>(x + row * ldx + c, narrow<T>(f), row < rows ? cols - c : 0);
  }
}

// Workgroups over `n` items of which each takes `per` at a time, the rest by
// stride.
unsigned blocks_for(int64_t n, int per, int most) {
  const int64_t b = (n + per - 1) / per;
  return (unsigned)(b < most ? b : most);
}

template <typename T, int NT, int R>
void pack_seg(const ActDims& A, const T* x, int64_t ldx, int8_t* codes,
              float* steps, hipStream_t st) {
  constexpr int BT = NT < 256 ? 256 : NT;
  // resident workgroups, each thread with the next group on its way
  const unsigned g = blocks_for(A.rows * A.groups, BT / NT, kCus * (2048 / BT));
  auto* k = A.cols % 8 ? k_act_pack_seg<T, NT, R, kRagged> : k_act_pack_seg<T, NT, R, kWhole>;
  if constexpr (NT == 64 && R == 1)
    if (row_end(A.cols) == kTiny) k = k_act_pack_seg<T, NT, R, kTiny>;
  k<<<g, BT, 0, st>>>(
      A.rows, (int)A.cols, (int)A.pitch, A.groups, A.group, x, ldx, codes, steps);
}

template <typename T>
int pack_t(const ActDims& A, const T* x, int64_t ldx, int8_t* codes, float* steps,
           hipStream_t st) {
  if (!A.whole_row && A.group <= 512) {
    const int G = group_lanes(A.group, A.pitch);
    // whole groups in each unit
    const Cover c(div_up(div_up(A.cols, 8), G) * G, kPackUnits);
    const RowEnd end = row_end(A.cols);
    auto* k = end == kWhole    ? k_act_pack_lanes<T, kWhole>
              : end == kRagged ? k_act_pack_lanes<T, kRagged>
                               : k_act_pack_lanes<T, kTiny>;
    for (int64_t r = 0; r < A.rows; r += c.rows) {
      const int64_t n = A.rows - r < c.rows ? A.rows - r : c.rows;
      k<<<(unsigned)c.blocks(n), kBlock, 0, st>>>(
          n, (int)A.cols, (int)A.pitch, A.groups, log2_up(G), c.turns, c.tlog, x + r * ldx, ldx,
          codes + r * A.pitch, steps + r * A.groups);
    }
  } else {
    // pitch, not cols: padding codes are written by the group's threads too
    const int n8 = (int)(A.group < A.pitch ? A.group : A.pitch) / 8;
    if (n8 <= 64) pack_seg<T, 64, 1>(A, x, ldx, codes, steps, st);
    else if (n8 <= 128) pack_seg<T, 64, 2>(A, x, ldx, codes, steps, st);
    else if (n8 <= 256) pack_seg<T, 256, 1>(A, x, ldx, codes, steps, st);
    else if (n8 <= 512) pack_seg<T, 256, 2>(A, x, ldx, codes, steps, st);
    else if (n8 <= 1024) pack_seg<T, 1024, 1>(A, x, ldx, codes, steps, st);
    else if (n8 <= 2048) pack_seg<T, 1024, 2>(A, x, ldx, codes, steps, st);
    else pack_seg<T, 1024, 0>(A, x, ldx, codes, steps, st);
  }
  return (int)hipGetLastError();
}

template <typename T>
int unpack_t(const ActDims& A, const int8_t* codes, const float* steps, T* x,
             int64_t ldx, hipStream_t st) {
  const Cover c(div_up(A.cols, 8), kUnpackUnits);
  int glog = 31;  // one step per row: index 0
  if (!A.whole_row) glog = log2_up(A.group);
  auto* k = A.cols % 8 ? k_act_unpack<T, kRagged> : k_act_unpack<T, kWhole>;
  for (int64_t r = 0; r < A.rows; r += c.rows) {
    const int64_t n = A.rows - r < c.rows ? A.rows - r : c.rows;
    k<<<(unsigned)c.blocks(n), kBlock, 0, st>>>(
        n, (int)A.cols, (int)A.pitch, A.groups, glog, c.turns, c.tlog, codes + r * A.pitch,
        steps + r * A.groups, x + r * ldx, ldx);
  }
  return (int)hipGetLastError();
}

}  // namespace

int launch_act_pack(const ActDims& A, const void* x, int64_t ldx, int8_t* codes,
                    float* steps, hipStream_t st) {
  if (A.rows == 0) return 0;
  switch (A.dtype) {
    case GQ_F32: return pack_t(A, (const float*)x, ldx, codes, steps, st);
    case GQ_BF16: return pack_t(A, (const __bf16*)x, ldx, codes, steps, st);
    default: return pack_t(A, (const _Float16*)x, ldx, codes, steps, st);
  }
}

int launch_act_unpack(const ActDims& A, const int8_t* codes, const float* steps,
                      void* x, int64_t ldx, hipStream_t st) {
  if (A.rows == 0) return 0;
  switch (A.dtype) {
    case GQ_F32: return unpack_t(A, codes, steps, (float*)x, ldx, st);
    case GQ_BF16: return unpack_t(A, codes, steps, (__bf16*)x, ldx, st);
    default: return unpack_t(A, codes, steps, (_Float16*)x, ldx, st);
  }
}

}  // namespace gq
