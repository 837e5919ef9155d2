// act_pack.hip — activations to and from their 8-bit form (act.hpp).
//
// Both directions are one pass over HBM: pack reads e bytes and writes 1
// (+ 4/group) per value, unpack the reverse.  A thread owns eight consecutive
// columns (16 bytes of bf16), so a wave's access is contiguous; a group of up
// to 512 columns lies in 4..64 neighbouring lanes and needs only lane
// exchanges, a longer one goes through LDS.
#include "act.hpp"

namespace gq {
namespace {

constexpr int kBlock = 256;

// Groups of G * 8 columns, G = 4..64 lanes.  tpr threads per row (a power of
// two); cpr: chunks of a row rounded up to whole groups.
template <typename T>
__global__ __launch_bounds__(kBlock) void k_act_pack_lanes(
    int64_t rows, int cols, int pitch, int groups, int G, int cpr, int tpr,
    const T* __restrict__ x, int64_t ldx, int8_t* __restrict__ codes,
    float* __restrict__ steps) {
  const int per = kBlock / tpr, lane = (int)threadIdx.x & (tpr - 1);
  for (int64_t r0 = (int64_t)blockIdx.x * per; r0 < rows;
       r0 += (int64_t)gridDim.x * per) {
    const int64_t row = r0 + (int)threadIdx.x / tpr;
    const bool live = row < rows;
    const T* xr = x + (live ? row : 0) * ldx;
    for (int c0 = 0; c0 < cpr; c0 += tpr) {
      const int c = c0 + lane;
      const int valid = live ? cols - c * 8 : 0;
      float f[8];
      widen(load8(xr + c * 8, valid), f);
      const Step s = step_of<T>(lanes_max(max_abs_bits(f), G));
      if (!live) continue;
      if (c * 8 < pitch)
        *reinterpret_cast<uint2*>(codes + row * pitch + c * 8) = codes8(f, s);
      const int grp = c / G;
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
template <typename T, int NT, int R>
__global__ __launch_bounds__(NT < 256 ? 256 : NT) void k_act_pack_seg(
    int64_t rows, int cols, int pitch, int groups, int group,
    const T* __restrict__ x, int64_t ldx, int8_t* __restrict__ codes,
    float* __restrict__ steps) {
  __shared__ uint32_t red[16];
  constexpr int BT = NT < 256 ? 256 : NT;
  constexpr int PER = BT / NT;
  const int lane = (int)threadIdx.x % NT;
  const int64_t total = rows * groups;
  for (int64_t s0 = (int64_t)blockIdx.x * PER + threadIdx.x / NT; s0 < total;
       s0 += (int64_t)gridDim.x * PER) {
    const int64_t row = groups == 1 ? s0 : s0 / groups;
    const int grp = (int)(s0 - row * groups);
    const int lo = grp * group;
    const int n = min(group, cols - lo);  // columns of this group
    // codes up to the pitch belong to the row's last group
    const int cn = grp == groups - 1 ? pitch - lo : n;
    const T* xr = x + row * ldx + lo;
    int8_t* cr = codes + row * pitch + lo;
    uint32_t m = 0;
    if constexpr (R > 0) {
      float f[R][8];
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const int c = (lane + i * NT) * 8;
        widen(load8(xr + c, n - c), f[i]);
        m = max(m, max_abs_bits(f[i]));
      }
      const Step s = step_of<T>(block_max<NT>(m, red));
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const int c = (lane + i * NT) * 8;
        if (c < cn) *reinterpret_cast<uint2*>(cr + c) = codes8(f[i], s);
      }
      if (lane == 0) steps[s0] = s.step;
    } else {
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
      if (lane == 0) steps[s0] = s.step;
    }
  }
}

template <typename T>
__global__ __launch_bounds__(kBlock) void k_act_unpack(
    int64_t rows, int cols, int pitch, int groups, int glog, int tpr,
    const int8_t* __restrict__ codes, const float* __restrict__ steps,
    T* __restrict__ x, int64_t ldx) {
  const int per = kBlock / tpr, lane = (int)threadIdx.x & (tpr - 1);
  for (int64_t row = (int64_t)blockIdx.x * per + (int)threadIdx.x / tpr; row < rows;
       row += (int64_t)gridDim.x * per) {
    const int8_t* cr = codes + row * pitch;
    const float* sr = steps + row * groups;
    T* xr = x + row * ldx;
    for (int c = lane * 8; c < cols; c += tpr * 8) {
      const uint2 w = *reinterpret_cast<const uint2*>(cr + c);
      float f[8];
      decode8(w, sr[c >> glog], f);
      store8(xr + c, narrow<T>(f), cols - c);
    }
  }
}

int pow2_up(int v) {
  int p = 1;
  while (p < v) p *= 2;
  return p;
}

// Workgroups over `n` items of which each takes `per`: enough to fill the
// chip many times, the rest by stride.
unsigned blocks_for(int64_t n, int per) {
  const int64_t b = (n + per - 1) / per;
  return (unsigned)(b < (1 << 20) ? b : (1 << 20));
}

template <typename T, int NT, int R>
void pack_seg(const ActDims& A, const T* x, int64_t ldx, int8_t* codes,
              float* steps, hipStream_t st) {
  constexpr int BT = NT < 256 ? 256 : NT;
  k_act_pack_seg<T, NT, R><<<blocks_for(A.rows * A.groups, BT / NT), BT, 0, st>>>(
      A.rows, (int)A.cols, (int)A.pitch, A.groups, A.group, x, ldx, codes, steps);
}

template <typename T>
int pack_t(const ActDims& A, const T* x, int64_t ldx, int8_t* codes, float* steps,
           hipStream_t st) {
  if (!A.whole_row && A.group <= 512) {
    const int G = A.group / 8;
    const int cpr = div_up(div_up(A.cols, 8), G) * G;
    const int tpr = cpr < kBlock ? pow2_up(cpr) : kBlock;
    k_act_pack_lanes<T><<<blocks_for(A.rows, kBlock / tpr), kBlock, 0, st>>>(
        A.rows, (int)A.cols, (int)A.pitch, A.groups, G, cpr, tpr, x, ldx, codes,
        steps);
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
  const int n8 = div_up(A.cols, 8);
  const int tpr = n8 < kBlock ? pow2_up(n8) : kBlock;
  int glog = 31;  // one step per row: index 0
  if (!A.whole_row)
    for (glog = 0; (1 << glog) < A.group;) ++glog;
  k_act_unpack<T><<<blocks_for(A.rows, kBlock / tpr), kBlock, 0, st>>>(
      A.rows, (int)A.cols, (int)A.pitch, A.groups, glog, tpr, codes, steps, x, ldx);
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
