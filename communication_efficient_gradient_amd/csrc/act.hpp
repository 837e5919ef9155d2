// act.hpp — the 8-bit activation form shared by act_pack, layer_norm,
// act_linear and act_wgrad, and their launchers.
//
// A matrix [rows, cols] of activations is kept as int8 codes [rows][pitch]
// (pitch = cols rounded up to 16, padding codes 0) and one fp32 step per
// group of columns of a row; x^ = code * step.  A step is a power of two, so
// x^ (7 significant bits) is exact in bf16 and in fp32 and every product with
// a bf16 value is exact in an fp32 accumulator: a weight gradient from the
// codes needs one matrix instruction per tile and rounds nothing on the way
// in.  Against a free fp32 step this costs up to one of the 8 bits.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "act_bounds.hpp"
#include "common.hpp"

namespace gq {

struct ActDims {
  int64_t rows, cols, pitch;
  int dtype;       // gq_dtype
  int group;       // columns per step (pitch when there is one per row)
  int groups;      // steps per row
  bool whole_row;  // desc group 0
};

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));

// ------------------------------------------------ eight columns at a time --
// Eight consecutive values of a row.  16-byte accesses need no alignment
// beyond the element's on gfx950 (unaligned global accesses are on), so odd
// strides and views take the same path; only a row's last, short chunk is
// read by elements.
template <typename T>
struct Raw8 {
  T v[8];
};

template <typename T>
__device__ __forceinline__ Raw8<T> load8(const T* __restrict__ p, int valid) {
  Raw8<T> r;
  if (valid >= 8) {
    __builtin_memcpy(&r, p, sizeof(r));
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) r.v[j] = j < valid ? p[j] : T(0);
  }
  return r;
}

template <typename T>
__device__ __forceinline__ void store8(T* __restrict__ p, const Raw8<T>& r, int valid) {
  if (valid >= 8) {
    __builtin_memcpy(p, &r, sizeof(r));
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < valid) p[j] = r.v[j];
  }
}

// Moves the values down by `n` places (0 .. 7) and clears what is left.
template <typename T>
__device__ __forceinline__ void shift_down(Raw8<T>& r, int n) {
  if constexpr (sizeof(T) == 2) {
    unsigned __int128 w;
    __builtin_memcpy(&w, &r, 16);
    w >>= n * 16;
    __builtin_memcpy(&r, &w, 16);
  } else {
#pragma unroll
    for (int s = 4; s > 0; s /= 2)
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (n & s) r.v[j] = j + s < 8 ? r.v[j + s] : T(0);
  }
}

// How a row ends.  kWhole: cols % 8 == 0, a chunk is the row's or past its end
// as a whole.  kRagged: the last chunk is short.  It is fetched as the row's
// last eight values, in the same instruction as the other lanes' chunks, and
// settle() moves it down where it is used.  kTiny: fewer than eight columns,
// read by elements.  A way through elements, or moving the values where they
// are loaded, makes loads of the wave wait for those before (backward pass of
// 1531 x 1001 fp16: 8.9 us with both in the kernel, 7.8 so; layer norm of 16384
// x 4096 bf16 with its input's 8-bit form: 93 us through elements, 62 with whole
// chunks).
enum RowEnd { kWhole = 0, kRagged = 1, kTiny = 2 };

inline RowEnd row_end(int64_t cols) {
  return cols % 8 == 0 ? kWhole : cols >= 8 ? kRagged : kTiny;
}

// Columns c .. c + 7 of a row that ends before column `end`; what lies past it
// is 0 (kRagged: once settled).
template <int END, typename T>
__device__ __forceinline__ Raw8<T> load_chunk(const T* __restrict__ row, int c, int end) {
  Raw8<T> r = {};
  const int valid = end - c;
  if constexpr (END == kWhole) {
    if (valid > 0) __builtin_memcpy(&r, row + c, sizeof(r));
  } else if constexpr (END == kRagged) {
    if (valid > 0) __builtin_memcpy(&r, row + min(c, end - 8), sizeof(r));
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < valid) r.v[j] = row[c + j];
  }
  return r;
}

template <int END, typename T>
__device__ __forceinline__ void settle(Raw8<T>& r, int c, int end) {
  const int valid = end - c;
  if (END == kRagged && valid > 0 && valid < 8) shift_down(r, 8 - valid);
}

template <int END, typename T>
__device__ __forceinline__ void store_chunk(T* p, const Raw8<T>& r, int valid) {
  if (END != kWhole) return store8(p, r, valid);
  if (valid > 0) __builtin_memcpy(p, &r, sizeof(r));
}

template <typename T>
__device__ __forceinline__ void widen(const Raw8<T>& r, float (&f)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = (float)r.v[j];
}

template <typename T>
__device__ __forceinline__ Raw8<T> narrow(const float (&f)[8]) {
  Raw8<T> r;
#pragma unroll
  for (int j = 0; j < 8; ++j) r.v[j] = (T)f[j];  // nearest, ties to even
  return r;
}

// ------------------------------------------------------------------ steps --
// Bits of |x|: as unsigned integers finite values, infinity and NaN are in
// ascending order, so one integer maximum carries both the largest magnitude
// and the presence of a value that is not finite.
__device__ __forceinline__ uint32_t abs_bits(float x) {
  return __float_as_uint(x) & 0x7fffffffu;
}

__device__ __forceinline__ uint32_t max_abs_bits(const float (&f)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = max(m, abs_bits(f[j]));
  return m;
}

// Largest step of a type, as a biased exponent: 127 * step stays finite in
// it (2^9 for fp16, 2^121 for bf16 and fp32); codes saturate at 127 there.
template <typename T>
constexpr uint32_t kMaxStepExp = 121 + 127;
template <>
inline constexpr uint32_t kMaxStepExp<_Float16> = 9 + 127;

// The smallest power of two with 127 * step >= M (M as abs_bits), at least
// 2^-126: 0 for M = 0, NaN if M is not finite.  inv = 1 / step, or 0 where
// all codes are 0.
struct Step {
  float step, inv;
};

template <typename T>
__device__ __forceinline__ Step step_of(uint32_t m) {
  const uint32_t ex = m >> 23, frac = m & 0x7fffffu;
  // M = 1.frac 2^ex; 127 = 1.984375 2^6
  uint32_t s = ex > 6 ? ex - 6 + (frac > 0x7e0000u ? 1u : 0u) : 1u;
  s = min(max(s, 1u), kMaxStepExp<T>);
  Step r;
  r.step = __uint_as_float(s << 23);
  r.inv = __uint_as_float((254u - s) << 23);
  if (m == 0) r.step = r.inv = 0.f;
  if (ex == 255) {
    r.step = __uint_as_float(0x7fc00000u);
    r.inv = 0.f;
  }
  return r;
}

// Eight codes round(x / step), ties to even, saturating at 127, as bytes.
// The product with a power of two is exact, so there is one rounding; adding
// 1.5 * 2^23 leaves the rounded integer in the low mantissa bits.
__device__ __forceinline__ uint2 codes8(const float (&f)[8], const Step& s) {
  uint32_t b[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float q = __builtin_amdgcn_fmed3f(f[j] * s.inv, -127.f, 127.f);
    b[j] = __float_as_uint(q + 12582912.f);
  }
  uint2 r;
  // bytes 0 of four words: perm selects from (first << 32 | second)
  const uint32_t l01 = __builtin_amdgcn_perm(b[1], b[0], 0x0c0c0400u);
  const uint32_t l23 = __builtin_amdgcn_perm(b[3], b[2], 0x04000c0cu);
  const uint32_t h01 = __builtin_amdgcn_perm(b[5], b[4], 0x0c0c0400u);
  const uint32_t h23 = __builtin_amdgcn_perm(b[7], b[6], 0x04000c0cu);
  r.x = l01 | l23;
  r.y = h01 | h23;
  if (s.inv == 0.f) r.x = r.y = 0;  // 0 * inf and 0 * NaN are not 0
  return r;
}

// x^ of four codes, -128 .. 127: each byte converts with its sign in one
// instruction, and the product with a power of two is exact (it overflows only
// for -128 at the largest step, whose x^ no type holds).
__device__ __forceinline__ void decode4(uint32_t w, float step, float* f) {
  f[0] = (float)(int8_t)w * step;
  f[1] = (float)(int8_t)(w >> 8) * step;
  f[2] = (float)(int8_t)(w >> 16) * step;
  f[3] = (float)((int32_t)w >> 24) * step;
}

__device__ __forceinline__ void decode8(uint2 w, float step, float (&f)[8]) {
  decode4(w.x, step, f);
  decode4(w.y, step, f + 4);
}

// The largest value over aligned groups of G lanes, G from 4 to 64.
__device__ __forceinline__ uint32_t lanes_max(uint32_t m, int G) {
  m = max(m, xshfl(m, 1));
  m = max(m, xshfl(m, 2));
  if (G > 4) m = max(m, xshfl(m, 4));
  if (G > 8) m = max(m, xshfl(m, 8));
  if (G > 16) m = max(m, xshfl(m, 16));
  if (G > 32) m = max(m, xshfl(m, 32));
  return m;
}

// ------------------------------------------------- global memory to LDS --
// A range of global memory that reads as zeros past its end (ranges of 4 GiB
// and more are cut there; a length below zero is none).  The accesses below are
// buffer instructions: the bounds are checked by the load itself, on the sum of
// its offsets, the scalar one included, and unlike the global form they do
// not make the compiler drain all LDS reads in flight before it uses one.
typedef __amdgpu_buffer_rsrc_t BufferRange;

__device__ __forceinline__ BufferRange range_of(const void* base, int64_t bytes) {
  const uint32_t n = (uint32_t)min(max(bytes, (int64_t)0), (int64_t)0xffffffff);
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, n, 0x00020000);
}

// An offset behind the end of any range below 2 GiB.
constexpr int kPastEnd = (int)0x80000000;

// 16 bytes per lane into LDS at `to` (the same in all lanes) + 16 * lane,
// without passing through registers; `each` differs by lane, `all` does not.
__device__ __forceinline__ void copy16_to_lds(
    BufferRange from, int each, int all, __attribute__((address_space(3))) void* to) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(from, to, 16, each, all, 0, 0);
}

// Tiles (i, j) of i_tiles x j_tiles, for each split of the sum, as a
// one-dimensional grid takes them.  Workgroups go round the eight XCDs in turn,
// so each XCD gets a run of the splits' tiles one after the other, and within a
// split takes columns of up to eight tiles i: what its L2 holds is used by
// many of its workgroups.  A grid smaller than the number of tiles walks its
// XCD's run.
struct Tile {
  int i, j, split;
};

struct TileWalk {
  int i_tiles, j_tiles, next, end, stride;

  __device__ __forceinline__ TileWalk(int i_tiles, int j_tiles, int splits)
      : i_tiles(i_tiles), j_tiles(j_tiles) {
    const int total = i_tiles * j_tiles * splits, xcd = (int)blockIdx.x % 8;
    const int per = total / 8, more = total % 8, first = xcd * per + min(xcd, more);
    next = first + (int)blockIdx.x / 8;
    end = first + per + (xcd < more ? 1 : 0);
    stride = ((int)gridDim.x + 7) / 8;
  }

  // Whether there is one; it is taken.
  __device__ __forceinline__ bool take(Tile* t) {
    if (next >= end) return false;
    const int tiles = i_tiles * j_tiles;
    t->split = next / tiles;
    const int in = next - t->split * tiles;
    const int first = in / (8 * j_tiles) * 8, h = min(8, i_tiles - first);
    const int k = in - first * j_tiles;
    t->i = first + k % h;
    t->j = k / h;
    next += stride;
    return true;
  }
};

__host__ __device__ inline int div_up(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

// ---------------------------------------------------------------- launchers --
int launch_act_pack(const ActDims& A, const void* x, int64_t ldx, int8_t* codes,
                    float* steps, hipStream_t st);
int launch_act_unpack(const ActDims& A, const int8_t* codes, const float* steps,
                      void* x, int64_t ldx, hipStream_t st);

struct LayerNormArgs {
  const void* x;
  int64_t ldx;
  const float *weight, *bias;
  float eps;
  void* y;
  int64_t ldy;
  float *mean, *rstd;
  int8_t* x_codes;
  float* x_steps;
  int8_t* y_codes;
  float* y_steps;
};
int launch_layer_norm(const ActDims& A, const LayerNormArgs& a, hipStream_t st);
// whether the 8-bit form of y is taken from y in memory (long rows and groups)
bool layer_norm_needs_y(const ActDims& A);

struct LayerNormBackArgs {
  const void* dy;
  int64_t lddy;
  const void* x;  // or the 8-bit form:
  int64_t ldx;
  const int8_t* codes;
  const float* steps;
  const float *mean, *rstd, *weight;
  void* dx;
  int64_t lddx;
  float beta;
  float *dweight, *dbias;
  float* ws;
};
int64_t layer_norm_workspace(const ActDims& A);
int launch_layer_norm_backward(const ActDims& A, const LayerNormBackArgs& a,
                               hipStream_t st);

int64_t act_linear_workspace(const ActDims& A, int64_t out);
int launch_act_linear(const ActDims& A, int64_t out, const int8_t* codes,
                      const float* steps, const int8_t* w_codes,
                      const float* w_steps, const float* bias, void* y,
                      int64_t ldy, void* ws, hipStream_t st);

int64_t act_wgrad_workspace(const ActDims& A, int64_t out);
int launch_act_wgrad(const ActDims& A, int64_t out, const void* dy, int64_t lddy,
                     const int8_t* codes, const float* steps, float beta,
                     float* dw, float* db, void* ws, hipStream_t st);

}  // namespace gq
