// fp8.hpp — the 8-bit floating point form shared by fp8_pack, fp8_linear and
// fp8_wgrad, and their launchers.
//
// A matrix [rows, cols] is kept as e4m3 codes (OCP: largest 448, smallest
// 2^-9) in rows of `pitch` bytes (cols rounded up to 16, padding codes 0) and
// one fp32 step per 128 columns: of each row for activations, of 128 rows for
// weights; x^ = code * step.  A step is a power of two.  With floating point
// codes that costs nothing (a free step would not make them finer), and it is
// what the matrix instructions scale by themselves: they take a biased exponent
// per row of an operand, which is bits 23 .. 30 of the fp32 step as it lies (0
// for a step of 0, whose codes are 0; 255, their NaN, for a step of NaN).  So a
// sum over all blocks stays in one accumulator, with no product or addition of
// the vector units between blocks.
#pragma once

#include "act.hpp"

namespace gq {

constexpr int kFp8Block = 128;      // columns of a step, and rows of a weight's
constexpr int kMaxExperts = 1024;

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

// The largest step, as a biased exponent: 448 * step is finite in the type.
template <typename T>
constexpr uint32_t kMaxFp8StepExp = 119 + 127;
template <>
inline constexpr uint32_t kMaxFp8StepExp<_Float16> = 7 + 127;

// The smallest power of two with top * step >= M (M as abs_bits), top = 1.75 *
// 2^TOP (448: TOP 8, e5m2's 57344: TOP 15), from 2^-126 to 2^(cap - 127): 0
// for M = 0, NaN if M is not finite.  inv = 1 / step, or 0 where all codes are 0.
template <int TOP>
__device__ __forceinline__ Step float_step(uint32_t m, uint32_t cap) {
  const uint32_t ex = m >> 23, frac = m & 0x7fffffu;
  uint32_t s = ex > TOP ? ex - TOP + (frac > 0x600000u ? 1u : 0u) : 1u;
  s = min(max(s, 1u), cap);
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

// Eight codes of x / step, nearest, ties to even, saturating.  The product
// with a power of two is exact but where it is far below the smallest code.
__device__ __forceinline__ uint2 fp8_codes8(const float (&f)[8], const Step& s) {
  float q[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) q[j] = __builtin_amdgcn_fmed3f(f[j] * s.inv, -448.f, 448.f);
  int a = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
  a = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], a, true);
  int b = __builtin_amdgcn_cvt_pk_fp8_f32(q[4], q[5], 0, false);
  b = __builtin_amdgcn_cvt_pk_fp8_f32(q[6], q[7], b, true);
  uint2 r = make_uint2((uint32_t)a, (uint32_t)b);
  if (s.inv == 0.f) r.x = r.y = 0;  // 0 * inf and 0 * NaN are not 0
  return r;
}

__device__ __forceinline__ void fp8_decode8(uint2 w, float step, float (&f)[8]) {
  const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w.x, false);
  const f32x2 b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w.x, true);
  const f32x2 c = __builtin_amdgcn_cvt_pk_f32_fp8((int)w.y, false);
  const f32x2 d = __builtin_amdgcn_cvt_pk_f32_fp8((int)w.y, true);
  f[0] = a[0] * step;
  f[1] = a[1] * step;
  f[2] = b[0] * step;
  f[3] = b[1] * step;
  f[4] = c[0] * step;
  f[5] = c[1] * step;
  f[6] = d[0] * step;
  f[7] = d[1] * step;
}

// Tokens of expert e, within the matrix whatever the table holds.  NULL: the
// one expert has them all.
struct Tokens {
  int64_t lo, hi;
};

__device__ __forceinline__ Tokens tokens_of(const int64_t* offsets, int e, int64_t rows) {
  if (!offsets) return {0, rows};
  const int64_t lo = min(max(offsets[e], (int64_t)0), rows);
  return {lo, min(max(offsets[e + 1], lo), rows)};
}

// ---------------------------------------------------------------- launchers --
int launch_fp8_pack(const ActDims& A, const void* x, int64_t ldx, uint8_t* codes,
                    float* steps, hipStream_t st);
int launch_fp8_unpack(const ActDims& A, const uint8_t* codes, const float* steps, void* x,
                      int64_t ldx, hipStream_t st);
// A: rows = output features, of each expert
int launch_fp8_pack_weight(const ActDims& A, int experts, const void* w, uint8_t* codes,
                           float* steps, uint8_t* t_codes, float* t_steps, hipStream_t st);

int64_t fp8_linear_workspace(const ActDims& A, int64_t out, int experts);
int launch_fp8_linear(const ActDims& A, int64_t out, int experts, const int64_t* offsets,
                      const uint8_t* codes, const float* steps, const uint8_t* w_codes,
                      const float* w_steps, const float* bias, void* y, int64_t ldy, void* ws,
                      hipStream_t st);

int64_t fp8_wgrad_workspace(const ActDims& A, int64_t out, int experts);
int launch_fp8_wgrad(const ActDims& A, int64_t out, int experts, const int64_t* offsets,
                     const void* dy, int64_t lddy, const uint8_t* codes, const float* steps,
                     float beta, float* dw, float* db, void* ws, hipStream_t st);

}  // namespace gq
