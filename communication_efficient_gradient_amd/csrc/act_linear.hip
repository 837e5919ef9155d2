// act_linear.hip — the product of a linear layer in 8-bit integers:
//   y[t, o] = (sum_c q[t, c] w[o, c]) s[t] v[o] + b[o]
// with one step s per token and one v per output feature.  The integer sums
// are exact (int32, |code| <= 128, so up to 131071 columns), in any order.
//
// Both operands are rows of int8 along the summed axis, 16-byte aligned and
// zero-padded, which is the layout the matrix instructions take: 16 (32x32x32)
// consecutive codes per lane, straight from LDS.
#include "act.hpp"

namespace gq {
namespace {

// Sixteen bytes of zeros for lanes past the end of a row.
__device__ __attribute__((aligned(16))) const int8_t kZeros[16] = {};

#define GQ_LDS __attribute__((address_space(3)))
#define GQ_GLOBAL __attribute__((address_space(1)))

// 16 bytes per lane from global memory into LDS at base + lane * 16, without
// passing through registers.
__device__ __forceinline__ void copy16_to_lds(const void* src, void* base) {
  __builtin_amdgcn_global_load_lds((const GQ_GLOBAL void*)src, (GQ_LDS void*)base, 16, 0, 0);
}

template <typename T>
__device__ __forceinline__ void store_out4(T* y, const float (&f)[4], int valid) {
  T o[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) o[j] = (T)f[j];
  if (valid >= 4) {
    __builtin_memcpy(y, o, sizeof(o));
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < valid) y[j] = o[j];
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
};

// A tile of BM tokens by BN outputs per workgroup, WM by WN of it per wave, in
// k-tiles of 128 codes.  LDS rows are 128 bytes in eight 16-byte chunks, chunk
// j of row r at place j ^ (r / 2 % 8): sixteen lanes that read one chunk of
// sixteen rows then touch every bank once.
template <typename T, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__((BM / WM) * (BN / WN) * 64) void k_act_linear(LinearArgs a) {
  constexpr int WAVES = (BM / WM) * (BN / WN);
  constexpr int MT = WM / 32, NTL = WN / 32;
  __shared__ __attribute__((aligned(16))) int8_t lds[2][(BM + BN) * 128];
  const int lane = (int)threadIdx.x & 63, wave = (int)threadIdx.x >> 6;
  const int wm = wave % (BM / WM) * WM, wn = wave / (BM / WM) * WN;
  const int64_t m0 = (int64_t)blockIdx.y * BM;
  const int n0 = (int)blockIdx.x * BN;
  const int kt0 = (int)blockIdx.z * a.per;
  const int nk = min(a.per, div_up(a.pitch, 128) - kt0);

  // copies: a wave instruction fills 8 rows
  constexpr int COPIES = (BM + BN) / 8 / WAVES;
  const int8_t* src[COPIES];
  int chunk[COPIES];
#pragma unroll
  for (int i = 0; i < COPIES; ++i) {
    const int r = (wave * COPIES + i) * 8 + lane / 8;
    chunk[i] = (lane % 8) ^ (r / 2 % 8);
    // rows past the end repeat the last one; what they give is not stored
    if (r < BM) {
      const int64_t m = min(m0 + r, a.rows - 1);
      src[i] = a.codes + m * a.pitch;
    } else {
      const int n = min(n0 + r - BM, a.out - 1);
      src[i] = a.w_codes + (int64_t)n * a.pitch;
    }
  }
  auto fill = [&](int kt, int buf) {
#pragma unroll
    for (int i = 0; i < COPIES; ++i) {
      const int k = (kt0 + kt) * 128 + chunk[i] * 16;
      copy16_to_lds(k < a.pitch ? src[i] + k : kZeros,
                    &lds[buf][(wave * COPIES + i) * 1024]);
    }
  };
  i32x16 acc[NTL][MT];
#pragma unroll
  for (int i = 0; i < NTL; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0;

  auto frag = [&](int buf, int row, int kk) {
    const int r = row + lane % 32;
    const int p = (kk * 2 + lane / 32) ^ (r / 2 % 8);
    return *reinterpret_cast<const i32x4*>(&lds[buf][r * 128 + p * 16]);
  };
  if (nk > 0) fill(0, 0);
  __syncthreads();
  for (int kt = 0; kt < nk; ++kt) {
    const int buf = kt & 1;
    if (kt + 1 < nk) fill(kt + 1, buf ^ 1);
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      i32x4 fm[MT], fn[NTL];
#pragma unroll
      for (int j = 0; j < MT; ++j) fm[j] = frag(buf, wm + j * 32, kk);
#pragma unroll
      for (int i = 0; i < NTL; ++i) fn[i] = frag(buf, BM + wn + i * 32, kk);
#pragma unroll
      for (int i = 0; i < NTL; ++i)
#pragma unroll
        for (int j = 0; j < MT; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fn[i], fm[j], acc[i][j], 0, 0, 0);
    }
    __syncthreads();
  }
  // a lane holds, of one token, four consecutive outputs in each of four
  // quarters of a 32 x 32 tile
#pragma unroll
  for (int j = 0; j < MT; ++j) {
    const int64_t m = m0 + wm + j * 32 + lane % 32;
    if (m >= a.rows) continue;
    const float s = a.steps[m];
#pragma unroll
    for (int i = 0; i < NTL; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int n = n0 + wn + i * 32 + q * 8 + lane / 32 * 4;
        if (n >= a.out) continue;
        if (a.splits > 1) {
          int32_t* p = a.ws + ((int64_t)blockIdx.z * a.rows + m) * a.out + n;
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (n + r < a.out) p[r] = acc[i][j][q * 4 + r];
        } else {
          float f[4];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int o = min(n + r, a.out - 1);
            f[r] = (float)acc[i][j][q * 4 + r] * s * a.w_steps[o] +
                   (a.bias ? a.bias[o] : 0.f);
          }
          store_out4((T*)a.y + m * a.ldy + n, f, a.out - n);
        }
      }
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

struct Plan {
  int splits, per;
};

Plan plan_linear(const ActDims& A, int64_t out) {
  const int kt = div_up(A.pitch, 128);
  const int64_t tiles = ((A.rows + 127) / 128) * ((out + 127) / 128);
  int splits = tiles >= kCus ? 1 : (int)(kCus / tiles);
  if (splits > kt / 4) splits = kt / 4 > 0 ? kt / 4 : 1;
  Plan p;
  p.per = div_up(kt, splits);
  p.splits = div_up(kt, p.per);
  return p;
}

template <typename T>
int linear_t(const ActDims& A, LinearArgs a, hipStream_t st) {
  const dim3 g(div_up(a.out, 128), div_up(A.rows, 128), a.splits);
  k_act_linear<T, 128, 128, 64, 64><<<g, 256, 0, st>>>(a);
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
                        bias,    y,        ldy,          (int32_t*)ws, p.splits, p.per};
  switch (A.dtype) {
    case GQ_F32: return linear_t<float>(A, a, st);
    case GQ_BF16: return linear_t<__bf16>(A, a, st);
    default: return linear_t<_Float16>(A, a, st);
  }
}

}  // namespace gq
