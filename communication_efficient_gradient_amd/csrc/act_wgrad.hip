// act_wgrad.hip — weight and bias gradient of a linear layer whose input is
// kept in 8 bits:
//   dw[o, c] <- beta dw[o, c] + sum_t dy[t, o] x^[t, c]
//   db[o]    <- beta db[o]    + sum_t dy[t, o]
//
// The sum runs over tokens, the slow axis of both operands, so tiles [t][col]
// go to LDS as they lie in memory and come out through the transposing LDS
// read (each lane gets consecutive tokens of one column, the operand layout
// of the matrix instructions).  x^ = code * step is exact in bf16.  dy in
// bf16 is used as it is; fp16 is split into two and fp32 into three bf16
// terms whose sum is the value itself (11 and 24 significant bits), one
// matrix product each: every product is exact and only the fp32 accumulation
// rounds.
#include "act.hpp"

namespace gq {
namespace {

#define GQ_LDS __attribute__((address_space(3)))

template <typename T>
constexpr int kPlanes = 1;
template <>
inline constexpr int kPlanes<_Float16> = 2;
template <>
inline constexpr int kPlanes<float> = 3;

struct WgradArgs {
  int64_t rows;
  int out, cols, pitch, groups, glog;
  const void* dy;
  int64_t lddy;
  const int8_t* codes;
  const float* steps;
  float beta;
  float *dw, *db;      // results, or the splits' parts [split][out][cols]
  float *ws_w, *ws_b;
  int splits;
  int64_t per;         // tokens of a split, a multiple of 32
};

// Element offset of 16-column chunk `ch` of token row t in a tile of W
// columns.  Chunks (32 bytes) change places with t so that the sixteen rows
// one transposing read touches fall on different banks.
template <int W>
__device__ __forceinline__ int place(int t, int ch) {
  return t * W + ((ch ^ ((t & 3) | (t >> 1 & 4))) << 4);
}

// Operand of a 16x16x32 product: column col0 + lane % 16, tokens 8 (lane / 16)
// + 0..7.  Sixteen lanes fetch four rows of 16 columns and get them
// transposed.
template <int W>
__device__ __forceinline__ bf16x8 operand(const short* tile, int ch, int lane) {
  const int t = lane / 16 * 8 + lane % 16 / 4, part = lane % 4 * 4;
  const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      (GQ_LDS s16x4*)(tile + place<W>(t, ch) + part));
  const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      (GQ_LDS s16x4*)(tile + place<W>(t + 4, ch) + part));
  return __builtin_bit_cast(
      bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

template <typename T>
__global__ __launch_bounds__(256) void k_act_wgrad(WgradArgs a) {
  constexpr int P = kPlanes<T>, BT = 128;
  __shared__ __attribute__((aligned(16))) short lds_a[P][32 * BT];
  __shared__ __attribute__((aligned(16))) short lds_b[32 * BT];
  __shared__ float lds_s[32][BT];
  const int tid = (int)threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wo = wave % 2 * 64, wc = wave / 2 * 64;
  const int o0 = (int)blockIdx.y * BT, c0 = (int)blockIdx.x * BT;
  const int64_t t0 = (int64_t)blockIdx.z * a.per;
  const int64_t t1 = min(t0 + a.per, a.rows);
  const int tr = tid / 8, ch = tid % 8;  // staging: row, 16-column chunk
  const bool sum_bias = a.db != nullptr && blockIdx.x == 0;
  float bsum[16] = {};
  f32x4 acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  for (int64_t t = t0; t < t1; t += 32) {
    const int64_t row = t + tr;
    const bool live = row < t1;
    float v[16];
    {
      const T* p = (const T*)a.dy + (live ? row : 0) * a.lddy + o0 + ch * 16;
      const int valid = live ? a.out - o0 - ch * 16 : 0;
      float f[8];
      widen(load8(p, valid), f);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = f[j];
      widen(load8(p + 8, valid - 8), f);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[8 + j] = f[j];
    }
    uint4 w = make_uint4(0, 0, 0, 0);
    float step = 0.f;
    const int c = c0 + ch * 16;
    if (live && c < a.pitch) {
      w = *reinterpret_cast<const uint4*>(a.codes + row * a.pitch + c);
      step = a.steps[row * a.groups + min(c >> a.glog, a.groups - 1)];
    }
    __syncthreads();
    if (sum_bias) {
#pragma unroll
      for (int j = 0; j < 16; ++j) bsum[j] += v[j];
    }
#pragma unroll
    for (int p = 0; p < P; ++p) {
      __bf16 h[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        // the first eight significant bits, exactly; the rest stays in v
        const uint32_t b = __float_as_uint(v[j]);
        h[j] = __builtin_bit_cast(__bf16, (uint16_t)(b >> 16));
        if (p + 1 < P) v[j] -= __uint_as_float(b & 0xffff0000u);
      }
      __builtin_memcpy(&lds_a[p][place<BT>(tr, ch)], h, 32);
    }
    {
      float f[16];
      decode4(w.x, step, f);
      decode4(w.y, step, f + 4);
      decode4(w.z, step, f + 8);
      decode4(w.w, step, f + 12);
      __bf16 h[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) h[j] = (__bf16)f[j];
      __builtin_memcpy(&lds_b[place<BT>(tr, ch)], h, 32);
    }
    __syncthreads();
    bf16x8 fb[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) fb[j] = operand<BT>(lds_b, wc / 16 + j, lane);
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bf16x8 fa = operand<BT>(lds_a[p], wo / 16 + i, lane);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[j], fa, acc[i][j], 0, 0, 0);
      }
  }
  // a lane holds four consecutive columns of one output feature
  const bool parts = a.splits > 1;
  float* dw = parts ? a.ws_w + (int64_t)blockIdx.z * a.out * a.cols : a.dw;
  const float beta = parts ? 0.f : a.beta;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int o = o0 + wo + i * 16 + lane % 16;
    if (o >= a.out) continue;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int c = c0 + wc + j * 16 + lane / 16 * 4;
      float* q = dw + (int64_t)o * a.cols + c;
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (c + r < a.cols) q[r] = beta == 0.f ? acc[i][j][r] : fmaf(beta, q[r], acc[i][j][r]);
    }
  }
  if (sum_bias) {
#pragma unroll
    for (int j = 0; j < 16; ++j) lds_s[tr][ch * 16 + j] = bsum[j];
    __syncthreads();
    const int o = o0 + tid;
    if (tid < BT && o < a.out) {
      float s = 0.f;
      for (int t = 0; t < 32; ++t) s += lds_s[t][tid];
      if (parts) {
        a.ws_b[(int64_t)blockIdx.z * a.out + o] = s;
      } else {
        a.db[o] = beta == 0.f ? s : fmaf(beta, a.db[o], s);
      }
    }
  }
}

// Adds the splits' parts, in order.
__global__ __launch_bounds__(256) void k_act_wgrad_join(int64_t n, int splits, float beta,
                                                        const float* __restrict__ parts,
                                                        float* __restrict__ out) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n;
       i += (int64_t)gridDim.x * 256) {
    float s = parts[i];
    for (int k = 1; k < splits; ++k) s += parts[k * n + i];
    out[i] = beta == 0.f ? s : fmaf(beta, out[i], s);
  }
}

struct Plan {
  int splits;
  int64_t per;
};

Plan plan_wgrad(const ActDims& A, int64_t out) {
  const int64_t tiles = ((out + 127) / 128) * ((A.cols + 127) / 128);
  const int64_t steps = (A.rows + 31) / 32;
  int64_t splits = tiles >= 2 * kCus ? 1 : 2 * kCus / tiles;
  if (splits > steps / 8) splits = steps / 8 > 0 ? steps / 8 : 1;
  Plan p;
  p.per = steps == 0 ? 32 : (steps + splits - 1) / splits * 32;
  p.splits = steps == 0 ? 1 : div_up(steps * 32, p.per);
  return p;
}

}  // namespace

int64_t act_wgrad_workspace(const ActDims& A, int64_t out) {
  const Plan p = plan_wgrad(A, out);
  return p.splits > 1 ? 4 * (int64_t)p.splits * out * (A.cols + 1) : 0;
}

int launch_act_wgrad(const ActDims& A, int64_t out, const void* dy, int64_t lddy,
                     const int8_t* codes, const float* steps, float beta,
                     float* dw, float* db, void* ws, hipStream_t st) {
  const Plan p = plan_wgrad(A, out);
  int glog = 31;
  if (!A.whole_row)
    for (glog = 0; (1 << glog) < A.group;) ++glog;
  float* w = (float*)ws;
  const WgradArgs a = {A.rows, (int)out, (int)A.cols, (int)A.pitch, A.groups, glog,
                       dy,     lddy,     codes,       steps,        beta,     dw,
                       db,     w,        w + (int64_t)p.splits * out * A.cols,
                       p.splits, p.per};
  const dim3 g(div_up(A.cols, 128), div_up(out, 128), p.splits);
  switch (A.dtype) {
    case GQ_F32: k_act_wgrad<float><<<g, 256, 0, st>>>(a); break;
    case GQ_BF16: k_act_wgrad<__bf16><<<g, 256, 0, st>>>(a); break;
    default: k_act_wgrad<_Float16><<<g, 256, 0, st>>>(a);
  }
  int rc = (int)hipGetLastError();
  if (rc == 0 && p.splits > 1) {
    const int64_t n = out * A.cols, b = (n + 255) / 256;
    k_act_wgrad_join<<<(unsigned)(b < 4096 ? b : 4096), 256, 0, st>>>(n, p.splits, beta,
                                                                     a.ws_w, dw);
    if (db)
      k_act_wgrad_join<<<div_up(out, 256), 256, 0, st>>>(out, p.splits, beta, a.ws_b, db);
    rc = (int)hipGetLastError();
  }
  return rc;
}

}  // namespace gq
