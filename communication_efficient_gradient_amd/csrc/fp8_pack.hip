// fp8_pack.hip — activations and weights to their 8-bit floating point form
// (fp8.hpp), and activations back.
//
// One pass over HBM each.  Activations: a thread owns eight consecutive
// columns, the 128 of a step lie in 16 neighbouring lanes and need only lane
// exchanges.  Weights: a workgroup owns a block of 128 x 128, a thread 8 x 8 of
// it in registers, which is all that both directions need: the transposed
// form of a block is the block's codes turned around, with the same step.
//
// At the rate of a large copy (5.05 TB/s here) from about 100 MB on:
// activations 8192 x 4096 bf16 21 to 25 us, 4.1 to 4.8 TB/s, and back 21 (16384 rows
// 38 both ways; fp32 30 and 34; 8192 x 4100 bf16 24 and 29, fp32 31 and 48); eight
// fp32 weights of 4096 x 4096, both directions 151 us, 5.3 TB/s, one 131 or 124; bf16
// 116 us, 4.6 TB/s, and 4.0 TB/s where rows are not whole 16 bytes (32 x 1001 x 2050:
// 66 us, 1008 x 2048 50).  Small ones are bounded by the latency of one load and one
// store: a weight of 4096 x 1024, one block per CU, 7.5 us of which 5 are its
// bytes'.
#include "act_bounds.hpp"
#include "fp8.hpp"

namespace gq {
namespace {

constexpr int kBlock = kCoverThreads;

// Workgroups of `turns` side by side cover kBlock >> tlog rows.
template <typename T, int END>
__global__ __launch_bounds__(kBlock) void k_fp8_pack(int64_t rows, int cols, int pitch,
                                                     int groups, int turns, int tlog,
                                                     const T* __restrict__ x, int64_t ldx,
                                                     uint8_t* __restrict__ codes,
                                                     float* __restrict__ steps) {
  const int tpr = 1 << tlog;
  const uint32_t unit = blockIdx.x / (uint32_t)turns;
  const int turn = (int)(blockIdx.x - unit * (uint32_t)turns);
  const int64_t row = (int64_t)unit * (kBlock >> tlog) + ((int)threadIdx.x >> tlog);
  const int chunk = turn * tpr + ((int)threadIdx.x & (tpr - 1)), c = chunk * 8;
  const int end = row < rows ? cols : 0;
  Raw8<T> raw = load_chunk<END>(x + row * ldx, c, end);
  settle<END>(raw, c, end);
  float f[8];
  widen(raw, f);
  const Step s = float_step<8>(lanes_max(max_abs_bits(f), 16), kMaxFp8StepExp<T>);
  if (row >= rows) return;
  if (c < pitch) *reinterpret_cast<uint2*>(codes + row * pitch + c) = fp8_codes8(f, s);
  if ((chunk & 15) == 0 && chunk / 16 < groups) steps[row * groups + chunk / 16] = s.step;
}

template <typename T, int END>
__global__ __launch_bounds__(kBlock) void k_fp8_unpack(int64_t rows, int cols, int pitch,
                                                       int groups, int turns, int tlog,
                                                       const uint8_t* __restrict__ codes,
                                                       const float* __restrict__ steps,
                                                       T* __restrict__ x, int64_t ldx) {
  const int tpr = 1 << tlog;
  const uint32_t unit = blockIdx.x / (uint32_t)turns;
  const int turn = (int)(blockIdx.x - unit * (uint32_t)turns);
  const int64_t row = (int64_t)unit * (kBlock >> tlog) + ((int)threadIdx.x >> tlog);
  const int c = (turn * tpr + ((int)threadIdx.x & (tpr - 1))) * 8;
  if (row >= rows || c >= cols) return;
  float f[8];
  fp8_decode8(*reinterpret_cast<const uint2*>(codes + row * pitch + c),
              steps[row * groups + c / kFp8Block], f);
  store_chunk<END>(x + row * ldx + c, narrow<T>(f), cols - c);
}

// The bytes of 4 x 4: out[j] byte i = in[i] byte j.
__device__ __forceinline__ void transpose4(const uint32_t (&in)[4], uint32_t (&out)[4]) {
  const uint32_t a = __builtin_amdgcn_perm(in[1], in[0], 0x05010400u);  // 00 10 01 11
  const uint32_t b = __builtin_amdgcn_perm(in[1], in[0], 0x07030602u);  // 02 12 03 13
  const uint32_t c = __builtin_amdgcn_perm(in[3], in[2], 0x05010400u);
  const uint32_t d = __builtin_amdgcn_perm(in[3], in[2], 0x07030602u);
  out[0] = __builtin_amdgcn_perm(c, a, 0x05040100u);
  out[1] = __builtin_amdgcn_perm(c, a, 0x07060302u);
  out[2] = __builtin_amdgcn_perm(d, b, 0x05040100u);
  out[3] = __builtin_amdgcn_perm(d, b, 0x07060302u);
}

struct WeightArgs {
  int64_t blocks;        // of all experts
  int out, cols, pitch, t_pitch, out_blocks, col_blocks;
  uint8_t *codes, *t_codes;
  float *steps, *t_steps;
};

template <typename T, int END>
__global__ __launch_bounds__(256) void k_fp8_pack_weight(WeightArgs a, const T* __restrict__ w) {
  __shared__ uint32_t red[4];
  const int tid = (int)threadIdx.x, tr = tid / 16 * 8, tc = tid % 16 * 8;
  for (int64_t at = blockIdx.x; at < a.blocks; at += gridDim.x) {
    const int64_t line = at / a.col_blocks;
    const int cb = (int)(at - line * a.col_blocks);
    const int64_t e = line / a.out_blocks;
    const int ob = (int)(line - e * a.out_blocks);
    const int o = ob * kFp8Block + tr, c = cb * kFp8Block + tc;
    const T* from = w + (e * a.out + o) * a.cols;
    Raw8<T> raw[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      raw[i] = load_chunk<END>(from + (int64_t)i * a.cols, c, o + i < a.out ? a.cols : 0);
    float f[8][8];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      settle<END>(raw[i], c, o + i < a.out ? a.cols : 0);
      widen(raw[i], f[i]);
      m = max(m, max_abs_bits(f[i]));
    }
    m = lanes_max(m, 64);
    __syncthreads();
    if (tid % 64 == 0) red[tid / 64] = m;
    __syncthreads();
    m = max(max(red[0], red[1]), max(red[2], red[3]));
    const Step s = float_step<8>(m, kMaxFp8StepExp<T>);
    uint2 q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = fp8_codes8(f[i], s);
    if (a.codes) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (o + i < a.out && c < a.pitch)
          *reinterpret_cast<uint2*>(a.codes + (e * a.out + o + i) * a.pitch + c) = q[i];
      if (tid == 0) a.steps[at] = s.step;
    }
    if (a.t_codes) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {   // columns c + 4 h .. c + 4 h + 3
        uint32_t lo[4], hi[4], tl[4], th[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          lo[i] = h ? q[i].y : q[i].x;
          hi[i] = h ? q[i + 4].y : q[i + 4].x;
        }
        transpose4(lo, tl);
        transpose4(hi, th);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int col = c + h * 4 + j;
          if (col < a.cols && o < a.t_pitch)
            *reinterpret_cast<uint2*>(a.t_codes + (e * a.cols + col) * a.t_pitch + o) =
                make_uint2(tl[j], th[j]);
        }
      }
      if (tid == 0) a.t_steps[(e * a.col_blocks + cb) * a.out_blocks + ob] = s.step;
    }
  }
}

template <typename T>
int pack_t(const ActDims& A, const T* x, int64_t ldx, uint8_t* codes, float* steps,
           hipStream_t st) {
  // whole steps in each workgroup
  const Cover c(A.groups * 16, 1);
  const RowEnd end = row_end(A.cols);
  auto* k = end == kWhole    ? k_fp8_pack<T, kWhole>
            : end == kRagged ? k_fp8_pack<T, kRagged>
                             : k_fp8_pack<T, kTiny>;
  for (int64_t r = 0; r < A.rows; r += c.rows) {
    const int64_t n = A.rows - r < c.rows ? A.rows - r : c.rows;
    k<<<(unsigned)c.blocks(n), kBlock, 0, st>>>(n, (int)A.cols, (int)A.pitch, A.groups, c.turns,
                                                c.tlog, x + r * ldx, ldx, codes + r * A.pitch,
                                                steps + r * A.groups);
  }
  return (int)hipGetLastError();
}

template <typename T>
int unpack_t(const ActDims& A, const uint8_t* codes, const float* steps, T* x, int64_t ldx,
             hipStream_t st) {
  const Cover c(div_up(A.cols, 8), 1);
  auto* k = A.cols % 8 ? k_fp8_unpack<T, kRagged> : k_fp8_unpack<T, kWhole>;
  for (int64_t r = 0; r < A.rows; r += c.rows) {
    const int64_t n = A.rows - r < c.rows ? A.rows - r : c.rows;
    k<<<(unsigned)c.blocks(n), kBlock, 0, st>>>(n, (int)A.cols, (int)A.pitch, A.groups, c.turns,
                                                c.tlog, codes + r * A.pitch,
                                                steps + r * A.groups, x + r * ldx, ldx);
  }
  return (int)hipGetLastError();
}

template <typename T>
int weight_t(const WeightArgs& a, const T* w, hipStream_t st) {
  const RowEnd end = row_end(a.cols);
  auto* k = end == kWhole    ? k_fp8_pack_weight<T, kWhole>
            : end == kRagged ? k_fp8_pack_weight<T, kRagged>
                             : k_fp8_pack_weight<T, kTiny>;
  const int64_t most = int64_t(1) << 20;
  k<<<(unsigned)(a.blocks < most ? a.blocks : most), 256, 0, st>>>(a, w);
  return (int)hipGetLastError();
}

}  // namespace

int launch_fp8_pack(const ActDims& A, const void* x, int64_t ldx, uint8_t* codes,
                    float* steps, hipStream_t st) {
  if (A.rows == 0) return 0;
  switch (A.dtype) {
    case GQ_F32: return pack_t(A, (const float*)x, ldx, codes, steps, st);
    case GQ_BF16: return pack_t(A, (const __bf16*)x, ldx, codes, steps, st);
    default: return pack_t(A, (const _Float16*)x, ldx, codes, steps, st);
  }
}

int launch_fp8_unpack(const ActDims& A, const uint8_t* codes, const float* steps, void* x,
                      int64_t ldx, hipStream_t st) {
  if (A.rows == 0) return 0;
  switch (A.dtype) {
    case GQ_F32: return unpack_t(A, codes, steps, (float*)x, ldx, st);
    case GQ_BF16: return unpack_t(A, codes, steps, (__bf16*)x, ldx, st);
    default: return unpack_t(A, codes, steps, (_Float16*)x, ldx, st);
  }
}

int launch_fp8_pack_weight(const ActDims& A, int experts, const void* w, uint8_t* codes,
                           float* steps, uint8_t* t_codes, float* t_steps, hipStream_t st) {
  if (A.rows == 0) return 0;
  const int ob = div_up(A.rows, kFp8Block), cb = A.groups;
  const WeightArgs a = {(int64_t)experts * ob * cb, (int)A.rows, (int)A.cols, (int)A.pitch,
                        (int)((A.rows + 15) / 16 * 16), ob, cb, codes, t_codes, steps, t_steps};
  switch (A.dtype) {
    case GQ_F32: return weight_t(a, (const float*)w, st);
    case GQ_BF16: return weight_t(a, (const __bf16*)w, st);
    default: return weight_t(a, (const _Float16*)w, st);
  }
}

}  // namespace gq
