// layer_norm.hip — layer norm forward and backward over the rows of an
// activation matrix, with the 8-bit form of its input and output.
//
//   forward   mu = sum x / C, r = 1 / sqrt(sum (x - mu)^2 / C + eps),
//             y = (x - mu) r w + b
//   backward  xh = (x - mu) r, a = dy w,
//             dx = r (a - mean(a) - xh mean(a xh)),
//             dw = sum_rows dy xh, db = sum_rows dy
//
// Up to 8192 columns all of it is bound by HBM: a row is read once and stays in
// registers (R chunks of eight columns in each of NT threads), so the forward moves
// 2 e bytes per value and the backward 3 e, or 2 e + 1 when it reads the
// 8-bit form of x.  Statistics and gradients are fp32; the variance is taken
// from the centred values in registers, which loses nothing where |mu| is
// large.  Workgroups stay resident and walk the rows: the weight is read
// once per workgroup, the next row is on its way while the present one is
// reduced, and each thread keeps the weight's and bias's gradient of its own
// columns in registers.  A second launch adds the workgroups' partial sums
// in a fixed order, so results repeat bit for bit.  16384 x 4096 bf16: forward
// with its input's 8-bit form 62 us, 5.4 TB/s, backward from that form 70 us and
// 6.2 for the partial sums (a large copy's rate is 5.1 TB/s); forward with its
// output's form 67 us, 92 as norm and pack.
//
// Two widths are further from that.  From 8193 to 16384 columns the backward
// pass with gradients has no registers for all it keeps (128 per thread: 108 to
// 220 bytes of scratch a lane): 4096 x 12288 bf16 182 us from x and 216 from the
// 8-bit form, 51 without gradients.  Over 16384 columns rows are read again:
// three times forward (4096 x 20000 bf16 176 us), twice backward and once more
// for the column sums (280 us).
#include "act.hpp"

namespace gq {
namespace {


// Sum over NT threads of A and B at once, in all of them; the order is fixed.
// red: 2 x 2 x 16 floats, alternated by `phase` so that one barrier suffices.
template <int NT>
__device__ __forceinline__ void block_sum2(float& a, float& b, float (*red)[2][16],
                                           int phase) {
  a = group_reduce<64>(a, [](float u, float v) { return u + v; });
  b = group_reduce<64>(b, [](float u, float v) { return u + v; });
  if constexpr (NT > 64) {
    const int wave = ((int)threadIdx.x % NT) >> 6;
    if ((threadIdx.x & 63) == 0) {
      red[phase][0][wave] = a;
      red[phase][1][wave] = b;
    }
    __syncthreads();
    a = red[phase][0][0];
    b = red[phase][1][0];
#pragma unroll
    for (int i = 1; i < NT / 64; ++i) {
      a += red[phase][0][i];
      b += red[phase][1][i];
    }
  }
}

template <int NT>
__device__ __forceinline__ uint32_t block_max(uint32_t m, uint32_t* red) {
  m = lanes_max(m, 64);
  if constexpr (NT > 64) {
    if ((threadIdx.x & 63) == 0) red[((int)threadIdx.x % NT) >> 6] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NT / 64; ++i) m = max(m, red[i]);
    __syncthreads();
  }
  return m;
}

// A vector's columns, or `none` where there is no vector; settled later.
template <int END>
__device__ __forceinline__ Raw8<float> load_vec(const float* __restrict__ p, int c, int cols,
                                                float none) {
  if (p != nullptr) return load_chunk<END>(p, c, cols);
  Raw8<float> r;
#pragma unroll
  for (int j = 0; j < 8; ++j) r.v[j] = none;
  return r;
}

template <int END>
__device__ __forceinline__ void use_vec(Raw8<float> r, const float* p, int c, int cols,
                                        float (&f)[8]) {
  if (p != nullptr) settle<END>(r, c, cols);
  widen(r, f);
}

// The 8-bit form of a row held as f[R][8]: one step per 2^Glog lanes, or (Glog
// < 0) per row.  A chunk below the pitch lies in one of the row's groups.
template <typename T, int NT, int R>
__device__ __forceinline__ void pack_row(const float (&f)[R][8], int lane, int pitch,
                                         int groups, int Glog, int8_t* codes,
                                         float* steps, uint32_t* red) {
  const int G = Glog < 0 ? 0 : 1 << Glog;
  uint32_t m[R];
#pragma unroll
  for (int i = 0; i < R; ++i) m[i] = max_abs_bits(f[i]);
  if (G == 0) {
    uint32_t t = m[0];
#pragma unroll
    for (int i = 1; i < R; ++i) t = max(t, m[i]);
    t = block_max<NT>(t, red);
#pragma unroll
    for (int i = 0; i < R; ++i) m[i] = t;
  } else {
#pragma unroll
    for (int i = 0; i < R; ++i) m[i] = lanes_max(m[i], G);
  }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int c = lane + i * NT;
    const Step s = step_of<T>(m[i]);
    if (c * 8 < pitch) {
      *reinterpret_cast<uint2*>(codes + c * 8) = codes8(f[i], s);
      if (G == 0 ? c == 0 : (c & (G - 1)) == 0) steps[G == 0 ? 0 : c >> Glog] = s.step;
    }
  }
}

// ---------------------------------------------------------------- forward --
// One row per NT threads; a workgroup of BT threads walks BT / NT rows at a
// time.  2^Glog lanes share a step of the 8-bit forms written in the same pass
// (Glog < 0: the row does).
template <typename T, int NT, int R, int END>
__global__ __launch_bounds__(NT < 256 ? 256 : NT) void k_layer_norm(
    int64_t rows, int cols, int pitch, int groups, int Glog, LayerNormArgs a) {
  constexpr int BT = NT < 256 ? 256 : NT;
  constexpr int PER = BT / NT;
  __shared__ float red[2][2][16];
  __shared__ uint32_t redm[16];
  const int lane = (int)threadIdx.x % NT;
  const T* x = (const T*)a.x;
  T* y = (T*)a.y;
  const int64_t stride = (int64_t)gridDim.x * PER;
  int64_t row = (int64_t)blockIdx.x * PER + threadIdx.x / NT;
  if (row >= rows) return;  // whole waves; the whole workgroup where PER = 1
  // everything is on its way before anything is used
  Raw8<T> raw[R];
  Raw8<float> rw[R], rb[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int c = (lane + i * NT) * 8;
    raw[i] = load_chunk<END>(x + row * a.ldx, c, cols);
    rw[i] = load_vec<END>(a.weight, c, cols, 1.f);
    rb[i] = load_vec<END>(a.bias, c, cols, 0.f);
  }
  float w[R][8], b[R][8];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int c = (lane + i * NT) * 8;
    use_vec<END>(rw[i], a.weight, c, cols, w[i]);
    use_vec<END>(rb[i], a.bias, c, cols, b[i]);
  }
  const float n = (float)cols;
  int phase = 0;
  for (;;) {
    float f[R][8], sum = 0.f, none = 0.f;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      settle<END>(raw[i], (lane + i * NT) * 8, cols);
      widen(raw[i], f[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) sum += f[i][j];
    }
    const int64_t next = row + stride;
    if (next < rows) {
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const int c = (lane + i * NT) * 8;
        raw[i] = load_chunk<END>(x + next * a.ldx, c, cols);
      }
    }
    if (a.x_codes)
      pack_row<T, NT, R>(f, lane, pitch, groups, Glog, a.x_codes + row * pitch,
                         a.x_steps + row * groups, redm);
    block_sum2<NT>(sum, none, red, phase);
    phase ^= 1;
    const float mean = sum / n;
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int c = (lane + i * NT) * 8;
      float q = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        f[i][j] -= mean;
        if (END != kWhole && c + j >= cols) f[i][j] = 0.f;
        q = fmaf(f[i][j], f[i][j], q);
      }
      ss += c < cols ? q : 0.f;
    }
    block_sum2<NT>(ss, none, red, phase);
    phase ^= 1;
    const float rstd = 1.f / sqrtf(ss / n + a.eps);
    if (lane == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int c = (lane + i * NT) * 8;
#pragma unroll
      for (int j = 0; j < 8; ++j) f[i][j] = fmaf(f[i][j] * rstd, w[i][j], b[i][j]);
      const Raw8<T> o = narrow<T>(f[i]);
      if (y) store_chunk<END>(y + row * a.ldy + c, o, cols - c);
      if (a.y_codes) {
        // the form of y as it is stored; columns past the last are 0
        widen(o, f[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (END != kWhole ? c + j >= cols : c >= cols) f[i][j] = 0.f;
      }
    }
    if (a.y_codes)
      pack_row<T, NT, R>(f, lane, pitch, groups, Glog, a.y_codes + row * pitch,
                         a.y_steps + row * groups, redm);
    row = next;
    if (row >= rows) return;
  }
}

// Rows longer than the registers hold: three reads, the last two from L2.
template <typename T>
__global__ __launch_bounds__(1024) void k_layer_norm_long(int64_t rows, int cols,
                                                          LayerNormArgs a) {
  __shared__ float red[2][2][16];
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const T* x = (const T*)a.x + row * a.ldx;
    float sum = 0.f, none = 0.f, f[8];
    for (int c = (int)threadIdx.x * 8; c < cols; c += 8192) {
      widen(load8(x + c, cols - c), f);
#pragma unroll
      for (int j = 0; j < 8; ++j) sum += f[j];
    }
    block_sum2<1024>(sum, none, red, 0);
    const float mean = sum / (float)cols;
    float ss = 0.f;
    for (int c = (int)threadIdx.x * 8; c < cols; c += 8192) {
      widen(load8(x + c, cols - c), f);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (c + j < cols) ss = fmaf(f[j] - mean, f[j] - mean, ss);
    }
    block_sum2<1024>(ss, none, red, 1);
    const float rstd = 1.f / sqrtf(ss / (float)cols + a.eps);
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
    for (int c = (int)threadIdx.x * 8; c < cols; c += 8192) {
      float w[8], b[8];
      widen(load8(x + c, cols - c), f);
      use_vec<kRagged>(load_vec<kRagged>(a.weight, c, cols, 1.f), a.weight, c, cols, w);
      use_vec<kRagged>(load_vec<kRagged>(a.bias, c, cols, 0.f), a.bias, c, cols, b);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = fmaf((f[j] - mean) * rstd, w[j], b[j]);
      store8((T*)a.y + row * a.ldy + c, narrow<T>(f), cols - c);
    }
  }
}

// --------------------------------------------------------------- backward --
// Keeps a chunk of 16-bit values as it was loaded up to here.  Otherwise its
// values may be taken apart where the next row is fetched, which waits for that
// load (forward and backward of 16384 x 4096 bf16, x kept in 8 bits: 146 us,
// 136 so).
template <typename T>
__device__ __forceinline__ void as_words(Raw8<T>& r) {
  if constexpr (sizeof(T) == 2) {
    u32x4 w;
    __builtin_memcpy(&w, &r, 16);
    asm("" : "+v"(w));
    __builtin_memcpy(&r, &w, 16);
  }
}

// x from memory or (FORM) from its codes; a chunk of eight columns lies in
// one group.
template <typename T, bool FORM>
struct XChunk;
template <typename T>
struct XChunk<T, false> {
  Raw8<T> raw;
  template <int END>
  __device__ __forceinline__ void load(const LayerNormBackArgs& a, int64_t row, int c,
                                       int cols, int, int, int) {
    raw = load_chunk<END>((const T*)a.x + row * a.ldx, c, cols);
  }
  __device__ __forceinline__ void as_words() {}
  template <int END>
  __device__ __forceinline__ void get(float (&f)[8], int c, int cols) {
    settle<END>(raw, c, cols);
    widen(raw, f);
  }
};
template <typename T>
struct XChunk<T, true> {
  uint2 w;
  float step;
  template <int END>
  __device__ __forceinline__ void load(const LayerNormBackArgs& a, int64_t row, int c,
                                       int cols, int pitch, int groups, int glog) {
    w = make_uint2(0, 0);
    step = 0.f;
    if (c < cols) {
      w = *reinterpret_cast<const uint2*>(a.codes + row * pitch + c);
      step = a.steps[row * groups + (c >> glog)];
    }
  }
  __device__ __forceinline__ void as_words() { asm("" : "+v"(w.x), "+v"(w.y)); }
  template <int END>
  __device__ __forceinline__ void get(float (&f)[8], int, int) {
    decode8(w, step, f);
  }
};

// Streams of NT threads walk the rows; BT / NT streams share a workgroup and
// add their gradients in LDS.  Partial sums of workgroup b:
// ws[b][0][cols] (weight), ws[b][1][cols] (bias).  GRAD = false: dx only.
template <typename T, int NT, int R, int BT, bool FORM, bool GRAD, int END>
__global__ __launch_bounds__(BT) void k_layer_norm_backward(
    int64_t rows, int cols, int pitch, int groups, int glog, LayerNormBackArgs a) {
  constexpr int S = BT / NT;
  __shared__ float red_all[S][2][2][16];
  extern __shared__ float part[];  // S > 1: [S][NT * R * 8]
  const int stream = (int)threadIdx.x / NT, lane = (int)threadIdx.x % NT;
  float(*red)[2][16] = red_all[stream];
  // every stream of a workgroup takes the same number of turns (barriers)
  const int64_t stride = (int64_t)gridDim.x * S;
  const int64_t first = (int64_t)blockIdx.x * S;
  float w[R][8], gw[R][8], gb[R][8];
  Raw8<float> rw[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    rw[i] = load_vec<END>(a.weight, (lane + i * NT) * 8, cols, 1.f);
#pragma unroll
    for (int j = 0; j < 8; ++j) gw[i][j] = gb[i][j] = 0.f;
  }
  Raw8<T> rdy[R];
  XChunk<T, FORM> rx[R];
  float mean = 0.f, rstd = 0.f;
  auto fetch = [&](int64_t row) {
    if (row < rows) {
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const int c = (lane + i * NT) * 8;
        rdy[i] = load_chunk<END>((const T*)a.dy + row * a.lddy, c, cols);
        rx[i].template load<END>(a, row, c, cols, pitch, groups, glog);
      }
      mean = a.mean[row];
      rstd = a.rstd[row];
    }
  };
  fetch(first + stream);
#pragma unroll
  for (int i = 0; i < R; ++i)
    use_vec<END>(rw[i], a.weight, (lane + i * NT) * 8, cols, w[i]);
  const float n = (float)cols;
  int phase = 0;
  for (int64_t base = first; base < rows; base += stride) {
    const int64_t row = base + stream;
    const bool live = row < rows;
    float d[R][8], xh[R][8], s1 = 0.f, s2 = 0.f;
    const float mu = live ? mean : 0.f, rs = live ? rstd : 0.f;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int c = (lane + i * NT) * 8;
      // 1024 threads that keep gradients have no registers left for whole chunks
      // of dy, but for codes (norm step of 4096 x 12288 bf16 from the 8-bit form:
      // 297 us with dy kept, 290 with neither, 278 with codes)
      if constexpr (NT < 1024 || !GRAD || END != kWhole) as_words(rdy[i]);
      else rx[i].as_words();
      settle<END>(rdy[i], c, cols);
      widen(rdy[i], d[i]);
      rx[i].template get<END>(xh[i], c, cols);
      if (!live) {
#pragma unroll
        for (int j = 0; j < 8; ++j) d[i][j] = xh[i][j] = 0.f;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        // past the end dy is 0 and (x - mu) is not: only dy counts there, but
        // a NaN or an infinity in mu or rs has to stay out
        xh[i][j] = (xh[i][j] - mu) * rs;
        if (END != kWhole ? c + j >= cols : c >= cols) xh[i][j] = 0.f;
        if constexpr (GRAD) {
          gw[i][j] = fmaf(d[i][j], xh[i][j], gw[i][j]);
          gb[i][j] += d[i][j];
        }
        d[i][j] *= w[i][j];
        s1 += d[i][j];
        s2 = fmaf(d[i][j], xh[i][j], s2);
      }
    }
    fetch(row + stride);
    block_sum2<NT>(s1, s2, red, phase);
    phase ^= 1;
    const float m1 = s1 / n, m2 = s2 / n;
    if (live) {
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const int c = (lane + i * NT) * 8;
#pragma unroll
        for (int j = 0; j < 8; ++j) d[i][j] = rs * (d[i][j] - fmaf(xh[i][j], m2, m1));
        store_chunk<END>((T*)a.dx + row * a.lddx + c, narrow<T>(d[i]), cols - c);
      }
    }
  }
  if constexpr (GRAD) {
    float* o = a.ws + (int64_t)blockIdx.x * 2 * cols;
    if constexpr (S > 1) {
      // the streams' sums side by side in LDS, then added in order
      constexpr int W = NT * R * 8;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const auto& g = k == 0 ? gw : gb;
        if (k > 0) __syncthreads();
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
          for (int j = 0; j < 8; j += 4)
            *reinterpret_cast<f32x4*>(&part[stream * W + (lane + i * NT) * 8 + j]) =
                f32x4{g[i][j], g[i][j + 1], g[i][j + 2], g[i][j + 3]};
        __syncthreads();
        for (int c = (int)threadIdx.x; c < cols; c += BT) {
          float t = part[c];
#pragma unroll
          for (int s = 1; s < S; ++s) t += part[s * W + c];
          o[k * cols + c] = t;
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const int c = (lane + i * NT) * 8;
        store8(o + c, narrow<float>(gw[i]), cols - c);
        store8(o + cols + c, narrow<float>(gb[i]), cols - c);
      }
    }
  }
}

// Rows longer than the registers hold: dx reads each row twice; the column
// sums are a pass of their own over strips of 2048 columns.
template <typename T, bool FORM>
__global__ __launch_bounds__(1024) void k_layer_norm_backward_long(
    int64_t rows, int cols, int pitch, int groups, int glog, LayerNormBackArgs a) {
  __shared__ float red[2][2][16];
  int phase = 0;
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const float mu = a.mean[row], rs = a.rstd[row];
    float s1 = 0.f, s2 = 0.f, d[8], xh[8], w[8];
    XChunk<T, FORM> rx;
    for (int c = (int)threadIdx.x * 8; c < cols; c += 8192) {
      widen(load8((const T*)a.dy + row * a.lddy + c, cols - c), d);
      rx.template load<kRagged>(a, row, c, cols, pitch, groups, glog);
      rx.template get<kRagged>(xh, c, cols);
      use_vec<kRagged>(load_vec<kRagged>(a.weight, c, cols, 1.f), a.weight, c, cols, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float v = c + j < cols ? d[j] * w[j] : 0.f;
        const float h = c + j < cols ? (xh[j] - mu) * rs : 0.f;
        s1 += v;
        s2 = fmaf(v, h, s2);
      }
    }
    block_sum2<1024>(s1, s2, red, phase);
    phase ^= 1;
    const float m1 = s1 / (float)cols, m2 = s2 / (float)cols;
    for (int c = (int)threadIdx.x * 8; c < cols; c += 8192) {
      widen(load8((const T*)a.dy + row * a.lddy + c, cols - c), d);
      rx.template load<kRagged>(a, row, c, cols, pitch, groups, glog);
      rx.template get<kRagged>(xh, c, cols);
      use_vec<kRagged>(load_vec<kRagged>(a.weight, c, cols, 1.f), a.weight, c, cols, w);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        d[j] = rs * (d[j] * w[j] - fmaf((xh[j] - mu) * rs, m2, m1));
      store8((T*)a.dx + row * a.lddx + c, narrow<T>(d), cols - c);
    }
  }
}

// A workgroup takes every gridDim.y-th row.  64 of them at a time are added up
// by themselves, so that a sum's longest chain of additions is 64 and one more
// per 4096 rows, as in the shorter rows' pass.
template <typename T, bool FORM>
__global__ __launch_bounds__(256) void k_layer_norm_columns(
    int64_t rows, int cols, int pitch, int groups, int glog, LayerNormBackArgs a) {
  const int c = ((int)blockIdx.x * 256 + (int)threadIdx.x) * 8;
  if (c >= cols) return;
  float tw[8] = {}, tb[8] = {};
  for (int64_t row = blockIdx.y; row < rows;) {
    float gw[8] = {}, gb[8] = {}, d[8], xh[8];
    for (int n = 0; n < 64 && row < rows; ++n, row += gridDim.y) {
      const float mu = a.mean[row], rs = a.rstd[row];
      widen(load8((const T*)a.dy + row * a.lddy + c, cols - c), d);
      XChunk<T, FORM> rx;
      rx.template load<kRagged>(a, row, c, cols, pitch, groups, glog);
      rx.template get<kRagged>(xh, c, cols);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        gw[j] = fmaf(d[j], (xh[j] - mu) * rs, gw[j]);
        gb[j] += d[j];
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      tw[j] += gw[j];
      tb[j] += gb[j];
    }
  }
  float* o = a.ws + (int64_t)blockIdx.y * 2 * cols;
  store8(o + c, narrow<float>(tw), cols - c);
  store8(o + cols + c, narrow<float>(tb), cols - c);
}

// dweight / dbias <- beta * old + the parts' sum.  32 columns by 32 slices of
// the parts per workgroup; slices are added in order.
__global__ __launch_bounds__(1024) void k_layer_norm_reduce(
    int parts, int cols, const float* __restrict__ ws, float beta,
    float* __restrict__ dw, float* __restrict__ db) {
  __shared__ float sh[32][33];
  const int col = (int)blockIdx.x * 32 + (int)(threadIdx.x & 31);  // of 2 * cols
  const int slice = (int)threadIdx.x >> 5;
  float s = 0.f;
  if (col < 2 * cols)
    for (int p = slice; p < parts; p += 32) s += ws[(int64_t)p * 2 * cols + col];
  sh[slice][threadIdx.x & 31] = s;
  __syncthreads();
  if (slice == 0 && col < 2 * cols) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) s += sh[i][threadIdx.x & 31];
    float* o = col < cols ? dw : db;
    if (o) {
      o += col < cols ? col : col - cols;
      *o = beta == 0.f ? s : fmaf(beta, *o, s);
    }
  }
}

// ----------------------------------------------------------------- launch --
// Calls f<NT, R>() for a row of `cols` columns: NT * R * 8 >= cols.
template <typename F>
void by_columns(int64_t cols, F f) {
  if (cols <= 512) f.template operator()<64, 1>();
  else if (cols <= 1024) f.template operator()<64, 2>();
  else if (cols <= 2048) f.template operator()<256, 1>();
  else if (cols <= 4096) f.template operator()<256, 2>();
  else if (cols <= 8192) f.template operator()<512, 2>();
  else f.template operator()<1024, 2>();
}
constexpr int64_t kLongRow = 16384;

// Whether the rows' 8-bit form is written by the norm's own pass.
bool fused_form(const ActDims& A) {
  return A.cols <= kLongRow && (A.whole_row || A.group <= 512);
}

// Threads of a workgroup of the backward pass.
template <int NT>
constexpr int kBackThreads = NT < 512 ? 512 : NT;

// Workgroups of the backward pass: rows are shared out over at most as many
// threads as the chip holds at the kernel's occupancy.
int back_streams(const ActDims& A, int nt, int bt) {
  const int64_t s = bt / nt, need = (A.rows + s - 1) / s;
  const int64_t most = (int64_t)kCus * (1024 / bt);
  return (int)(need < most ? need : most);
}

int glog_of(const ActDims& A) {
  int g = 31;
  if (!A.whole_row)
    for (g = 0; (1 << g) < A.group;) ++g;
  return g;
}

template <typename T>
struct Forward {
  const ActDims& A;
  const LayerNormArgs& a;
  hipStream_t st;
  template <int NT, int R>
  void operator()() {
    constexpr int BT = NT < 256 ? 256 : NT, PER = BT / NT;
    const int64_t need = (A.rows + PER - 1) / PER, most = (int64_t)kCus * (2048 / BT);
    const unsigned g = (unsigned)(need < most ? need : most);
    auto* k = A.cols % 8 ? k_layer_norm<T, NT, R, kRagged> : k_layer_norm<T, NT, R, kWhole>;
    if constexpr (NT == 64 && R == 1)
      if (row_end(A.cols) == kTiny) k = k_layer_norm<T, NT, R, kTiny>;
    k<<<g, BT, 0, st>>>(A.rows, (int)A.cols, (int)A.pitch, A.groups,
                        A.whole_row ? -1 : glog_of(A) - 3, a);
  }
};

template <typename T>
int forward_t(const ActDims& A, const LayerNormArgs& a, hipStream_t st) {
  if (A.cols <= kLongRow) {
    by_columns(A.cols, Forward<T>{A, a, st});
  } else {
    k_layer_norm_long<T><<<(unsigned)(A.rows < 512 ? A.rows : 512), 1024, 0, st>>>(
        A.rows, (int)A.cols, a);
  }
  return (int)hipGetLastError();
}


template <typename T, bool FORM, bool GRAD>
struct Backward {
  const ActDims& A;
  const LayerNormBackArgs& a;
  hipStream_t st;
  int* parts;
  template <int NT, int R>
  void operator()() {
    constexpr int BT = kBackThreads<NT>, S = BT / NT;
    *parts = back_streams(A, NT, BT);
    const size_t lds = S > 1 && GRAD ? sizeof(float) * S * NT * R * 8 : 0;
    auto* k = A.cols % 8 ? k_layer_norm_backward<T, NT, R, BT, FORM, GRAD, kRagged>
                         : k_layer_norm_backward<T, NT, R, BT, FORM, GRAD, kWhole>;
    if constexpr (NT == 64 && R == 1)
      if (row_end(A.cols) == kTiny)
        k = k_layer_norm_backward<T, NT, R, BT, FORM, GRAD, kTiny>;
    k<<<(unsigned)*parts, BT, lds, st>>>(A.rows, (int)A.cols, (int)A.pitch, A.groups,
                                         glog_of(A), a);
  }
};

constexpr int kColumnSlices = 64;

template <typename T, bool FORM>
int backward_t(const ActDims& A, const LayerNormBackArgs& a, hipStream_t st) {
  const bool grad = a.dweight || a.dbias;
  int parts = 0;
  if (A.rows > 0) {
    if (A.cols <= kLongRow) {
      if (grad) by_columns(A.cols, Backward<T, FORM, true>{A, a, st, &parts});
      else by_columns(A.cols, Backward<T, FORM, false>{A, a, st, &parts});
    } else {
      // the column sums first: dx may be written over dy
      if (grad) {
        parts = (int)(A.rows < kColumnSlices ? A.rows : kColumnSlices);
        k_layer_norm_columns<T, FORM>
            <<<dim3(div_up(A.cols, 2048), parts), 256, 0, st>>>(
                A.rows, (int)A.cols, (int)A.pitch, A.groups, glog_of(A), a);
      }
      k_layer_norm_backward_long<T, FORM>
          <<<(unsigned)(A.rows < 512 ? A.rows : 512), 1024, 0, st>>>(
              A.rows, (int)A.cols, (int)A.pitch, A.groups, glog_of(A), a);
    }
  }
  int rc = (int)hipGetLastError();
  if (rc == 0 && grad) {
    k_layer_norm_reduce<<<div_up(2 * A.cols, 32), 1024, 0, st>>>(
        parts, (int)A.cols, a.ws, a.beta, a.dweight, a.dbias);
    rc = (int)hipGetLastError();
  }
  return rc;
}

struct Parts {
  const ActDims& A;
  int* parts;
  template <int NT, int R>
  void operator()() { *parts = back_streams(A, NT, kBackThreads<NT>); }
};

}  // namespace

int launch_layer_norm(const ActDims& A, const LayerNormArgs& in, hipStream_t st) {
  if (A.rows == 0) return 0;
  LayerNormArgs a = in;
  const bool fused = fused_form(A);
  if (!fused) {
    // x first: y may be written over it
    if (a.x_codes) {
      const int rc = launch_act_pack(A, a.x, a.ldx, a.x_codes, a.x_steps, st);
      if (rc) return rc;
    }
    a.x_codes = a.y_codes = nullptr;
  }
  int rc;
  switch (A.dtype) {
    case GQ_F32: rc = forward_t<float>(A, a, st); break;
    case GQ_BF16: rc = forward_t<__bf16>(A, a, st); break;
    default: rc = forward_t<_Float16>(A, a, st);
  }
  if (rc == 0 && !fused && in.y_codes)
    rc = launch_act_pack(A, a.y, a.ldy, in.y_codes, in.y_steps, st);
  return rc;
}

bool layer_norm_needs_y(const ActDims& A) { return !fused_form(A); }

int64_t layer_norm_workspace(const ActDims& A) {
  int parts = kColumnSlices;
  if (A.cols <= kLongRow) by_columns(A.cols, Parts{A, &parts});
  return (int64_t)parts * 2 * A.cols * (int64_t)sizeof(float);
}

int launch_layer_norm_backward(const ActDims& A, const LayerNormBackArgs& a,
                               hipStream_t st) {
  switch (A.dtype) {
    case GQ_F32:
      return a.codes ? backward_t<float, true>(A, a, st) : backward_t<float, false>(A, a, st);
    case GQ_BF16:
      return a.codes ? backward_t<__bf16, true>(A, a, st)
                     : backward_t<__bf16, false>(A, a, st);
    default:
      return a.codes ? backward_t<_Float16, true>(A, a, st)
                     : backward_t<_Float16, false>(A, a, st);
  }
}

}  // namespace gq
