// adamw.hip — the AdamW step over all tensors of a flat parameter vector, and
// the norm that its gradient is clipped to.
//
//   g' = grad_scale g,  m <- b1 m + (1 - b1) g',  v <- b2 v + (1 - b2) g'^2
//   p <- p - (lr c1 m / (sqrt(v) c2 + eps) + lr wd p)
//
// fp32 arithmetic, each operation rounded by itself.  States are fp32, or 8-bit
// floats with a power-of-two step per 256 values: m in e4m3, v, which spans
// twice the range, in e5m2.  A step of the average changes v by 0.1 % where
// neighbouring codes lie 25 % apart, so rounding to the nearest code would
// stop it; codes are rounded at random, up with the probability of the place
// between them, which keeps the averages right in the mean, as long as the key is
// not one that gq_quantize rounded the gradient by (its words are these).  v > 0
// never becomes 0, since m / eps would follow.
//
// One pass over HBM: 28 bytes per value with fp32 states, 16.1 with 8-bit ones.
// A wave owns a block of 256 values, four to a lane, so a step needs only lane
// exchanges.  64 M values: 328 us with fp32 states, 5.5 TB/s; 203 us with 8-bit
// ones, 5.1 TB/s (a large copy: 5.05; the random numbers, the codes and IEEE
// division and root fit under the loads).  25.6 M values, clipped: 160 us in a loop;
// under the profiler the norm takes 34 there, behind an update that has written 307 MB,
// its join 5, the update 123.  By itself the norm takes 20, 5.1 TB/s (24 in a loop,
// with its join).
#include <type_traits>

#include "adamw.hpp"
#include "fp8.hpp"

namespace gq {
namespace {

// An 8-bit float whose code is the upper bits of a fp32 number, `BIAS` below
// its exponent: z = y 2^(BIAS - 127) has the code's bits from bit 23 - MAN up,
// and what lies below is the place between two codes.  MOST: the largest code;
// CAP: the largest step, as a biased exponent, with which it is a finite number.
struct E4M3 {
  static constexpr int MAN = 3, TOP = 8;
  static constexpr uint32_t MOST = 0x7e, CAP = 119 + 127;
  static constexpr float DOWN = 0x1p-120f, UP = 0x1p120f;
};
struct E5M2 {
  static constexpr int MAN = 2, TOP = 15;
  static constexpr uint32_t MOST = 0x7b, CAP = 112 + 127;
  static constexpr float DOWN = 0x1p-112f, UP = 0x1p112f;
};

template <typename F>
__device__ __forceinline__ float state_value(uint32_t code, float step) {
  const uint32_t bits = (code & 0x7fu) << (23 - F::MAN) | (code & 0x80u) << 24;
  return __uint_as_float(bits) * F::UP * step;
}

// r16: sixteen random bits.  Saturates, which only a step of CAP leaves to do.
template <typename F>
__device__ __forceinline__ uint32_t state_code(float x, const Step& s, uint32_t r16) {
  const float z = fabsf(x) * s.inv * F::DOWN;
  return min((__float_as_uint(z) + (r16 << (7 - F::MAN))) >> (23 - F::MAN), F::MOST);
}

struct Layer {
  float size, decay;   // lr c1, lr wd
};

template <int BITS, typename H>
__global__ __launch_bounds__(256) void k_adamw(AdamwArgs a, int64_t blocks, int64_t per) {
  const float gs = a.grad_scale ? *a.grad_scale : 1.f;
  if (!(fabsf(gs) <= 3.4028234664e38f)) return;   // not finite: no step
  float lr = a.lr, c1 = a.c1, c2 = a.c2;
  uint32_t step = a.step;
  if (a.schedule) {
    lr = a.schedule[0];
    c1 = a.schedule[1];
    c2 = a.schedule[2];
    step = __float_as_uint(a.schedule[3]);
  }
  const int lane = (int)threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  int64_t at = (int64_t)blockIdx.x * per + wave;
  const int64_t stop = min(((int64_t)blockIdx.x + 1) * per, blocks);
  if (at >= stop) return;

  // the layer of the wave's next value: the last that begins at or before it
  int layer = 0;
  if (a.offsets) {
    int hi = a.layers;
    while (hi - layer > 1) {
      const int mid = layer + (hi - layer) / 2;
      if (a.offsets[mid] <= at * kStateBlock) layer = mid;
      else hi = mid;
    }
  }
  auto values_of = [&](int l) {
    const float r = a.lr_scale ? lr * a.lr_scale[l] : lr;
    const float wd = a.decay ? a.decay[l] : a.weight_decay;
    return Layer{r * c1, r * wd};
  };
  Layer now = values_of(layer);
  int64_t layer_end = a.offsets && layer + 1 < a.layers ? a.offsets[layer + 1] : a.n;

  for (; at < stop; at += 4) {
    const int64_t base = at * kStateBlock, i0 = base + lane * 4;
    const int count = (int)min(max(a.n - i0, (int64_t)0), (int64_t)4);
    // layers that end at or before this block's first value are done with
    while (layer + 1 < a.layers && layer_end <= base) {
      ++layer;
      now = values_of(layer);
      layer_end = layer + 1 < a.layers ? a.offsets[layer + 1] : a.n;
    }
    Layer of[4] = {now, now, now, now};
    if (layer + 1 < a.layers && layer_end < min(base + kStateBlock, a.n)) {
      // more than one layer in this block: each value finds its own
      int l = layer;
      int64_t end = layer_end;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        while (l + 1 < a.layers && end <= i0 + j) {
          ++l;
          end = l + 1 < a.layers ? a.offsets[l + 1] : a.n;
        }
        of[j] = values_of(l);
      }
    }
    float g[4] = {}, p[4] = {}, m[4] = {}, v[4] = {};
    auto load = [&](const float* from, float (&to)[4]) {
      if (count == 4) {
        __builtin_memcpy(to, from + i0, 16);
      } else {
#pragma unroll
        for (int j = 0; j < 3; ++j)
          if (j < count) to[j] = from[i0 + j];
      }
    };
    auto store = [&](float* to, const float (&from)[4]) {
      if (count == 4) {
        __builtin_memcpy(to + i0, from, 16);
      } else {
#pragma unroll
        for (int j = 0; j < 3; ++j)
          if (j < count) to[i0 + j] = from[j];
      }
    };
    load(a.g, g);
    load(a.p, p);
    if constexpr (BITS == 32) {
      load((const float*)a.m, m);
      load((const float*)a.v, v);
    } else {
      uint32_t mc = 0, vc = 0;
      if (count == 4) {
        mc = *reinterpret_cast<const uint32_t*>((const uint8_t*)a.m + i0);
        vc = *reinterpret_cast<const uint32_t*>((const uint8_t*)a.v + i0);
      } else {
#pragma unroll
        for (int j = 0; j < 3; ++j)
          if (j < count) {
            mc |= (uint32_t)((const uint8_t*)a.m)[i0 + j] << (8 * j);
            vc |= (uint32_t)((const uint8_t*)a.v)[i0 + j] << (8 * j);
          }
      }
      const float ms = a.m_steps[at], vs = a.v_steps[at];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        m[j] = state_value<E4M3>(mc >> (8 * j), ms);
        v[j] = state_value<E5M2>(vc >> (8 * j), vs);
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float d = g[j] * gs;
      m[j] = m[j] * a.b1 + d * a.a1;
      v[j] = v[j] * a.b2 + d * a.a2 * d;
      const float root = sqrtf(v[j]) * c2 + a.eps;
      p[j] = p[j] - (of[j].size * m[j] / root + of[j].decay * p[j]);
    }
    store(a.p, p);
    if constexpr (!std::is_same_v<H, void>) {
      H h[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) h[j] = (H)p[j];
      if (count == 4) {
        __builtin_memcpy((H*)a.p16 + i0, h, sizeof(h));
      } else {
#pragma unroll
        for (int j = 0; j < 3; ++j)
          if (j < count) ((H*)a.p16)[i0 + j] = h[j];
      }
    }
    if constexpr (BITS == 32) {
      store((float*)a.m, m);
      store((float*)a.v, v);
    } else {
      uint32_t mm = 0, vm = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < count) {
          mm = max(mm, abs_bits(m[j]));
          vm = max(vm, abs_bits(v[j]));
        }
      const Step ms = float_step<E4M3::TOP>(lanes_max(mm, 64), E4M3::CAP);
      const Step vs = float_step<E5M2::TOP>(lanes_max(vm, 64), E5M2::CAP);
      const uint64_t q = (uint64_t)i0 / 4;
      const uint4 w = philox4x32_10(a.key0, a.key1, (uint32_t)q, (uint32_t)(q >> 32), step, 0);
      const uint32_t r[4] = {w.x, w.y, w.z, w.w};
      uint32_t mc = 0, vc = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t cm = state_code<E4M3>(m[j], ms, r[j] >> 16);
        const uint32_t cv = state_code<E5M2>(v[j], vs, r[j] & 0xffffu);
        if (ms.inv != 0.f) mc |= (cm | (m[j] < 0.f ? 0x80u : 0u)) << (8 * j);
        if (vs.inv != 0.f) vc |= (v[j] > 0.f ? max(cv, 1u) : cv) << (8 * j);
      }
      if (count == 4) {
        *reinterpret_cast<uint32_t*>((uint8_t*)a.m + i0) = mc;
        *reinterpret_cast<uint32_t*>((uint8_t*)a.v + i0) = vc;
      } else {
#pragma unroll
        for (int j = 0; j < 3; ++j)
          if (j < count) {
            ((uint8_t*)a.m)[i0 + j] = (uint8_t)(mc >> (8 * j));
            ((uint8_t*)a.v)[i0 + j] = (uint8_t)(vc >> (8 * j));
          }
      }
      if (lane == 0) {
        a.m_steps[at] = ms.step;
        a.v_steps[at] = vs.step;
      }
    }
  }
}

// ------------------------------------------------------------------ norm --
constexpr int kNormBlocks = 2048;

// Sums of squares in 64 bits, a part per workgroup, in the same order whatever
// runs beside.
__global__ __launch_bounds__(256) void k_grad_norm(int64_t n, const float* __restrict__ g,
                                                   double* __restrict__ parts) {
  __shared__ double red[4];
  double s0 = 0., s1 = 0., s2 = 0., s3 = 0.;
  const int64_t quads = n / 4;
  auto add = [&](const float4& w) {
    s0 = fma((double)w.x, (double)w.x, s0);
    s1 = fma((double)w.y, (double)w.y, s1);
    s2 = fma((double)w.z, (double)w.z, s2);
    s3 = fma((double)w.w, (double)w.w, s3);
  };
  const float4* from = reinterpret_cast<const float4*>(g);
  const int64_t stride = (int64_t)gridDim.x * 256;
  int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  for (; i + 3 * stride < quads; i += 4 * stride) {   // four loads in flight
    float4 w[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) w[u] = from[i + u * stride];
#pragma unroll
    for (int u = 0; u < 4; ++u) add(w[u]);
  }
  for (; i < quads; i += stride) add(from[i]);
  if (blockIdx.x == 0 && (int64_t)threadIdx.x < n - quads * 4) {
    const double w = (double)g[quads * 4 + threadIdx.x];
    s0 = fma(w, w, s0);
  }
  double s = group_reduce<64>((s0 + s1) + (s2 + s3), [](double a, double b) { return a + b; });
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) parts[blockIdx.x] = (red[0] + red[1]) + (red[2] + red[3]);
}

__global__ __launch_bounds__(256) void k_grad_norm_join(int parts, const double* __restrict__ ws,
                                                        float max_norm, float* norm,
                                                        float* scale) {
  __shared__ double red[4];
  double s = 0.;
  for (int i = (int)threadIdx.x; i < parts; i += 256) s += ws[i];
  s = group_reduce<64>(s, [](double a, double b) { return a + b; });
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x != 0) return;
  const double r = sqrt((red[0] + red[1]) + (red[2] + red[3]));
  if (norm) *norm = (float)r;
  if (scale) {
    // inf / inf and anything with NaN: NaN, so that no step is made
    const double f = r > (double)max_norm ? (double)max_norm / r : 1.;
    *scale = r - r == 0. ? (float)f : __uint_as_float(0x7fc00000u);
  }
}

int norm_blocks(int64_t n) {
  const int64_t b = (n / 4 + 255) / 256;
  return (int)(b < 1 ? 1 : b < kNormBlocks ? b : kNormBlocks);
}

template <int BITS>
int adamw_t(const AdamwArgs& a, int p16_dtype, hipStream_t st) {
  const int64_t blocks = (a.n + kStateBlock - 1) / kStateBlock;
  // Blocks of 256 values per workgroup of four waves: few, so that workgroups
  // that start together do not end together (64 M values, 32 bits, 4 / 16 / 64:
  // 329 / 346 / 361 us; 8 bits, which have more to compute and find their layer
  // first, 4 / 8 / 16 / 64: 213 / 202 / 200 / 216 us, 3 M values 15.7 / 15.4 / 17.0 /
  // 32), but no more workgroups than 2^22.
  int64_t per = BITS == 32 ? 4 : 8;
  const int64_t least = (blocks + (1 << 22) - 1) >> 22;
  if (per < least) per = (least + 3) / 4 * 4;
  const unsigned g = (unsigned)((blocks + per - 1) / per);
  if (!a.p16) k_adamw<BITS, void><<<g, 256, 0, st>>>(a, blocks, per);
  else if (p16_dtype == GQ_BF16) k_adamw<BITS, __bf16><<<g, 256, 0, st>>>(a, blocks, per);
  else k_adamw<BITS, _Float16><<<g, 256, 0, st>>>(a, blocks, per);
  return (int)hipGetLastError();
}

}  // namespace

int launch_adamw(const AdamwArgs& a, int bits, int p16_dtype, hipStream_t st) {
  return bits == 32 ? adamw_t<32>(a, p16_dtype, st) : adamw_t<8>(a, p16_dtype, st);
}

int64_t grad_norm_workspace(int64_t n) { return 8 * (int64_t)norm_blocks(n); }

int launch_grad_norm(int64_t n, const float* g, float max_norm, float* norm, float* scale,
                     void* ws, hipStream_t st) {
  const int b = norm_blocks(n);
  k_grad_norm<<<b, 256, 0, st>>>(n, g, (double*)ws);
  int rc = (int)hipGetLastError();
  if (rc == 0) {
    k_grad_norm_join<<<1, 256, 0, st>>>(b, (const double*)ws, max_norm, norm, scale);
    rc = (int)hipGetLastError();
  }
  return rc;
}

}  // namespace gq
