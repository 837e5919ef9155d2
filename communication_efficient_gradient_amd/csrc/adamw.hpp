// adamw.hpp — launchers of the optimizer's step.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gq.h"

namespace gq {

constexpr int kStateBlock = 256;   // values of an 8-bit state that share a step

struct AdamwArgs {
  int64_t n;
  int layers;
  const int64_t* offsets;              // or NULL: one layer
  const float *lr_scale, *decay;       // of each layer, or NULL
  const float *g, *grad_scale;
  float* p;
  void *m, *v;
  float *m_steps, *v_steps;
  void* p16;
  const float* schedule;               // lr, c1, c2, step; or NULL
  float lr, c1, c2;                    // c1 = 1 / (1 - b1^t), c2 = 1 / sqrt(1 - b2^t)
  float b1, b2, a1, a2;                // a = 1 - b
  float eps, weight_decay;
  uint32_t step, key0, key1;
};

int launch_adamw(const AdamwArgs& a, int bits, int p16_dtype, hipStream_t st);

int64_t grad_norm_workspace(int64_t n);
int launch_grad_norm(int64_t n, const float* g, float max_norm, float* norm, float* scale,
                     void* ws, hipStream_t st);

}  // namespace gq
