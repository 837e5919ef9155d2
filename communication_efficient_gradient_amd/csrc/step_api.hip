// step_api.hip — the C entry points of the 8-bit floating point products and of
// the optimizer's step: argument validation on the host, then dispatch to the
// kernel launchers.  No allocation, no global state, no device synchronization.
#include "gq.h"

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "act_check.hpp"
#include "adamw.hpp"
#include "fp8.hpp"

namespace {

constexpr int64_t kMaxValues = int64_t(1) << 38;
constexpr int64_t kMaxWgradTiles = int64_t(1) << 22;  // of 128 x 128 results
constexpr int64_t kMaxWgradRows = int64_t(1) << 34;

// The form has a step per 128 columns.
int check_fp8(const gq_act* act, gq::ActDims* A) {
  const int rc = check_act(act, A);
  if (rc) return rc;
  return act->group == gq::kFp8Block ? GQ_OK : GQ_EUNSUPPORTED;
}

// `experts` weights [out, cols], and the tokens' table of them.
int check_experts(const gq::ActDims& A, int64_t out, int32_t experts) {
  if (experts < 1) return GQ_EINVAL;
  const int rc = check_out(A, out);
  if (rc) return rc;
  if (experts > gq::kMaxExperts) return GQ_EUNSUPPORTED;
  return out * A.cols > kMaxElements / experts ? GQ_EINVAL : GQ_OK;
}

bool table(const int64_t* offsets, int32_t experts) {
  return offsets ? aligned(offsets, 8) : experts == 1;
}

int64_t blocks_of(int64_t n) { return (n + gq::kFp8Block - 1) / gq::kFp8Block; }

int check_fp8_linear(const gq::ActDims& A, int64_t out, int32_t experts) {
  const int rc = check_experts(A, out, experts);
  if (rc) return rc;
  // tiles that one launch numbers
  return (A.rows + 63) / 64 > kMaxTiles / ((out + 63) / 64) ? GQ_EUNSUPPORTED : GQ_OK;
}

int check_fp8_wgrad(const gq::ActDims& A, int64_t out, int32_t experts) {
  const int rc = check_experts(A, out, experts);
  if (rc) return rc;
  if (A.rows > kMaxWgradRows) return GQ_EUNSUPPORTED;
  return blocks_of(out) * blocks_of(A.cols) > kMaxWgradTiles / experts ? GQ_EUNSUPPORTED : GQ_OK;
}

Range codes_range(const uint8_t* p, int64_t rows, int64_t cols) {
  return {p, rows * ((cols + 15) / 16 * 16)};
}

// A form of activations: both buffers.
bool fp8_form(const gq::ActDims& A, const uint8_t* codes, const float* steps, Range* c,
              Range* s) {
  return form(A, reinterpret_cast<const int8_t*>(codes), steps, c, s);
}

// A weight's codes and steps: both, or none where that is allowed.
bool weight_form(const uint8_t* codes, const float* steps) {
  return codes && steps && aligned(codes, 16) && aligned(steps, 4);
}

int check_adamw(const gq_adamw_desc* d) {
  if (!d || !std::isfinite((float)d->lr) || !std::isfinite((float)d->weight_decay))
    return GQ_EINVAL;
  if (!(d->beta1 >= 0. && d->beta1 < 1.) || !(d->beta2 >= 0. && d->beta2 < 1.)) return GQ_EINVAL;
  if (!((float)d->eps > 0.f) || !std::isfinite((float)d->eps)) return GQ_EINVAL;
  return d->bits == 32 || d->bits == 8 ? GQ_OK : GQ_EUNSUPPORTED;
}

}  // namespace

extern "C" {

int gq_block_pack(const gq_act* act, const void* x, int64_t ldx, uint8_t* codes, float* steps,
                void* stream) {
  gq::ActDims A;
  const int rc = check_fp8(act, &A);
  if (rc) return rc;
  Range rx, rc8, rs;
  if (!matrix(A, x, A.cols, ldx, &rx) || !fp8_form(A, codes, steps, &rc8, &rs))
    return GQ_EINVAL;
  if (any_overlap({rc8, rs}, {rx})) return GQ_EINVAL;
  return launch_status(
      gq::launch_fp8_pack(A, x, ldx, codes, steps, static_cast<hipStream_t>(stream)));
}

int gq_block_unpack(const gq_act* act, const uint8_t* codes, const float* steps, void* x,
                  int64_t ldx, void* stream) {
  gq::ActDims A;
  const int rc = check_fp8(act, &A);
  if (rc) return rc;
  Range rx, rc8, rs;
  if (!matrix(A, x, A.cols, ldx, &rx) || !fp8_form(A, codes, steps, &rc8, &rs))
    return GQ_EINVAL;
  if (any_overlap({rx}, {rc8, rs})) return GQ_EINVAL;
  return launch_status(
      gq::launch_fp8_unpack(A, codes, steps, x, ldx, static_cast<hipStream_t>(stream)));
}

int gq_block_pack_weight(const gq_act* weight, int32_t experts, const void* w, uint8_t* codes,
                       float* steps, uint8_t* t_codes, float* t_steps, void* stream) {
  gq::ActDims A;
  int rc = check_fp8(weight, &A);
  if (rc) return rc;
  const int64_t out = A.rows;
  if (experts < 1 || out < 1 || out > kMaxCols) return GQ_EINVAL;
  if (experts > gq::kMaxExperts) return GQ_EUNSUPPORTED;
  if (out * A.cols > kMaxElements / experts) return GQ_EINVAL;
  if (!w || !aligned(w, (uintptr_t)dtype_bytes(A.dtype))) return GQ_EINVAL;
  const bool here = codes || steps, turned = t_codes || t_steps;
  if (!here && !turned) return GQ_EINVAL;
  if (here && !weight_form(codes, steps)) return GQ_EINVAL;
  if (turned && !weight_form(t_codes, t_steps)) return GQ_EINVAL;
  const int64_t step_bytes = 4 * experts * blocks_of(out) * blocks_of(A.cols);
  if (any_overlap({codes_range(codes, experts * out, A.cols), Range{steps, step_bytes},
                   codes_range(t_codes, experts * A.cols, out), Range{t_steps, step_bytes}},
                  {Range{w, experts * out * A.cols * dtype_bytes(A.dtype)}}))
    return GQ_EINVAL;
  return launch_status(gq::launch_fp8_pack_weight(A, experts, w, codes, steps, t_codes, t_steps,
                                                  static_cast<hipStream_t>(stream)));
}

int gq_block_linear_workspace(const gq_act* act, int64_t out, int32_t experts, int64_t* bytes) {
  gq::ActDims A;
  int rc = check_fp8(act, &A);
  if (rc == GQ_OK) rc = check_fp8_linear(A, out, experts);
  if (rc) return rc;
  if (!bytes) return GQ_EINVAL;
  *bytes = gq::fp8_linear_workspace(A, out, experts);
  return GQ_OK;
}

int gq_block_linear(const gq_act* act, int64_t out, int32_t experts, const int64_t* offsets,
                  const uint8_t* codes, const float* steps, const uint8_t* w_codes,
                  const float* w_steps, const float* bias, void* y, int64_t ldy,
                  void* workspace, int64_t workspace_bytes, void* stream) {
  gq::ActDims A;
  int rc = check_fp8(act, &A);
  if (rc == GQ_OK) rc = check_fp8_linear(A, out, experts);
  if (rc) return rc;
  Range ry, rc8, rs;
  if (!matrix(A, y, out, ldy, &ry) || !fp8_form(A, codes, steps, &rc8, &rs)) return GQ_EINVAL;
  if (!weight_form(w_codes, w_steps) || !vec_or_null(bias) || !table(offsets, experts))
    return GQ_EINVAL;
  const int64_t need = gq::fp8_linear_workspace(A, out, experts);
  if (!space(workspace, workspace_bytes, need)) return GQ_EINVAL;
  if (any_overlap(
          {ry, Range{workspace, need}},
          {rc8, rs, codes_range(w_codes, experts * out, A.cols),
           Range{w_steps, 4 * experts * blocks_of(out) * A.groups},
           Range{bias, 4 * experts * out}, Range{offsets, 8 * ((int64_t)experts + 1)}}))
    return GQ_EINVAL;
  return launch_status(gq::launch_fp8_linear(A, out, experts, offsets, codes, steps, w_codes,
                                             w_steps, bias, y, ldy, workspace,
                                             static_cast<hipStream_t>(stream)));
}

int gq_block_wgrad_workspace(const gq_act* act, int64_t out, int32_t experts, int64_t* bytes) {
  gq::ActDims A;
  int rc = check_fp8(act, &A);
  if (rc == GQ_OK) rc = check_fp8_wgrad(A, out, experts);
  if (rc) return rc;
  if (!bytes) return GQ_EINVAL;
  *bytes = gq::fp8_wgrad_workspace(A, out, experts);
  return GQ_OK;
}

int gq_block_wgrad(const gq_act* act, int64_t out, int32_t experts, const int64_t* offsets,
                 const void* dy, int64_t lddy, const uint8_t* codes, const float* steps,
                 float beta, float* dweight, float* dbias, void* workspace,
                 int64_t workspace_bytes, void* stream) {
  gq::ActDims A;
  int rc = check_fp8(act, &A);
  if (rc == GQ_OK) rc = check_fp8_wgrad(A, out, experts);
  if (rc) return rc;
  Range rd, rc8, rs;
  if (!matrix(A, dy, out, lddy, &rd) || !fp8_form(A, codes, steps, &rc8, &rs)) return GQ_EINVAL;
  if (!vec(dweight) || !vec_or_null(dbias) || !std::isfinite(beta) || !table(offsets, experts))
    return GQ_EINVAL;
  const int64_t need = gq::fp8_wgrad_workspace(A, out, experts);
  if (!space(workspace, workspace_bytes, need)) return GQ_EINVAL;
  if (any_overlap({Range{dweight, 4 * experts * out * A.cols}, Range{dbias, 4 * experts * out},
                   Range{workspace, need}},
                  {rd, rc8, rs, Range{offsets, 8 * ((int64_t)experts + 1)}}))
    return GQ_EINVAL;
  return launch_status(gq::launch_fp8_wgrad(A, out, experts, offsets, dy, lddy, codes, steps,
                                            beta, dweight, dbias, workspace,
                                            static_cast<hipStream_t>(stream)));
}

int gq_adamw(const gq_adamw_desc* desc, int64_t n, int32_t nl, const int64_t* layer_offsets,
             const float* lr_scale, const float* decay, const float* g, const float* grad_scale,
             int64_t step, const float* schedule, float* p, void* m, float* m_steps, void* v,
             float* v_steps, void* p16, int32_t p16_dtype, uint64_t seed, void* stream) {
  const int rc = check_adamw(desc);
  if (rc) return rc;
  if (n < 1 || n > kMaxValues || nl < 1) return GQ_EINVAL;
  if (step < 1 || step > (int64_t)UINT32_MAX) return GQ_EINVAL;
  if (layer_offsets ? !aligned(layer_offsets, 8) : nl != 1) return GQ_EINVAL;
  if (!vec_or_null(lr_scale) || !vec_or_null(decay) || !vec_or_null(grad_scale) ||
      !aligned(schedule, 16))
    return GQ_EINVAL;
  if (!g || !p || !m || !v || !aligned(g, 16) || !aligned(p, 16) || !aligned(m, 16) ||
      !aligned(v, 16))
    return GQ_EINVAL;
  const bool small = desc->bits == 8;
  if (small ? !vec(m_steps) || !vec(v_steps) : m_steps || v_steps) return GQ_EINVAL;
  if (p16) {
    if (p16_dtype != GQ_BF16 && p16_dtype != GQ_F16) return GQ_EUNSUPPORTED;
    if (!aligned(p16, 16)) return GQ_EINVAL;
  }
  const int64_t state = small ? n : 4 * n;
  const int64_t state_steps = 4 * ((n + gq::kStateBlock - 1) / gq::kStateBlock);
  if (any_overlap({Range{p, 4 * n}, Range{m, state}, Range{v, state},
                   Range{m_steps, state_steps}, Range{v_steps, state_steps}, Range{p16, 2 * n}},
                  {Range{g, 4 * n}, Range{layer_offsets, 8 * ((int64_t)nl + 1)},
                   Range{lr_scale, 4 * (int64_t)nl}, Range{decay, 4 * (int64_t)nl},
                   Range{grad_scale, 4}, Range{schedule, 16}}))
    return GQ_EINVAL;
  gq::AdamwArgs a = {};
  a.n = n;
  a.layers = nl;
  a.offsets = layer_offsets;
  a.lr_scale = lr_scale;
  a.decay = decay;
  a.g = g;
  a.grad_scale = grad_scale;
  a.p = p;
  a.m = m;
  a.v = v;
  a.m_steps = m_steps;
  a.v_steps = v_steps;
  a.p16 = p16;
  a.schedule = schedule;
  a.lr = (float)desc->lr;
  a.c1 = (float)(1. / (1. - std::pow(desc->beta1, (double)step)));
  a.c2 = (float)(1. / std::sqrt(1. - std::pow(desc->beta2, (double)step)));
  a.b1 = (float)desc->beta1;
  a.b2 = (float)desc->beta2;
  a.a1 = (float)(1. - desc->beta1);
  a.a2 = (float)(1. - desc->beta2);
  a.eps = (float)desc->eps;
  a.weight_decay = (float)desc->weight_decay;
  a.step = (uint32_t)step;
  a.key0 = (uint32_t)seed;
  a.key1 = (uint32_t)(seed >> 32);
  return launch_status(
      gq::launch_adamw(a, desc->bits, p16_dtype, static_cast<hipStream_t>(stream)));
}

int gq_grad_norm_workspace(int64_t n, int64_t* bytes) {
  if (n < 1 || n > kMaxValues || !bytes) return GQ_EINVAL;
  *bytes = gq::grad_norm_workspace(n);
  return GQ_OK;
}

int gq_grad_norm(int64_t n, const float* g, float max_norm, float* norm, float* scale,
                 void* workspace, int64_t workspace_bytes, void* stream) {
  if (n < 1 || n > kMaxValues || !g || !aligned(g, 16)) return GQ_EINVAL;
  if (!(max_norm > 0.f)) return GQ_EINVAL;
  if ((!norm && !scale) || !vec_or_null(norm) || !vec_or_null(scale)) return GQ_EINVAL;
  const int64_t need = gq::grad_norm_workspace(n);
  if (!space(workspace, workspace_bytes, need)) return GQ_EINVAL;
  if (any_overlap({Range{norm, 4}, Range{scale, 4}, Range{workspace, need}}, {Range{g, 4 * n}}))
    return GQ_EINVAL;
  return launch_status(gq::launch_grad_norm(n, g, max_norm, norm, scale, workspace,
                                            static_cast<hipStream_t>(stream)));
}

}  // extern "C"
