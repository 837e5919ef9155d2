// act_api.hip — the C entry points of the 8-bit activation operators: argument
// validation on the host, then dispatch to the kernel launchers.  No
// allocation, no global state, no device synchronization.
#include "gq.h"

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "act.hpp"
#include "act_check.hpp"

extern "C" {

int gq_act_size(const gq_act* act, int64_t* code_bytes, int64_t* steps) {
  gq::ActDims A;
  const int rc = check_act(act, &A);
  if (rc) return rc;
  if (code_bytes) *code_bytes = A.rows * A.pitch;
  if (steps) *steps = A.rows * A.groups;
  return GQ_OK;
}

int gq_act_pack(const gq_act* act, const void* x, int64_t ldx, int8_t* codes,
                float* steps, void* stream) {
  gq::ActDims A;
  const int rc = check_act(act, &A);
  if (rc) return rc;
  Range rx, rc8, rs;
  if (!matrix(A, x, A.cols, ldx, &rx) || !form(A, codes, steps, &rc8, &rs))
    return GQ_EINVAL;
  if (any_overlap({rc8, rs}, {rx})) return GQ_EINVAL;
  return launch_status(gq::launch_act_pack(A, x, ldx, codes, steps,
                                           static_cast<hipStream_t>(stream)));
}

int gq_act_unpack(const gq_act* act, const int8_t* codes, const float* steps,
                  void* x, int64_t ldx, void* stream) {
  gq::ActDims A;
  const int rc = check_act(act, &A);
  if (rc) return rc;
  Range rx, rc8, rs;
  if (!matrix(A, x, A.cols, ldx, &rx) || !form(A, codes, steps, &rc8, &rs))
    return GQ_EINVAL;
  if (any_overlap({rx}, {rc8, rs})) return GQ_EINVAL;
  return launch_status(gq::launch_act_unpack(A, codes, steps, x, ldx,
                                             static_cast<hipStream_t>(stream)));
}

int gq_act_linear_workspace(const gq_act* act, int64_t out, int64_t* bytes) {
  gq::ActDims A;
  int rc = check_act(act, &A);
  if (rc == GQ_OK) rc = check_out(A, out);
  if (rc) return rc;
  if (!bytes) return GQ_EINVAL;
  rc = check_linear(A, out);
  if (rc) return rc;
  *bytes = gq::act_linear_workspace(A, out);
  return GQ_OK;
}

int gq_act_linear(const gq_act* act, int64_t out, const int8_t* codes,
                  const float* steps, const int8_t* w_codes,
                  const float* w_steps, const float* bias, void* y,
                  int64_t ldy, void* workspace, int64_t workspace_bytes,
                  void* stream) {
  gq::ActDims A;
  int rc = check_act(act, &A);
  if (rc == GQ_OK) rc = check_out(A, out);
  if (rc == GQ_OK) rc = check_linear(A, out);
  if (rc) return rc;
  Range ry, rc8, rs;
  if (!matrix(A, y, out, ldy, &ry) || !form(A, codes, steps, &rc8, &rs))
    return GQ_EINVAL;
  if (!w_codes || !aligned(w_codes, 16) || !vec(w_steps) || !vec_or_null(bias))
    return GQ_EINVAL;
  const int64_t need = gq::act_linear_workspace(A, out);
  if (!space(workspace, workspace_bytes, need)) return GQ_EINVAL;
  const Range ws = {workspace, need};
  if (any_overlap({ry, ws}, {rc8, rs, Range{w_codes, out * A.pitch},
                             Range{w_steps, 4 * out}, Range{bias, 4 * out}}))
    return GQ_EINVAL;
  return launch_status(gq::launch_act_linear(A, out, codes, steps, w_codes, w_steps,
                                             bias, y, ldy, workspace,
                                             static_cast<hipStream_t>(stream)));
}

int gq_act_wgrad_workspace(const gq_act* act, int64_t out, int64_t* bytes) {
  gq::ActDims A;
  int rc = check_act(act, &A);
  if (rc == GQ_OK) rc = check_out(A, out);
  if (rc) return rc;
  if (!bytes) return GQ_EINVAL;
  *bytes = gq::act_wgrad_workspace(A, out);
  return GQ_OK;
}

int gq_act_wgrad(const gq_act* act, int64_t out, const void* dy, int64_t lddy,
                 const int8_t* codes, const float* steps, float beta,
                 float* dweight, float* dbias, void* workspace,
                 int64_t workspace_bytes, void* stream) {
  gq::ActDims A;
  int rc = check_act(act, &A);
  if (rc == GQ_OK) rc = check_out(A, out);
  if (rc) return rc;
  Range rd, rc8, rs;
  if (!matrix(A, dy, out, lddy, &rd) || !form(A, codes, steps, &rc8, &rs))
    return GQ_EINVAL;
  if (!vec(dweight) || !vec_or_null(dbias) || !std::isfinite(beta)) return GQ_EINVAL;
  const int64_t need = gq::act_wgrad_workspace(A, out);
  if (!space(workspace, workspace_bytes, need)) return GQ_EINVAL;
  if (any_overlap({Range{dweight, 4 * out * A.cols}, Range{dbias, 4 * out},
                   Range{workspace, need}},
                  {rd, rc8, rs}))
    return GQ_EINVAL;
  return launch_status(gq::launch_act_wgrad(A, out, dy, lddy, codes, steps, beta,
                                            dweight, dbias, workspace,
                                            static_cast<hipStream_t>(stream)));
}

int gq_layer_norm(const gq_act* act, const void* x, int64_t ldx,
                  const float* weight, const float* bias, float eps, void* y,
                  int64_t ldy, float* mean, float* rstd, int8_t* x_codes,
                  float* x_steps, int8_t* y_codes, float* y_steps,
                  void* stream) {
  gq::ActDims A;
  const int rc = check_act(act, &A);
  if (rc) return rc;
  if (!(eps >= 0.f) || !std::isfinite(eps)) return GQ_EINVAL;
  Range rx, ry = {nullptr, 0}, xc = ry, xs = ry, yc = ry, ys = ry;
  if (!matrix(A, x, A.cols, ldx, &rx)) return GQ_EINVAL;
  if (y && !matrix(A, y, A.cols, ldy, &ry)) return GQ_EINVAL;
  if ((x_codes || x_steps) && !form(A, x_codes, x_steps, &xc, &xs)) return GQ_EINVAL;
  if ((y_codes || y_steps) && !form(A, y_codes, y_steps, &yc, &ys)) return GQ_EINVAL;
  if (!vec_or_null(weight) || !vec_or_null(bias) || !vec_or_null(mean) ||
      !vec_or_null(rstd))
    return GQ_EINVAL;
  if (A.rows > 0 && !y) {
    if (!y_codes) return GQ_EINVAL;
    if (gq::layer_norm_needs_y(A)) return GQ_EUNSUPPORTED;
  }
  const Range in_x = y && same(rx, ldx, ry, ldy) ? Range{nullptr, 0} : rx;
  if (any_overlap({ry, Range{mean, 4 * A.rows}, Range{rstd, 4 * A.rows}, xc, xs, yc, ys},
                  {in_x, Range{weight, 4 * A.cols}, Range{bias, 4 * A.cols}}))
    return GQ_EINVAL;
  // x written over by y must still not meet the other outputs
  if (any_overlap({Range{mean, 4 * A.rows}, Range{rstd, 4 * A.rows}, xc, xs, yc, ys}, {rx}))
    return GQ_EINVAL;
  gq::LayerNormArgs a = {x,    ldx,  weight,  bias,    eps,     y,      ldy,
                         mean, rstd, x_codes, x_steps, y_codes, y_steps};
  return launch_status(gq::launch_layer_norm(A, a, static_cast<hipStream_t>(stream)));
}

int gq_layer_norm_workspace(const gq_act* act, int64_t* bytes) {
  gq::ActDims A;
  const int rc = check_act(act, &A);
  if (rc) return rc;
  if (!bytes) return GQ_EINVAL;
  *bytes = gq::layer_norm_workspace(A);
  return GQ_OK;
}

int gq_layer_norm_backward(const gq_act* act, const void* dy, int64_t lddy,
                           const void* x, int64_t ldx, const int8_t* codes,
                           const float* steps, const float* mean,
                           const float* rstd, const float* weight, void* dx,
                           int64_t lddx, float beta, float* dweight,
                           float* dbias, void* workspace,
                           int64_t workspace_bytes, void* stream) {
  gq::ActDims A;
  const int rc = check_act(act, &A);
  if (rc) return rc;
  Range rd, rx = {nullptr, 0}, rc8 = rx, rs = rx, ro;
  if (!matrix(A, dy, A.cols, lddy, &rd) || !matrix(A, dx, A.cols, lddx, &ro))
    return GQ_EINVAL;
  if (codes || steps) {
    if (x || !form(A, codes, steps, &rc8, &rs)) return GQ_EINVAL;
  } else if (!matrix(A, x, A.cols, ldx, &rx)) {
    return GQ_EINVAL;
  }
  if (A.rows > 0 && (!vec(mean) || !vec(rstd))) return GQ_EINVAL;
  if (!vec_or_null(weight) || !vec_or_null(dweight) || !vec_or_null(dbias) ||
      !std::isfinite(beta))
    return GQ_EINVAL;
  const int64_t need = dweight || dbias ? gq::layer_norm_workspace(A) : 0;
  if (!space(workspace, workspace_bytes, need)) return GQ_EINVAL;
  const Range in_dy = same(rd, lddy, ro, lddx) ? Range{nullptr, 0} : rd;
  const Range in_x = same(rx, ldx, ro, lddx) ? Range{nullptr, 0} : rx;
  if (any_overlap({ro, Range{dweight, 4 * A.cols}, Range{dbias, 4 * A.cols},
                   Range{workspace, need}},
                  {in_dy, in_x, rc8, rs, Range{mean, 4 * A.rows},
                   Range{rstd, 4 * A.rows}, Range{weight, 4 * A.cols}}))
    return GQ_EINVAL;
  // what is left out of the overlap test above may still meet the others
  if (any_overlap({Range{dweight, 4 * A.cols}, Range{dbias, 4 * A.cols},
                   Range{workspace, need}},
                  {rd, rx}))
    return GQ_EINVAL;
  gq::LayerNormBackArgs a = {dy,   lddy, x,      ldx, codes, steps, mean,    rstd,
                             weight, dx, lddx, beta, dweight, dbias, (float*)workspace};
  return launch_status(
      gq::launch_layer_norm_backward(A, a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
