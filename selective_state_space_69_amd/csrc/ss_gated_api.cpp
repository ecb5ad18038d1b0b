// C-ABI entry points of a gated recurrent block's operators: the gated linear
// recurrence, the gated half of a feed-forward block, projections in 8-bit integers.
// As for the scan, validation is plain host logic that runs before any HIP call; then
// the device is checked and the kernels are launched.
#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "ss_internal.h"

namespace ss {
namespace {

constexpr int64_t kMaxElems = int64_t(1) << 40;
constexpr int64_t kMaxDim = int64_t(1) << 20;
// of 64 channels, two workgroups of 512 threads each: a grid's threads stay below 2^32
constexpr int64_t kMaxGroups = int64_t(1) << 21;

bool row_aligned(const void* p, int64_t stride, int32_t dtype) {
  return !p || aligned(p, row_align(stride, dtype));
}

// whether two of the outputs, or an output and an input, are one buffer (NULL never is)
bool aliased(std::initializer_list<const void*> outs, std::initializer_list<const void*> ins) {
  for (auto a = outs.begin(); a != outs.end(); ++a) {
    if (!*a) continue;
    for (auto b = outs.begin(); b != a; ++b)
      if (*b == *a) return true;
    for (const void* i : ins)
      if (i == *a) return true;
  }
  return false;
}

bool bad_workspace(const void* workspace, size_t ws_bytes, size_t need) {
  return need > 0 && (!workspace || ws_bytes < need || !aligned(workspace, kAlign));
}

int check_rec(const ss_rec_desc_t* d) {
  if (!d) return SS_ERR_INVALID_ARG;
  if (d->batch < 1 || d->seqlen < 1 || d->seqlen > INT32_MAX || d->dim < 1 || d->dim > kMaxDim)
    return SS_ERR_INVALID_ARG;
  if (d->batch > kMaxGroups / ((d->dim + 63) / 64)) return SS_ERR_INVALID_ARG;
  for (int64_t s : {d->x_stride, d->r_stride, d->i_stride, d->z_stride}) {
    if (bad_stride(s, d->dim, kMaxDim)) return SS_ERR_INVALID_ARG;
    if (d->seqlen > kMaxElems / d->batch / (s ? s : d->dim)) return SS_ERR_INVALID_ARG;
  }
  if (!valid_dtype(d->in_dtype) || !valid_dtype(d->out_dtype)) return SS_ERR_UNSUPPORTED;
  if (!(d->decay > 0.0f && std::isfinite(d->decay)) || d->reserved != 0) return SS_ERR_INVALID_ARG;
  return SS_OK;
}

// x, r, i, z of a recurrence's call
int check_rec_inputs(const ss_rec_desc_t* d, const void* x, const void* r, const void* i,
                     const float* lam, const void* z) {
  const int rc = check_rec(d);
  if (rc != SS_OK) return rc;
  if (!x || !r || !i || !lam) return SS_ERR_INVALID_ARG;
  if (!row_aligned(x, d->x_stride, d->in_dtype) || !row_aligned(r, d->r_stride, d->in_dtype) ||
      !row_aligned(i, d->i_stride, d->in_dtype) || !row_aligned(z, d->z_stride, d->in_dtype))
    return SS_ERR_INVALID_ARG;
  return all_aligned({lam}) ? SS_OK : SS_ERR_INVALID_ARG;
}

constexpr int64_t kMaxRows = int64_t(1) << 28;       // 64 x 64 tiles of any product stay below 2^24
constexpr int64_t kMaxMatrix = int64_t(1) << 35;     // elements

int check_glu(const ss_glu_desc_t* d, int op) {
  if (!d) return SS_ERR_INVALID_ARG;
  if (op != SS_GLU_FWD && op != SS_GLU_BWD) return SS_ERR_INVALID_ARG;
  if (d->rows < 1 || d->rows > kMaxRows || d->in_dim < 1 || d->in_dim > kMaxDim ||
      d->out_dim < 1 || d->out_dim > kMaxDim / 2)
    return SS_ERR_INVALID_ARG;
  if (d->rows > kMaxMatrix / d->in_dim || d->rows > kMaxMatrix / (2 * d->out_dim) ||
      2 * d->out_dim > kMaxMatrix / d->in_dim)
    return SS_ERR_INVALID_ARG;
  if (bad_stride(d->x_stride, d->in_dim, kMaxDim)) return SS_ERR_INVALID_ARG;
  if (!valid_dtype(d->in_dtype) || !valid_dtype(d->out_dtype) ||
      (op == SS_GLU_BWD && !valid_dtype(d->grad_dtype)))
    return SS_ERR_UNSUPPORTED;
  if (d->act != SS_ACT_NONE && d->act != SS_ACT_SILU && d->act != SS_ACT_GELU)
    return SS_ERR_UNSUPPORTED;
  return SS_OK;
}

int check_q8_pack(const ss_q8_pack_desc_t* d) {
  if (!d) return SS_ERR_INVALID_ARG;
  if (d->rows < 1 || d->rows > INT32_MAX || d->dim < 1 || d->dim > kMaxDim)
    return SS_ERR_INVALID_ARG;
  if (bad_stride(d->x_stride, d->dim, kMaxDim) || bad_stride(d->q_stride, d->dim, kMaxDim) ||
      d->reserved != 0)
    return SS_ERR_INVALID_ARG;
  return valid_dtype(d->dtype) ? SS_OK : SS_ERR_UNSUPPORTED;
}

int check_q8(const ss_q8_desc_t* d) {
  if (!d) return SS_ERR_INVALID_ARG;
  if (d->rows < 1 || d->rows > kMaxRows || d->in_dim < 1 || d->in_dim > (1 << 16) ||
      d->out_dim < 1 || d->out_dim > kMaxDim)
    return SS_ERR_INVALID_ARG;
  if (d->rows > kMaxMatrix / d->in_dim || d->rows > kMaxMatrix / d->out_dim)
    return SS_ERR_INVALID_ARG;
  if (bad_stride(d->x_stride, d->in_dim, kMaxDim) || bad_stride(d->w_stride, d->in_dim, kMaxDim) ||
      d->reserved != 0)
    return SS_ERR_INVALID_ARG;
  if (!valid_dtype(d->out_dtype) || !valid_dtype(d->res_dtype)) return SS_ERR_UNSUPPORTED;
  if (d->act < SS_ACT_NONE || d->act > SS_ACT_SOFTPLUS) return SS_ERR_UNSUPPORTED;
  return SS_OK;
}

int done(int hip) { return hip == 0 ? SS_OK : SS_ERR_HIP; }

}  // namespace
}  // namespace ss

using namespace ss;

extern "C" {

size_t ss_rec_workspace_bytes(const ss_rec_desc_t* desc, int op) {
  if (check_rec(desc) != SS_OK || (op != SS_REC_FWD && op != SS_REC_BWD)) return 0;
  return plan_rec(*desc, op).bytes;
}

int ss_rec_fwd(const ss_rec_desc_t* desc, const void* x, const void* r, const void* i,
               const float* lam, const void* z, const float* h0, const uint8_t* starts,
               const int32_t* lengths, void* y, float* h_last, float* states, void* workspace,
               size_t ws_bytes, void* stream) {
  int rc = check_rec_inputs(desc, x, r, i, lam, z);
  if (rc != SS_OK) return rc;
  if (!y || aliased({y, h_last, states}, {x, r, i, lam, z, starts, lengths}) ||
      aliased({y, states}, {h0}))
    return SS_ERR_INVALID_ARG;
  if (!all_aligned({h0, lengths, y, h_last, states})) return SS_ERR_INVALID_ARG;
  const RecPlan plan = plan_rec(*desc, SS_REC_FWD);
  if (bad_workspace(workspace, ws_bytes, plan.bytes)) return SS_ERR_WORKSPACE;
  if ((rc = check_device()) != SS_OK) return rc;
  return done(launch_rec_fwd(*desc, plan, x, r, i, lam, z, h0, starts, lengths, y, h_last, states,
                             static_cast<char*>(workspace), stream));
}

int ss_rec_bwd(const ss_rec_desc_t* desc, const void* x, const void* r, const void* i,
               const float* lam, const void* z, const uint8_t* starts, const int32_t* lengths,
               const float* states, const void* dy, const float* dh_last, void* dx, void* dr,
               void* di, void* dz, float* dlam, float* dh0, void* workspace, size_t ws_bytes,
               void* stream) {
  int rc = check_rec_inputs(desc, x, r, i, lam, z);
  if (rc != SS_OK) return rc;
  if (!states || !dy || !dx || !dr || !di || !dlam || (z != nullptr) != (dz != nullptr))
    return SS_ERR_INVALID_ARG;
  if (aliased({dx, dr, di, dz, dlam, dh0},
              {x, r, i, lam, z, starts, lengths, states, dy, dh_last}))
    return SS_ERR_INVALID_ARG;
  if (!all_aligned({lengths, states, dy, dh_last, dx, dr, di, dz, dlam, dh0}))
    return SS_ERR_INVALID_ARG;
  const RecPlan plan = plan_rec(*desc, SS_REC_BWD);
  if (bad_workspace(workspace, ws_bytes, plan.bytes)) return SS_ERR_WORKSPACE;
  if ((rc = check_device()) != SS_OK) return rc;
  return done(launch_rec_bwd(*desc, plan, x, r, i, lam, z, starts, lengths, states, dy, dh_last,
                             dx, dr, di, dz, dlam, dh0, static_cast<char*>(workspace), stream));
}

int ss_rec_step(const ss_rec_desc_t* desc, float* h, const void* x, const void* r, const void* i,
                const float* lam, const void* z, void* y, void* stream) {
  int rc = check_rec_inputs(desc, x, r, i, lam, z);
  if (rc != SS_OK) return rc;
  if (desc->seqlen != 1 || !h || !y || aliased({h, y}, {x, r, i, lam, z}))
    return SS_ERR_INVALID_ARG;
  if (!all_aligned({h, y})) return SS_ERR_INVALID_ARG;
  if ((rc = check_device()) != SS_OK) return rc;
  return done(launch_rec_step(*desc, h, x, r, i, lam, z, y, stream));
}

size_t ss_glu_workspace_bytes(const ss_glu_desc_t* desc, int op) {
  if (check_glu(desc, op) != SS_OK) return 0;
  return plan_glu(*desc, op).bytes;
}

int ss_glu_fwd(const ss_glu_desc_t* desc, const void* x, const void* w, const float* bias, void* y,
               void* pre, void* workspace, size_t ws_bytes, void* stream) {
  int rc = check_glu(desc, SS_GLU_FWD);
  if (rc != SS_OK) return rc;
  if (!x || !w || !y || aliased({y, pre}, {x, w, bias})) return SS_ERR_INVALID_ARG;
  if (!row_aligned(x, desc->x_stride, desc->in_dtype) || !all_aligned({w, bias, y, pre}))
    return SS_ERR_INVALID_ARG;
  const LinearPlan plan = plan_glu(*desc, SS_GLU_FWD);
  if (bad_workspace(workspace, ws_bytes, plan.bytes)) return SS_ERR_WORKSPACE;
  if ((rc = check_device()) != SS_OK) return rc;
  return done(launch_glu_fwd(*desc, plan, x, w, bias, y, pre, static_cast<char*>(workspace),
                             stream));
}

int ss_glu_bwd(const ss_glu_desc_t* desc, const void* x, const void* w, const void* pre,
               const void* dy, void* dx, void* dw, float* dbias, void* workspace, size_t ws_bytes,
               void* stream) {
  int rc = check_glu(desc, SS_GLU_BWD);
  if (rc != SS_OK) return rc;
  if (!w || !pre || !dy || (!dx && !dw && !dbias) || (dw && !x)) return SS_ERR_INVALID_ARG;
  if (aliased({dx, dw, dbias}, {x, w, pre, dy})) return SS_ERR_INVALID_ARG;
  if (!row_aligned(x, desc->x_stride, desc->in_dtype) ||
      !all_aligned({w, pre, dy, dx, dw, dbias}))
    return SS_ERR_INVALID_ARG;
  const LinearPlan plan = plan_glu(*desc, SS_GLU_BWD);
  if (bad_workspace(workspace, ws_bytes, plan.bytes)) return SS_ERR_WORKSPACE;
  if ((rc = check_device()) != SS_OK) return rc;
  return done(launch_glu_bwd(*desc, plan, x, w, pre, dy, dx, dw, dbias,
                             static_cast<char*>(workspace), stream));
}

int ss_q8_pack(const ss_q8_pack_desc_t* desc, const void* x, int8_t* q, float* s, void* stream) {
  int rc = check_q8_pack(desc);
  if (rc != SS_OK) return rc;
  if (!x || !q || !s || aliased({q, s}, {x})) return SS_ERR_INVALID_ARG;
  if (!row_aligned(x, desc->x_stride, desc->dtype) || !all_aligned({q, s}))
    return SS_ERR_INVALID_ARG;
  if ((rc = check_device()) != SS_OK) return rc;
  return done(launch_q8_pack(*desc, x, q, s, stream));
}

size_t ss_q8_workspace_bytes(const ss_q8_desc_t* desc) {
  if (check_q8(desc) != SS_OK) return 0;
  return plan_q8(*desc).bytes;
}

int ss_q8_linear(const ss_q8_desc_t* desc, const int8_t* xq, const float* xs, const int8_t* wq,
                 const float* ws, const float* bias, const void* residual, void* y,
                 void* workspace, size_t ws_bytes, void* stream) {
  int rc = check_q8(desc);
  if (rc != SS_OK) return rc;
  if (!xq || !xs || !wq || !ws || !y || aliased({y}, {xq, xs, wq, ws, bias}))
    return SS_ERR_INVALID_ARG;
  if (y == residual && desc->res_dtype != desc->out_dtype) return SS_ERR_INVALID_ARG;
  if ((desc->x_stride == 0 && !aligned(xq, kPtrAlign)) ||
      (desc->w_stride == 0 && !aligned(wq, kPtrAlign)) ||
      !all_aligned({xs, ws, bias, residual, y}))
    return SS_ERR_INVALID_ARG;
  const Q8Plan plan = plan_q8(*desc);
  if (bad_workspace(workspace, ws_bytes, plan.bytes)) return SS_ERR_WORKSPACE;
  if ((rc = check_device()) != SS_OK) return rc;
  return done(launch_q8_linear(*desc, plan, xq, xs, wq, ws, bias, residual, y,
                               static_cast<char*>(workspace), stream));
}

}  // extern "C"
