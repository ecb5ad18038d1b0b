// C-ABI entry points of the operators around the scan in a Mamba block: layer
// norm, linear projections and 8-bit checkpoints.  As for the scan, validation
// is plain host logic that runs before any HIP call; then the device is checked
// and the kernels are launched.
#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "ss_internal.h"

namespace ss {
namespace {

constexpr int64_t kMaxElems = int64_t(1) << 40;
constexpr int64_t kMaxRows = INT32_MAX;
constexpr int64_t kMaxStride = int64_t(1) << 24;
constexpr int64_t kMaxLinear = int64_t(1) << 20;
// 64 x 64 tiles of any product stay below 2^24, a grid's threads below 2^32
constexpr int64_t kMaxLinearRows = int64_t(1) << 28;
constexpr int64_t kMaxLinearElems = int64_t(1) << 35;
constexpr int64_t kMaxNormDim = 32768;

size_t elem(int32_t dtype) { return dtype == SS_BF16 ? 2 : 4; }

bool bad_stride(int64_t stride, int64_t dim, int64_t most) {
  return stride != 0 && (stride < dim || stride > most);
}

// Rows read or written with a stride need their element alignment only.
size_t row_align(int64_t stride, int32_t dtype) {
  return stride == 0 ? kPtrAlign : elem(dtype);
}

bool all_aligned(std::initializer_list<const void*> ptrs) {
  for (const void* p : ptrs)
    if (p && !aligned(p, kPtrAlign)) return false;
  return true;
}

// whether p is one of the given pointers (NULL never is)
bool among(const void* p, std::initializer_list<const void*> ptrs) {
  if (!p) return false;
  for (const void* o : ptrs)
    if (p == o) return true;
  return false;
}

int check_norm(const ss_norm_desc_t* d, bool forward) {
  if (!d) return SS_ERR_INVALID_ARG;
  if (d->rows < 1 || d->rows > kMaxRows || d->dim < 1) return SS_ERR_INVALID_ARG;
  if (d->dim > kMaxNormDim) return SS_ERR_UNSUPPORTED;
  if (bad_stride(d->x_stride, d->dim, kMaxStride)) return SS_ERR_INVALID_ARG;
  if (!valid_dtype(d->in_dtype) || !valid_dtype(d->res_dtype) || !valid_dtype(d->out_dtype))
    return SS_ERR_UNSUPPORTED;
  if (forward && !(d->eps > 0.0f && std::isfinite(d->eps))) return SS_ERR_INVALID_ARG;
  return SS_OK;
}

int check_ckpt(const ss_ckpt_desc_t* d) {
  if (!d) return SS_ERR_INVALID_ARG;
  if (d->rows < 1 || d->dim < 1 || d->rows > kMaxElems || d->dim > kMaxStride ||
      d->rows > kMaxElems / d->dim)
    return SS_ERR_INVALID_ARG;
  if (bad_stride(d->x_stride, d->dim, kMaxStride)) return SS_ERR_INVALID_ARG;
  if (d->reserved != 0) return SS_ERR_INVALID_ARG;
  if (!valid_dtype(d->dtype)) return SS_ERR_UNSUPPORTED;
  return SS_OK;
}

int check_linear(const ss_linear_desc_t* d, int op) {
  if (!d) return SS_ERR_INVALID_ARG;
  if (op != SS_LINEAR_FWD && op != SS_LINEAR_BWD && op != SS_LINEAR_BWD_CKPT)
    return SS_ERR_INVALID_ARG;
  if (d->rows < 1 || d->rows > kMaxLinearRows || d->in_dim < 1 || d->out_dim < 1 ||
      d->in_dim > kMaxLinear || d->out_dim > kMaxLinear)
    return SS_ERR_INVALID_ARG;
  if (d->rows > kMaxLinearElems / d->in_dim || d->rows > kMaxLinearElems / d->out_dim ||
      d->out_dim > kMaxLinearElems / d->in_dim)
    return SS_ERR_INVALID_ARG;
  if (bad_stride(d->x_stride, d->in_dim, kMaxLinear)) return SS_ERR_INVALID_ARG;
  if (d->reserved != 0) return SS_ERR_INVALID_ARG;
  if (!valid_dtype(d->in_dtype) || !valid_dtype(d->out_dtype)) return SS_ERR_UNSUPPORTED;
  if (op == SS_LINEAR_FWD ? !valid_dtype(d->res_dtype) : !valid_dtype(d->grad_dtype))
    return SS_ERR_UNSUPPORTED;
  if (d->act < SS_ACT_NONE || d->act > SS_ACT_SOFTPLUS) return SS_ERR_UNSUPPORTED;
  if (op == SS_LINEAR_BWD_CKPT && d->x_stride != 0) return SS_ERR_UNSUPPORTED;
  return SS_OK;
}

int linear_bwd(const ss_linear_desc_t* d, int op, const void* x, const int8_t* q, const uint8_t* e,
               const void* w, const void* pre, const void* dy, void* dx, void* dw, float* dbias,
               void* workspace, size_t ws_bytes, void* stream) {
  int rc = check_linear(d, op);
  if (rc != SS_OK) return rc;
  if (!w || !dy || (!dx && !dw && !dbias)) return SS_ERR_INVALID_ARG;
  if ((d->act != SS_ACT_NONE) != (pre != nullptr)) return SS_ERR_INVALID_ARG;
  if (op == SS_LINEAR_BWD) {
    if (dw && !x) return SS_ERR_INVALID_ARG;
    if (x && !aligned(x, row_align(d->x_stride, d->in_dtype))) return SS_ERR_INVALID_ARG;
  } else if ((dw && (!q || !e)) || !all_aligned({q, e})) {
    return SS_ERR_INVALID_ARG;
  }
  const void *dxv = dx, *dwv = dw, *dbv = dbias;
  if (among(dxv, {x, q, e, w, pre, dy, dwv, dbv}) || among(dwv, {x, q, e, w, pre, dy, dbv}) ||
      among(dbv, {x, q, e, w, pre, dy}))
    return SS_ERR_INVALID_ARG;
  if (!all_aligned({w, pre, dy, dx, dw, dbias})) return SS_ERR_INVALID_ARG;
  const LinearPlan plan = plan_linear(*d, op);
  if (plan.bytes > 0 && (!workspace || ws_bytes < plan.bytes || !aligned(workspace, kAlign)))
    return SS_ERR_WORKSPACE;
  if ((rc = check_device()) != SS_OK) return rc;
  return launch_linear_bwd(*d, plan, x, q, e, w, pre, dy, dx, dw, dbias,
                           static_cast<char*>(workspace), stream) == 0
             ? SS_OK
             : SS_ERR_HIP;
}

}  // namespace
}  // namespace ss

using namespace ss;

extern "C" {

int ss_layernorm_fwd(const ss_norm_desc_t* desc, const void* x, const void* residual,
                     const float* weight, const float* bias, void* y, void* sum, float* mean,
                     float* rstd, void* stream) {
  int rc = check_norm(desc, true);
  if (rc != SS_OK) return rc;
  if (!x || !y || (mean != nullptr) != (rstd != nullptr)) return SS_ERR_INVALID_ARG;
  if (among(y, {x, residual, weight, bias, sum, mean, rstd}) ||
      among(sum, {x, weight, bias, mean, rstd}) ||
      among(mean, {x, residual, weight, bias, rstd}) || among(rstd, {x, residual, weight, bias}))
    return SS_ERR_INVALID_ARG;
  if (!aligned(x, row_align(desc->x_stride, desc->in_dtype)) ||
      !all_aligned({residual, weight, bias, y, sum, mean, rstd}))
    return SS_ERR_INVALID_ARG;
  if ((rc = check_device()) != SS_OK) return rc;
  return launch_norm_fwd(*desc, x, residual, weight, bias, y, sum, mean, rstd, stream) == 0
             ? SS_OK
             : SS_ERR_HIP;
}

size_t ss_layernorm_workspace_bytes(const ss_norm_desc_t* desc) {
  if (check_norm(desc, false) != SS_OK) return 0;
  return plan_norm(*desc).bytes;
}

int ss_layernorm_bwd(const ss_norm_desc_t* desc, const void* s, const float* weight,
                     const float* mean, const float* rstd, const void* dy, const void* dsum,
                     void* dx, float* dweight, float* dbias, void* workspace, size_t ws_bytes,
                     void* stream) {
  int rc = check_norm(desc, false);
  if (rc != SS_OK) return rc;
  if (!s || !mean || !rstd || !dy || !dx) return SS_ERR_INVALID_ARG;
  if (among(dx, {s, weight, mean, rstd, dy, dweight, dbias}) ||
      among(dweight, {s, weight, mean, rstd, dy, dsum, dbias}) ||
      among(dbias, {s, weight, mean, rstd, dy, dsum}))
    return SS_ERR_INVALID_ARG;
  if (!aligned(s, row_align(desc->x_stride, desc->in_dtype)) ||
      !all_aligned({weight, mean, rstd, dy, dsum, dx, dweight, dbias}))
    return SS_ERR_INVALID_ARG;
  const NormPlan plan = plan_norm(*desc);
  if ((dweight || dbias) &&
      (!workspace || ws_bytes < plan.bytes || !aligned(workspace, kAlign)))
    return SS_ERR_WORKSPACE;
  if ((rc = check_device()) != SS_OK) return rc;
  return launch_norm_bwd(*desc, plan, s, weight, mean, rstd, dy, dsum, dx, dweight, dbias,
                         static_cast<char*>(workspace), stream) == 0
             ? SS_OK
             : SS_ERR_HIP;
}

int ss_ckpt_pack(const ss_ckpt_desc_t* desc, const void* x, int8_t* q, uint8_t* e, void* stream) {
  int rc = check_ckpt(desc);
  if (rc != SS_OK) return rc;
  if (!x || !q || !e) return SS_ERR_INVALID_ARG;
  const void *qv = q, *ev = e;
  if (among(x, {qv, ev}) || qv == ev) return SS_ERR_INVALID_ARG;
  if (!aligned(x, row_align(desc->x_stride, desc->dtype)) || !all_aligned({qv, ev}))
    return SS_ERR_INVALID_ARG;
  if ((rc = check_device()) != SS_OK) return rc;
  return launch_ckpt_pack(*desc, x, q, e, stream) == 0 ? SS_OK : SS_ERR_HIP;
}

int ss_ckpt_unpack(const ss_ckpt_desc_t* desc, const int8_t* q, const uint8_t* e, void* x,
                   void* stream) {
  int rc = check_ckpt(desc);
  if (rc != SS_OK) return rc;
  if (!x || !q || !e) return SS_ERR_INVALID_ARG;
  const void *qv = q, *ev = e;
  if (among(x, {qv, ev})) return SS_ERR_INVALID_ARG;
  if (!aligned(x, row_align(desc->x_stride, desc->dtype)) || !all_aligned({qv, ev}))
    return SS_ERR_INVALID_ARG;
  if ((rc = check_device()) != SS_OK) return rc;
  return launch_ckpt_unpack(*desc, q, e, x, stream) == 0 ? SS_OK : SS_ERR_HIP;
}

size_t ss_linear_workspace_bytes(const ss_linear_desc_t* desc, int op) {
  if (check_linear(desc, op) != SS_OK) return 0;
  return plan_linear(*desc, op).bytes;
}

int ss_linear_fwd(const ss_linear_desc_t* desc, const void* x, const void* w, const float* bias,
                  const void* residual, void* y, void* pre, void* workspace, size_t ws_bytes,
                  void* stream) {
  int rc = check_linear(desc, SS_LINEAR_FWD);
  if (rc != SS_OK) return rc;
  if (!x || !w || !y) return SS_ERR_INVALID_ARG;
  if (among(y, {x, w, bias, pre}) || among(pre, {x, w, bias, residual})) return SS_ERR_INVALID_ARG;
  if (y == residual && desc->res_dtype != desc->out_dtype) return SS_ERR_INVALID_ARG;
  if (!aligned(x, row_align(desc->x_stride, desc->in_dtype)) ||
      !all_aligned({w, bias, residual, y, pre}))
    return SS_ERR_INVALID_ARG;
  const LinearPlan plan = plan_linear(*desc, SS_LINEAR_FWD);
  if (plan.bytes > 0 && (!workspace || ws_bytes < plan.bytes || !aligned(workspace, kAlign)))
    return SS_ERR_WORKSPACE;
  if ((rc = check_device()) != SS_OK) return rc;
  return launch_linear_fwd(*desc, x, w, bias, residual, y, pre, static_cast<char*>(workspace),
                           stream) == 0
             ? SS_OK
             : SS_ERR_HIP;
}

int ss_linear_bwd(const ss_linear_desc_t* desc, const void* x, const void* w, const void* pre,
                  const void* dy, void* dx, void* dw, float* dbias, void* workspace,
                  size_t ws_bytes, void* stream) {
  return linear_bwd(desc, SS_LINEAR_BWD, x, nullptr, nullptr, w, pre, dy, dx, dw, dbias, workspace,
                    ws_bytes, stream);
}

int ss_linear_bwd_ckpt(const ss_linear_desc_t* desc, const int8_t* q, const uint8_t* e,
                       const void* w, const void* pre, const void* dy, void* dx, void* dw,
                       float* dbias, void* workspace, size_t ws_bytes, void* stream) {
  return linear_bwd(desc, SS_LINEAR_BWD_CKPT, nullptr, q, e, w, pre, dy, dx, dw, dbias, workspace,
                    ws_bytes, stream);
}

}  // extern "C"
