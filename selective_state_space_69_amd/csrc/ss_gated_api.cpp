// C-ABI entry points of a gated recurrent block's operators: the gated linear
// recurrence.  As for the scan, validation is plain host logic that runs before any
// HIP call; then the device is checked and the kernels are launched.
#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "ss_internal.h"

namespace ss {
namespace {

constexpr int64_t kMaxElems = int64_t(1) << 40;
constexpr int64_t kMaxDim = int64_t(1) << 20;
constexpr int64_t kMaxGroups = int64_t(1) << 22;     // of 64 channels: a grid's threads stay below 2^32

size_t elem(int32_t dtype) { return dtype == SS_BF16 ? 2 : 4; }

bool bad_stride(int64_t stride, int64_t dim, int64_t most) {
  return stride != 0 && (stride < dim || stride > most);
}

// A tensor read with a row stride needs its element alignment only.
bool row_aligned(const void* p, int64_t stride, int32_t dtype) {
  return !p || aligned(p, stride == 0 ? kPtrAlign : elem(dtype));
}

bool all_aligned(std::initializer_list<const void*> ptrs) {
  for (const void* p : ptrs)
    if (p && !aligned(p, kPtrAlign)) return false;
  return true;
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
  if (d->batch < 1 || d->seqlen < 1 || d->seqlen > INT32_MAX || d->dim < 1 || d->dim > kMaxDim) return SS_ERR_INVALID_ARG;
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

}  // extern "C"
