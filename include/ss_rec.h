/*
 * ss_rec.h -- C ABI of the gated linear recurrence, forward, backward and single
 * tokens (same library, libssscan.so).
 *
 * The operation: one real state per channel whose decay and input weight are
 * gated by the input, in the place of the selective scan's N states ("A Survey of
 * Mamba" summary, csdn, section "SSM": a linear recurrence; Selection: its
 * coefficients follow the input).  With r and i the gates' pre-activations
 * (columns of a projection), lam one parameter per channel and c the decay
 * constant,
 *     log a_t = -c softplus(lam[d]) sigmoid(r[b,t,d])
 *     g_t     = sqrt(1 - a_t^2) sigmoid(i[b,t,d]) x[b,t,d]
 *     h_t     = a_t h_(t-1) + g_t             (g_t alone where starts[b,t] != 0)
 *     y[b,t,d] = h_t,  or  h_t silu(z[b,t,d])  with z   (the block's gate)
 * so that |h| keeps the scale of x whatever the decay.  Steps at and behind
 * lengths[b] leave the state as it is; y is 0 there.  starts marks the first token
 * of each document of a packed row.
 *
 * Backward, with v_t = dy_t silu(z_t) and the adjoint of the state
 *     u_t = v_t + a_(t+1) u_(t+1)     (no second term before a start; dh_last
 *                                      enters behind the last step)
 *     dx = u sqrt(1 - a^2) sigmoid(i)       di = dx x (1 - sigmoid(i))
 *     dl = u (a h_(t-1) - a^2 / sqrt(1 - a^2) sigmoid(i) x)   (of log a)
 *     dr = dl log a (1 - sigmoid(r))        dz = dy h silu'(z)
 *     dlam = -c sigmoid(lam) sum_(b,t) dl sigmoid(r)          dh0 = a_0 u_0
 * The states are recomputed from those that the forward kept, one in front of
 * every SS_REC_CHUNK-th step.
 *
 * Conventions (as in ss_scan.h): x, r, i, z, y, dy, dx, dr, di, dz : (B, L, D),
 * last index fastest; lam, dlam : (D) float32; h0, h_last, dh_last, dh0, the
 * decode state h : (B, D) float32; states : (B, ceil(L / SS_REC_CHUNK), D)
 * float32; starts : (B, L) uint8; lengths : (B) int32, values outside 0..L count
 * as the nearest of them.  Dense, except that x, r, i and z may each have a row
 * stride (column ranges of wider projections).  DEVICE pointers owned by the
 * caller, 16-byte aligned (a tensor with a row stride: aligned to its element
 * size; starts: any address).  Asynchronous on `stream`; validation before any HIP
 * call; no allocation; deterministic.  Status codes of ss_scan.h.  Everything
 * between input and output is float32, and a decay near 1 keeps the relative
 * accuracy of 1 - a however long its state is remembered (ss_rec_step rounds the
 * state to float32 once a token); y and the gradients are rounded once.  What is NaN
 * or infinite behind a length or in front of a start does not reach the other side;
 * within a document an infinite state may turn into NaN.
 */
#ifndef SS_REC_H
#define SS_REC_H

#include <stddef.h>
#include <stdint.h>

#include "ss_scan.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SS_REC_CHUNK 64 /* steps between two kept states */

/* batch, seqlen, dim >= 1; seqlen < 2^31; dim <= 2^20; batch * ceil(dim / 64) <= 2^21; a tensor
 * spans at most 2^40 elements. */
typedef struct ss_rec_desc {
  int64_t batch;     /* B */
  int64_t seqlen;    /* L (1 for ss_rec_step) */
  int64_t dim;       /* D, channels */
  int64_t x_stride;  /* elements from one row (b, t) of x to the next; 0 = dense, */
  int64_t r_stride;  /* else dim <= stride <= 2^20; the same for r, i and z */
  int64_t i_stride;
  int64_t z_stride;
  int32_t in_dtype;  /* ss_dtype_t of x, r, i, z and their gradients */
  int32_t out_dtype; /* ss_dtype_t of y (backward: dy) */
  float decay;       /* c > 0, finite */
  int32_t reserved;  /* must be 0 */
} ss_rec_desc_t;

/* Operations for ss_rec_workspace_bytes. */
#define SS_REC_FWD 0
#define SS_REC_BWD 1

/* Bytes of device workspace the operation needs (0 when none, or for an invalid
 * description).  Depends only on the description.  Contents are scratch. */
size_t ss_rec_workspace_bytes(const ss_rec_desc_t* desc, int op);

/*
 * Forward.  x, r, i, lam, y required; z, h0, starts, lengths optional; h_last and
 * states optional outputs.  h_last may be the same buffer as h0; otherwise no
 * output may alias another argument.
 *   workspace, ws_bytes : at least ss_rec_workspace_bytes(desc, SS_REC_FWD),
 *   256-byte aligned; may be NULL when that is 0.
 */
int ss_rec_fwd(const ss_rec_desc_t* desc, const void* x, const void* r, const void* i,
               const float* lam, const void* z, const float* h0, const uint8_t* starts,
               const int32_t* lengths, void* y, float* h_last, float* states, void* workspace,
               size_t ws_bytes, void* stream);

/*
 * Backward.  x, r, i, lam, z, starts, lengths as in the forward; states: what it
 * kept (its first row holds h0); dy required; dh_last optional (0).  dx, dr, di,
 * dlam required, dz required iff z is given, dh0 optional; all overwritten (zeros
 * behind the lengths).  No output may alias another argument.
 */
int ss_rec_bwd(const ss_rec_desc_t* desc, const void* x, const void* r, const void* i,
               const float* lam, const void* z, const uint8_t* starts, const int32_t* lengths,
               const float* states, const void* dy, const float* dh_last, void* dx, void* dr,
               void* di, void* dz, float* dlam, float* dh0, void* workspace, size_t ws_bytes,
               void* stream);

/*
 * One token of every sequence: h : (B, D) is read and overwritten; x, r, i, z, y :
 * (B, D).  desc->seqlen must be 1.  y must not alias another argument.
 */
int ss_rec_step(const ss_rec_desc_t* desc, float* h, const void* x, const void* r, const void* i,
                const float* lam, const void* z, void* y, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SS_REC_H */
