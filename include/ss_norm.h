/*
 * ss_norm.h -- C ABI of the layer norm in front of a Mamba block, with the
 * block's residual add, forward and backward (same library, libssscan.so).
 *
 * The operation: a Mamba block normalises its input over the channels, and the
 * block's output is added to what came in (Gu & Dao wiki note, git.lyz.one,
 * section "Mamba architecture": LayerNorm -> Linear -> ... -> Linear -> +
 * residual).  Fused here: the residual add of the previous block and the norm
 * of the next one.  Per row (token) of D channels
 *     s    = x + residual                        (s = x without a residual)
 *     mean = sum_d s / D      rstd = 1 / sqrt(sum_d (s - mean)^2 / D + eps)
 *     y    = (s - mean) rstd weight + bias       (weight = 1, bias = 0 if NULL)
 * and backward, with xh = (s - mean) rstd and g = dy weight,
 *     dx      = rstd (g - sum_d g / D - xh sum_d (g xh) / D) + dsum
 *     dweight = sum_rows dy xh      dbias = sum_rows dy
 * dx is the gradient of x and of the residual alike; dsum is the gradient that
 * reaches s from elsewhere (the residual stream).
 *
 * Conventions (as in ss_scan.h): dense row-major tensors, last index fastest,
 *   x, residual, sum, y, s, dy, dsum, dx : (rows, D);  weight, bias, dweight,
 *   dbias : (D) float32;  mean, rstd : (rows) float32;
 * except that x (backward: s) may have a row stride.  DEVICE pointers owned by
 * the caller, 16-byte aligned (x or s with a row stride: aligned to its element
 * size).  Asynchronous on `stream`; validation before any HIP call; no
 * allocation; deterministic.  Status codes of ss_scan.h.  All sums are float32;
 * the variance is taken about the mean (no difference of squares).  NaN and Inf
 * propagate within their row (and into dweight, dbias).
 */
#ifndef SS_NORM_H
#define SS_NORM_H

#include <stddef.h>
#include <stdint.h>

#include "ss_scan.h"

#ifdef __cplusplus
extern "C" {
#endif

/* rows, dim >= 1; dim <= 32768; eps > 0 and finite. */
typedef struct ss_norm_desc {
  int64_t rows;       /* tokens, B * L */
  int64_t dim;        /* D, channels */
  int64_t x_stride;   /* elements from one row of x (backward: s) to the next;
                         0 = dense, else dim <= x_stride <= 2^24 */
  int32_t in_dtype;   /* ss_dtype_t of x (backward: s) */
  int32_t res_dtype;  /* ss_dtype_t of residual and sum (backward: dsum and dx) */
  int32_t out_dtype;  /* ss_dtype_t of y (backward: dy) */
  float eps;          /* not read by the backward */
} ss_norm_desc_t;

/*
 * Forward.  x, y required; residual, weight, bias optional.
 *   sum        : optional output s in res_dtype (the new residual stream).  The
 *                norm itself takes s before that rounding.  It may be the same
 *                buffer as residual (the stream is then advanced in place).
 *   mean, rstd : optional outputs, both or neither (the backward needs them).
 * Otherwise no output may alias another argument.
 */
int ss_layernorm_fwd(const ss_norm_desc_t* desc, const void* x, const void* residual,
                     const float* weight, const float* bias, void* y, void* sum, float* mean,
                     float* rstd, void* stream);

/* Bytes of device workspace ss_layernorm_bwd needs (partial sums of dweight and
 * dbias); 0 for an invalid description. */
size_t ss_layernorm_workspace_bytes(const ss_norm_desc_t* desc);

/*
 * Backward.  s is what was normalised (x, or the forward's sum), mean and rstd
 * the forward's; dy and dx required; weight, dsum optional; dweight and dbias
 * optional outputs, overwritten.  dx may be the same buffer as dsum and must
 * not alias anything else.
 *   workspace, ws_bytes : at least ss_layernorm_workspace_bytes(desc), 256-byte
 *   aligned; may be NULL when neither dweight nor dbias is asked for.
 */
int ss_layernorm_bwd(const ss_norm_desc_t* desc, const void* s, const float* weight,
                     const float* mean, const float* rstd, const void* dy, const void* dsum,
                     void* dx, float* dweight, float* dbias, void* workspace, size_t ws_bytes,
                     void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SS_NORM_H */
