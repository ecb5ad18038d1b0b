/*
 * ss_glu.h -- C ABI of the gated half of a feed-forward block: both projections, the
 * activation and the product in one kernel, forward and backward (same library,
 * libssscan.so).
 *
 * The operation: beside the recurrence, a residual block of such models widens its
 * input by two projections, one of which gates the other, as silu(z) gates the scan's
 * output (Gu & Dao wiki note, git.lyz.one, section "Mamba architecture": the gated
 * block).  For M rows (tokens), K inputs and F outputs
 *     gate = x wg^T + bg     up = x wu^T + bu     x : (M, K)   wg, wu : (F, K)
 *     y    = act(gate) up    act : none | silu | gelu
 * with both weights in one tensor w : (2 F, K), the rows of wg in front of those of
 * wu, and so bias : (2 F) and pre = [gate, up] : (M, 2 F).  Backward, with
 *     d  = [dy up act'(gate), dy act(gate)]    (M, 2 F)
 *     dx = d w (M, K)     dw = d^T x (2 F, K)     dbias = sum_rows d (2 F)
 * The projection back to K channels is ss_linear_fwd, whose residual is the block's.
 * A few rows (decoding) run in kernels of their own that stream w once.
 *
 * Conventions (as in ss_linear.h): dense row-major tensors, last index fastest, except
 * that x may have a row stride.  DEVICE pointers owned by the caller, 16-byte aligned
 * (x with a row stride: aligned to its element size).  Asynchronous on `stream`;
 * validation before any HIP call; no allocation; deterministic.  Status codes of
 * ss_scan.h.  Products are summed in float32; bias, activation and gating are float32
 * on the sums, and y and pre are each rounded once.
 */
#ifndef SS_GLU_H
#define SS_GLU_H

#include <stddef.h>
#include <stdint.h>

#include "ss_linear.h"
#include "ss_scan.h"

#ifdef __cplusplus
extern "C" {
#endif

/* 1 <= rows <= 2^28; 1 <= in_dim <= 2^20, 1 <= out_dim <= 2^19; x, w, y and pre of at
 * most 2^35 elements each. */
typedef struct ss_glu_desc {
  int64_t rows;       /* M, tokens */
  int64_t in_dim;     /* K */
  int64_t out_dim;    /* F */
  int64_t x_stride;   /* elements from one row of x to the next; 0 = dense, else
                         in_dim <= x_stride <= 2^20 */
  int32_t in_dtype;   /* ss_dtype_t of x, w and pre */
  int32_t out_dtype;  /* ss_dtype_t of y (backward: dy) */
  int32_t grad_dtype; /* ss_dtype_t of dx and dw (not read by the forward) */
  int32_t act;        /* ss_act_t: SS_ACT_NONE, SS_ACT_SILU or SS_ACT_GELU */
} ss_glu_desc_t;

/* Operations for ss_glu_workspace_bytes. */
#define SS_GLU_FWD 0
#define SS_GLU_BWD 1

/* Bytes of device workspace the operation needs (0 when none, or for an invalid
 * description).  Depends only on the description.  Contents are scratch. */
size_t ss_glu_workspace_bytes(const ss_glu_desc_t* desc, int op);

/*
 * Forward.  x, w, y required; bias (float32) optional; pre: optional output, both
 * pre-activations in in_dtype for the backward.  No output may alias another argument.
 *   workspace, ws_bytes : at least ss_glu_workspace_bytes(desc, SS_GLU_FWD), 256-byte
 *   aligned; may be NULL when that is 0.
 */
int ss_glu_fwd(const ss_glu_desc_t* desc, const void* x, const void* w, const float* bias, void* y,
               void* pre, void* workspace, size_t ws_bytes, void* stream);

/*
 * Backward.  w, pre and dy required; outputs dx, dw (grad_dtype) and dbias (float32)
 * optional, at least one, all overwritten; x required iff dw is asked for.  With bf16
 * operands d enters both products by the gradients' type, as in ss_linear_bwd: rounded
 * to bf16 for bf16 gradients, as the sum of two bf16 (to 2^-16) for float32 ones, at
 * twice the matrix work.  dbias is summed before that rounding.  No output may alias
 * another argument.
 */
int ss_glu_bwd(const ss_glu_desc_t* desc, const void* x, const void* w, const void* pre,
               const void* dy, void* dx, void* dw, float* dbias, void* workspace, size_t ws_bytes,
               void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SS_GLU_H */
