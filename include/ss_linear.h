/*
 * ss_linear.h -- C ABI of the linear projections of a Mamba block, with bias,
 * activation and residual in the product's epilogue, forward and backward (same
 * library, libssscan.so).
 *
 * The operation: a block expands its input by a linear layer, projects x to the
 * scan's B, C and (low-rank) step sizes and ends in a linear layer whose output
 * is added to the residual (Gu & Dao wiki note, git.lyz.one, sections "From S4
 * to S6" and "Mamba architecture"; "Mamba: S4 epic upgrade", hk.pswp.cn,
 * parameter-efficient data dependence).  For M rows (tokens), K inputs and N
 * outputs
 *     pre = x w^T + bias           x : (M, K)   w : (N, K)   bias : (N)
 *     y   = act(pre) + residual    y, pre, residual : (M, N)
 *     act : none | silu v sigmoid(v) | gelu v Phi(v) (Phi: the normal
 *           distribution function) | softplus log(1 + e^v)
 * and backward, with dpre = dy act'(pre),
 *     dx = dpre w (M, K)     dw = dpre^T x (N, K)     dbias = sum_rows dpre (N)
 * (the residual's gradient is dy itself).  A few rows (decoding) run in kernels
 * of their own that stream w once.
 *
 * Conventions (as in ss_scan.h): dense row-major tensors, last index fastest,
 * except that x may have a row stride (the step-size projection reads a column
 * range of the x projection's output).  DEVICE pointers owned by the caller,
 * 16-byte aligned (x with a row stride: aligned to its element size).
 * Asynchronous on `stream`; validation before any HIP call; no allocation;
 * deterministic.  Status codes of ss_scan.h.  Products are summed in float32;
 * bias is added, the activation taken and the residual added in float32, and y
 * is rounded once.
 */
#ifndef SS_LINEAR_H
#define SS_LINEAR_H

#include <stddef.h>
#include <stdint.h>

#include "ss_ckpt.h"
#include "ss_scan.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { SS_ACT_NONE = 0, SS_ACT_SILU = 1, SS_ACT_GELU = 2, SS_ACT_SOFTPLUS = 3 } ss_act_t;

/* 1 <= rows <= 2^28; 1 <= in_dim, out_dim <= 2^20; x, w and y of at most 2^35
 * elements each. */
typedef struct ss_linear_desc {
  int64_t rows;       /* M, tokens */
  int64_t in_dim;     /* K */
  int64_t out_dim;    /* N */
  int64_t x_stride;   /* elements from one row of x to the next; 0 = dense, else
                         in_dim <= x_stride <= 2^20; ss_linear_bwd_ckpt takes 0 */
  int32_t in_dtype;   /* ss_dtype_t of x, w and pre */
  int32_t out_dtype;  /* ss_dtype_t of y (backward: dy) */
  int32_t res_dtype;  /* ss_dtype_t of residual (not read by the backward) */
  int32_t grad_dtype; /* ss_dtype_t of dx and dw (not read by the forward) */
  int32_t act;        /* ss_act_t */
  int32_t reserved;   /* must be 0 */
} ss_linear_desc_t;

/* Operations for ss_linear_workspace_bytes. */
#define SS_LINEAR_FWD 0
#define SS_LINEAR_BWD 1       /* ss_linear_bwd */
#define SS_LINEAR_BWD_CKPT 2  /* ss_linear_bwd_ckpt */

/* Bytes of device workspace the operation needs (0 when none, or for an invalid
 * description).  Depends only on the description.  Contents are scratch. */
size_t ss_linear_workspace_bytes(const ss_linear_desc_t* desc, int op);

/*
 * Forward.  x, w, y required; bias (float32), residual optional; pre: optional
 * output, pre-activation values in in_dtype for the backward.  y may be the
 * same buffer as residual when their types are equal (the residual stream is
 * then advanced in place); otherwise no output may alias another argument.
 *   workspace, ws_bytes : at least ss_linear_workspace_bytes(desc,
 *   SS_LINEAR_FWD), 256-byte aligned; may be NULL when that is 0.
 */
int ss_linear_fwd(const ss_linear_desc_t* desc, const void* x, const void* w, const float* bias,
                  const void* residual, void* y, void* pre, void* workspace, size_t ws_bytes,
                  void* stream);

/*
 * Backward.  w and dy required; pre required iff act is not SS_ACT_NONE (in
 * in_dtype); outputs dx, dw (grad_dtype) and dbias (float32) optional, at least
 * one, all overwritten; x required iff dw is asked for.  With bf16 operands a
 * bf16 dy without activation enters both products as it is.  Any other dpre is
 * float32, and grad_dtype says what the products see of it: bf16 gradients, its
 * value rounded to bf16; float32 ones, the sum of two bf16 values (2^-16 of it),
 * for twice the matrix work (a caller who wants float32 sums of a rounded dpre at
 * the single price rounds dy to bf16 first).  dbias is summed before either
 * rounding.  No output may alias another argument.
 */
int ss_linear_bwd(const ss_linear_desc_t* desc, const void* x, const void* w, const void* pre,
                  const void* dy, void* dx, void* dw, float* dbias, void* workspace,
                  size_t ws_bytes, void* stream);

/*
 * ss_linear_bwd with x given as an 8-bit checkpoint (ss_ckpt.h): q : (M, K)
 * int8, e : (M, ceil(K / 32)) uint8, required iff dw is asked for.  Same
 * results, bit for bit, as ss_linear_bwd on the checkpoint's values.
 */
int ss_linear_bwd_ckpt(const ss_linear_desc_t* desc, const int8_t* q, const uint8_t* e,
                       const void* w, const void* pre, const void* dy, void* dx, void* dw,
                       float* dbias, void* workspace, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SS_LINEAR_H */
