/*
 * ss_q8.h -- C ABI of the linear projection in 8-bit integers, with a scale per token
 * and per output channel (same library, libssscan.so).
 *
 * The operation: a served block's projections read their weights and inputs as signed
 * 8-bit integers, a row of either sharing one scale:
 *     s = max_k |x[m,k]| / 127      q[m,k] = 127 x[m,k] / max_k |x[m,k]| to the nearest
 *                                   whole number, ties to even
 *     x[m,k] ~ q[m,k] s[m]
 * for x : (M, K), and the same for w : (N, K), packed once.  Whole numbers are summed
 * exactly, so that
 *     y = act(xs[m] ws[n] sum_k xq[m,k] wq[n,k] + bias[n]) + residual
 * differs from the product of the packed values only by the epilogue's float32
 * rounding.  The nearest whole number is that of the real quotient (no rounded
 * reciprocal decides it).  A row of zeros has s = 0; a row with a NaN or an infinity has
 * s = NaN and q = 0, and reads back as NaN.
 *
 * Conventions (as in ss_linear.h): row-major tensors, last index fastest; q : (rows, dim)
 * int8, s : (rows) float32.  DEVICE pointers owned by the caller, 16-byte aligned (a
 * tensor with a row stride: aligned to its element size).  Asynchronous on `stream`;
 * validation before any HIP call; no allocation; deterministic.  Status codes of
 * ss_scan.h.
 */
#ifndef SS_Q8_H
#define SS_Q8_H

#include <stddef.h>
#include <stdint.h>

#include "ss_linear.h"
#include "ss_scan.h"

#ifdef __cplusplus
extern "C" {
#endif

/* 1 <= rows < 2^31; 1 <= dim <= 2^20. */
typedef struct ss_q8_pack_desc {
  int64_t rows;
  int64_t dim;
  int64_t x_stride;  /* elements from one row of x to the next; 0 = dense, else
                        dim <= x_stride <= 2^20 */
  int64_t q_stride;  /* the same for q; the bytes between its rows are set to 0 */
  int32_t dtype;     /* ss_dtype_t of x */
  int32_t reserved;  /* must be 0 */
} ss_q8_pack_desc_t;

/* x -> (q, s).  All required; no aliasing.  The rows of q take rows * q_stride bytes:
 * behind the last one too. */
int ss_q8_pack(const ss_q8_pack_desc_t* desc, const void* x, int8_t* q, float* s, void* stream);

/* 1 <= rows <= 2^28; 1 <= in_dim <= 2^16 (sums stay below 2^31), 1 <= out_dim <= 2^20;
 * x, w and y of at most 2^35 elements each. */
typedef struct ss_q8_desc {
  int64_t rows;       /* M, tokens */
  int64_t in_dim;     /* K */
  int64_t out_dim;    /* N */
  int64_t x_stride;   /* bytes from one row of xq to the next; 0 = dense, else
                         in_dim <= x_stride <= 2^20 */
  int64_t w_stride;   /* the same for wq */
  int32_t out_dtype;  /* ss_dtype_t of y */
  int32_t res_dtype;  /* ss_dtype_t of residual */
  int32_t act;        /* ss_act_t */
  int32_t reserved;   /* must be 0 */
} ss_q8_desc_t;

/* Bytes of device workspace ss_q8_linear needs (0 when none, or for an invalid
 * description).  Depends only on the description.  Contents are scratch. */
size_t ss_q8_workspace_bytes(const ss_q8_desc_t* desc);

/*
 * xq : (M, K), xs : (M), wq : (N, K), ws : (N), y required; bias (N) float32,
 * residual (M, N) optional.  y may be the same buffer as residual when their types are
 * equal; otherwise it may not alias another argument.
 *   workspace, ws_bytes : at least ss_q8_workspace_bytes(desc), 256-byte aligned; may be
 *   NULL when that is 0.
 */
int ss_q8_linear(const ss_q8_desc_t* desc, const int8_t* xq, const float* xs, const int8_t* wq,
                 const float* ws, const float* bias, const void* residual, void* y,
                 void* workspace, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SS_Q8_H */
