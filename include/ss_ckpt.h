/*
 * ss_ckpt.h -- C ABI of activation checkpoints in 8 bits (same library,
 * libssscan.so).
 *
 * What a backward pass needs of its forward is either recomputed or kept ("A
 * Survey of Mamba" summary, csdn, hardware-aware computation: recomputation
 * extends to the projection, convolution and activation of the block).  A
 * checkpoint keeps a tensor at 8.25 bits per value instead of 16 or 32: blocks
 * of 32 channels of a row share one power-of-two unit and hold signed 8-bit
 * multiples of it.
 *     e = max(1, E - 6)     E: the biased float32 exponent of the block's largest |x|
 *     q = clamp(round(x 2^(127 - e)), -127, 127)      ties to even
 *     x ~ q 2^(e - 127)
 * so that the block's largest value lands in [64, 127].  An error is at most
 * half a unit, or a whole one where 127.5 units and more are held as 127.
 * Scaling by a power of two is exact: the stored bits and the values read back
 * are the same whatever precision computes them, and every value read back is
 * exact in bf16 as well.  A block with a NaN or an infinity has e = 255, q = 0
 * and reads back as NaN.  The last block of a row may be shorter.
 * ss_linear_bwd_ckpt (ss_linear.h) takes such a checkpoint for its input.
 *
 * Conventions (as in ss_scan.h): x : (rows, D) in dtype, with an optional row
 * stride; q : (rows, D) int8; e : (rows, ceil(D / 32)) uint8; last index
 * fastest.  DEVICE pointers, 16-byte aligned (x with a row stride: aligned to
 * its element size).  Asynchronous on `stream`; validation before any HIP call;
 * no allocation, no workspace; deterministic.  Status codes of ss_scan.h.
 */
#ifndef SS_CKPT_H
#define SS_CKPT_H

#include <stddef.h>
#include <stdint.h>

#include "ss_scan.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SS_CKPT_BLOCK 32 /* channels that share one exponent */

/* rows, dim >= 1. */
typedef struct ss_ckpt_desc {
  int64_t rows;
  int64_t dim;       /* D */
  int64_t x_stride;  /* elements from one row of x to the next; 0 = dense, else
                        dim <= x_stride <= 2^24 */
  int32_t dtype;     /* ss_dtype_t of x */
  int32_t reserved;  /* must be 0 */
} ss_ckpt_desc_t;

/* x -> (q, e).  All required; no aliasing. */
int ss_ckpt_pack(const ss_ckpt_desc_t* desc, const void* x, int8_t* q, uint8_t* e, void* stream);

/* (q, e) -> x.  All required; no aliasing.  Elements of x between rows (row
 * stride) are left as they were. */
int ss_ckpt_unpack(const ss_ckpt_desc_t* desc, const int8_t* q, const uint8_t* e, void* x,
                   void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SS_CKPT_H */
