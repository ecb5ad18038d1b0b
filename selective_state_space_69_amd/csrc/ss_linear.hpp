// What the matrix-product kernels of the linear projections share: the problem
// as each of the three products states it, and the epilogue.
//
// Every product is written O[r][s] = sum_t R(r, t) S(s, t), O row-major with s
// contiguous:
//   forward  y  (M, N): R = x    (t = k contiguous)   S = w  (t = k contiguous)
//   backward dx (M, K): R = dpre (t = n contiguous)   S = w  (s = k contiguous)
//            dw (N, K): R = dpre (r = n contiguous)   S = x  (s = k contiguous)
// S feeds the A side of the MFMA and R the B side, so that a lane's four
// accumulator registers are four neighbours of one output row.
#pragma once

#include "ss_device.hpp"

namespace ss {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));

// what is multiplied and what comes of it: plain products, two gated by each other, 8-bit
// integers
enum { kMm, kGlu, kInt8 };

// 16 bytes of t of either operand, T's
template <typename T, typename V, typename Acc>
__device__ __forceinline__ Acc mfma(V a, V b, Acc c) {
#if defined(__HIP_DEVICE_COMPILE__)
  if constexpr (sizeof(T) == 1) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a),
                                                 __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
  } else if constexpr (sizeof(T) == 2) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a[i]), __uint_as_float(b[i]), c, 0,
                                               0, 0);
  }
#endif
  return c;
}

struct MmParams {
  const void* R;
  const void* S;
  int64_t ldr, lds;      // elements from one row of the operand's storage to the next
  int64_t nR;            // output rows
  int32_t nS;            // output columns
  int64_t nT;            // contraction length
  int64_t t_split;       // contraction length of one split (a multiple of the tile's)
  int32_t splits;
  int32_t tiles_r, tiles_s;
  // epilogue
  const float* bias;     // (nS) or null
  const void* res;       // (nR, nS) or null
  void* out;
  void* pre;             // (nR, nS) or null
  float* part;           // (splits, nR, nS) when splits > 1
  int32_t act, out_bf16, res_bf16, pre_bf16;
  // 8-bit integers: R's and S's unit per row
  const float* row_scale;
  const float* col_scale;
};

// max(v, 0) in one instruction (fmaxf spends two more on quieting NaNs; a NaN here
// reaches the result through the logarithm)
__device__ __forceinline__ float max0(float v) {
#if defined(__HIP_DEVICE_COMPILE__)
  float r;
  asm("v_max_f32 %0, 0, %1" : "=v"(r) : "v"(v));
  return r;
#else
  return v > 0.0f ? v : 0.0f;
#endif
}
// Upper tail of the normal distribution, Q(z) = 1 - Phi(z) at z = |v|, and its
// density's exponential g = e^(-z^2/2).  Q = g G(t) with t = 1 / (1 + 0.23 z): e^(z^2/2)
// Q(z) is smooth in t on (0, 1], and G is the degree 8 polynomial of least relative
// error (4.8e-8, fitted for z in [0, 14]), so both sides of the GELU keep their
// relative accuracy.  No branch, two transcendentals: a third of the work of erff
// (fp32 3001 x 770 x 1537 with GELU: 91 us with erff, 78 so).
__device__ __forceinline__ float normal_tail(float v, float& g) {
  const float t = hw_rcp(__builtin_fmaf(__builtin_fabsf(v), 0.23f, 1.0f));
  float p = -0.07846643577207714f;
  p = __builtin_fmaf(p, t, 0.2904092622834526f);
  p = __builtin_fmaf(p, t, -0.27811700323595473f);
  p = __builtin_fmaf(p, t, 0.30146138824941776f);
  p = __builtin_fmaf(p, t, -0.032912219220029286f);
  p = __builtin_fmaf(p, t, 0.11951057618200757f);
  p = __builtin_fmaf(p, t, 0.08576384069547627f);
  p = __builtin_fmaf(p, t, 0.0923783211191706f);
  p = __builtin_fmaf(p, t, -2.7754017451191973e-05f);
  g = hw_exp2(v * v * (-0.5f * kLog2e));
  return p * g;
}
__device__ __forceinline__ float apply_act(int act, float v) {
  switch (act) {
    case SS_ACT_SILU: return silu(v);
    case SS_ACT_GELU: {
      float g;
      const float q = normal_tail(v, g);
      return v * (v > 0.0f ? 1.0f - q : q);
    }
    case SS_ACT_SOFTPLUS:   // max(v, 0) + log(1 + e^-|v|): the largest v pass through
      return __builtin_fmaf(log2_1p_exp2(__builtin_fabsf(v) * -kLog2e), kLn2, max0(v));
    default: return v;
  }
}
__device__ __forceinline__ float act_grad(int act, float v) {
  switch (act) {
    case SS_ACT_SILU: {
      const float s = hw_rcp(1.0f + hw_exp2(-v * kLog2e));
      return s * __builtin_fmaf(v, 1.0f - s, 1.0f);
    }
    case SS_ACT_GELU: {
      float g;
      const float q = normal_tail(v, g);
      return __builtin_fmaf(v * 0.39894228040143268f, g, v > 0.0f ? 1.0f - q : q);
    }
    case SS_ACT_SOFTPLUS: return hw_rcp(1.0f + hw_exp2(-v * kLog2e));
    default: return 1.0f;
  }
}

// Output tile of work item `id`.  Neighbouring items (one XCD's) share operand
// rows in its L2: tiles run down columns of a band of up to 8 tile rows.
// 32 bits: a grid has fewer items, and a 64-bit division takes half a microsecond of
// a tile's time.
__device__ __forceinline__ void tile_of(const MmParams& p, uint32_t id, int64_t* tr, int* ts) {
  constexpr uint32_t kBand = 8;
  const uint32_t per_band = kBand * uint32_t(p.tiles_s);
  const uint32_t band = id / per_band;
  const uint32_t in = id - band * per_band;
  const uint32_t left = uint32_t(p.tiles_r) - band * kBand;
  const uint32_t h = left < kBand ? left : kBand;
  const uint32_t q = in / h;
  *tr = band * kBand + (in - q * h);
  *ts = int(q);
}

}  // namespace ss
