// Interface between the projections' launchers (ss_linear.hip) and their bf16
// matrix-core kernels, and the wide epilogue of the latter.
#pragma once

#include <type_traits>

#include "ss_linear.hpp"

namespace ss {

// O = R S^T on 256 x 256 (bf16, one split) or 128 x 128 tiles, as p.tiles_r,
// p.tiles_s and p.splits say; rt, st: whether t is the operand's contiguous axis
// (rt or not st).  An activation only with rt and st.
// Operands are read in 16-byte units: rows are 16-byte aligned, and a row's last
// unit is inside its storage, with zeros past the contraction's end where t is the
// contiguous axis.
enum class MmTile { kBig, kSmall, kSmallF32 };
void launch_mm(const MmParams& p, MmTile tile, bool rt, bool st, hipStream_t stream);

// O = R S^T for at most kRowsMax rows of R (t contiguous in both), with the
// epilogue; vec: both operands' rows are 16-byte aligned and nT is a whole number
// of 16-byte units.  One launch, no splits.
constexpr int64_t kRowsMax = 32;
void launch_rows(const MmParams& p, bool bf16, bool vec, hipStream_t stream);

__device__ __forceinline__ void store8(void* base, int64_t i, int bf16, const float (&v)[8]) {
  if (bf16) {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + i) =
        make_uint4(cvt_bf16x2(v[0], v[1]), cvt_bf16x2(v[2], v[3]), cvt_bf16x2(v[4], v[5]),
                   cvt_bf16x2(v[6], v[7]));
  } else {
    float4* d = reinterpret_cast<float4*>(static_cast<float*>(base) + i);
    d[0] = make_float4(v[0], v[1], v[2], v[3]);
    d[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}

// One element of the output, or of a split's partial sums.
template <int ACT>
__device__ __forceinline__ void epilogue1(const MmParams& p, int64_t r, int32_t s, float v,
                                          int split) {
  if (r >= p.nR || s >= p.nS) return;
  const int64_t o = r * p.nS + s;
  if (p.splits > 1) {
    p.part[split * p.nR * p.nS + o] = v;
    return;
  }
  if (p.bias) v += p.bias[s];
  if (p.pre) {
    if (p.pre_bf16) static_cast<uint16_t*>(p.pre)[o] = f32_to_bf16(v);
    else static_cast<float*>(p.pre)[o] = v;
  }
  v = apply_act(ACT, v);
  if (p.res)
    v += p.res_bf16 ? to_f32(static_cast<const uint16_t*>(p.res)[o])
                    : static_cast<const float*>(p.res)[o];
  if (p.out_bf16) static_cast<uint16_t*>(p.out)[o] = f32_to_bf16(v);
  else static_cast<float*>(p.out)[o] = v;
}

// Eight neighbours s..s+7 of output row r; nS and s are multiples of 8.
template <int ACT>
__device__ __forceinline__ void epilogue8(const MmParams& p, int64_t r, int32_t s, float (&v)[8],
                                          int split) {
  if (r >= p.nR || s >= p.nS) return;
  const int64_t o = r * p.nS + s;
  if (p.splits > 1) {
    store8(p.part, split * p.nR * p.nS + o, 0, v);
    return;
  }
  if (p.bias) {
    const float4 b0 = *reinterpret_cast<const float4*>(p.bias + s);
    const float4 b1 = *reinterpret_cast<const float4*>(p.bias + s + 4);
    v[0] += b0.x; v[1] += b0.y; v[2] += b0.z; v[3] += b0.w;
    v[4] += b1.x; v[5] += b1.y; v[6] += b1.z; v[7] += b1.w;
  }
  if (p.pre) store8(p.pre, o, p.pre_bf16, v);
  if constexpr (ACT != SS_ACT_NONE) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = apply_act(ACT, v[j]);
  }
  if (p.res) {
    if (p.res_bf16) {
      const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.res) + o);
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[2 * j] += __uint_as_float(u[j] << 16);
        v[2 * j + 1] += __uint_as_float(u[j] & 0xffff0000u);
      }
    } else {
      const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(p.res) + o);
      const float4 b0 = f[0], b1 = f[1];
      v[0] += b0.x; v[1] += b0.y; v[2] += b0.z; v[3] += b0.w;
      v[4] += b1.x; v[5] += b1.y; v[6] += b1.z; v[7] += b1.w;
    }
  }
  store8(p.out, o, p.out_bf16, v);
}

}  // namespace ss
