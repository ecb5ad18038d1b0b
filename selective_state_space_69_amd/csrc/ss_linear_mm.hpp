// Interface between the projections' launchers (ss_linear.hip) and their bf16
// matrix-core kernels, and the wide epilogue of the latter.
#pragma once

#include <type_traits>

#include "ss_linear.hpp"

namespace ss {

// O = R S^T on 256 x 256 (bf16, one split), 128 x 128 (bf16) or 64 x 64 (fp32) tiles,
// as p.tiles_r, p.tiles_s and p.splits say; rt, st: whether t is the operand's contiguous axis
// (rt or not st).  An activation only with rt and st.
// Operands are read in 16-byte units: rows are 16-byte aligned, and a row's last
// unit is inside its storage, with zeros past the contraction's end where t is the
// contiguous axis.
// kSmallPair: 128 x 128 tiles by two groups of waves, at most one tile per CU.
// kSmallF32Any: operands at any element address, of any row length; nothing past a row
// is read.
// kSmallSingle: 128 x 128 tiles, four to a CU (three with a residual), with one buffer each.
enum class MmTile { kBig, kSmall, kSmallPair, kSmallSingle, kSmallF32, kSmallF32Any };
// sum2 (bf16, not with rt and st): R's values are sums of two bf16.
void launch_mm(const MmParams& p, MmTile tile, bool rt, bool st, bool sum2, hipStream_t stream);
// dx (rt, not st) and dw (neither) in one launch; not on kSmallSingle.  kBig: the
// workgroups below `behind`, those that dw's last round reaches (0: it reaches all),
// take `few` of dx's tiles each, the others the rest.
void launch_mm_both(const MmParams& dx, const MmParams& dw, MmTile tile, int behind, int few,
                    bool sum2, hipStream_t stream);

// O = R S^T for at most kRowsMax rows of R (t contiguous in both), with the
// epilogue; vec: both operands' rows are 16-byte aligned and nT is a whole number
// of 16-byte units.  One launch, no splits.
constexpr int64_t kRowsMax = 32;
void launch_rows(const MmParams& p, bool bf16, bool vec, hipStream_t stream);

// Accesses of the epilogue: to global memory (said so, since the parameters may have
// come back from memory as plain words), eight neighbours at any element address
// (16-byte accesses need no alignment).
template <typename T> using Global = __attribute__((address_space(1))) T;
typedef uint32_t Halves8 __attribute__((ext_vector_type(4), aligned(2)));
typedef float Floats4 __attribute__((ext_vector_type(4), aligned(4)));

// STREAM: bf16 past the caches, for outputs larger than they are (16384 x 10240: 676
// -> 662 us; they keep the operands instead).  fp32 goes through them: its two
// 16-byte halves of a lane make whole lines only there (16384 x 5120: 370 us, 382
// streamed).
template <bool STREAM = false>
__device__ __forceinline__ void store8(void* base, int64_t i, int bf16, const float (&v)[8]) {
  if (bf16) {
    Global<Halves8>* d = (Global<Halves8>*)((Global<uint16_t>*)base + i);
    const Halves8 x{cvt_bf16x2(v[0], v[1]), cvt_bf16x2(v[2], v[3]), cvt_bf16x2(v[4], v[5]),
                    cvt_bf16x2(v[6], v[7])};
    if constexpr (STREAM) __builtin_nontemporal_store(x, d);
    else *d = x;
  } else {
    Global<float>* d = (Global<float>*)base + i;
    *(Global<Floats4>*)d = Floats4{v[0], v[1], v[2], v[3]};
    *(Global<Floats4>*)(d + 4) = Floats4{v[4], v[5], v[6], v[7]};
  }
}
__device__ __forceinline__ void load8(const float* src, float (&v)[8]) {
  const Global<Floats4>* s = (const Global<Floats4>*)src;
  const Floats4 a = *s, b = *(const Global<Floats4>*)((const Global<float>*)src + 4);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[j] = a[j];
    v[4 + j] = b[j];
  }
}
__device__ __forceinline__ void store1(void* base, int64_t i, int bf16, float v) {
  if (bf16) ((Global<uint16_t>*)base)[i] = f32_to_bf16(v);
  else ((Global<float>*)base)[i] = v;
}
__device__ __forceinline__ float load1(const void* base, int64_t i, int bf16) {
  return bf16 ? to_f32(uint16_t(((const Global<uint16_t>*)base)[i]))
              : float(((const Global<float>*)base)[i]);
}

// One element of the output: bias, activation, residual, stores.
__device__ __forceinline__ void epilogue1(const MmParams& p, int act, int64_t r, int32_t s,
                                          float v) {
  const int64_t o = r * p.nS + s;
  if (p.bias) v += load1(p.bias, s, 0);
  if (p.pre) store1(p.pre, o, p.pre_bf16, v);
  v = apply_act(act, v);
  if (p.res) v += load1(p.res, o, p.res_bf16);
  store1(p.out, o, p.out_bf16, v);
}

// Eight neighbours of the residual from element o on, fetched ahead in their storage
// form; left unset where there is none (to clear it for nothing costs as much as the
// rest of a piece's addresses).
struct Res8 { uint32_t w[8]; };
__device__ __forceinline__ Res8 fetch_res8(const MmParams& p, int64_t o, bool inside) {
  Res8 f;
  if (p.res && inside) {
    if (p.res_bf16) {
      const Halves8 h = *(const Global<Halves8>*)((const Global<uint16_t>*)p.res + o);
#pragma unroll
      for (int j = 0; j < 4; ++j) f.w[j] = h[j];
    } else {
      float v[8];
      load8(static_cast<const float*>(p.res) + o, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) f.w[j] = __float_as_uint(v[j]);
    }
  }
  return f;
}

// Eight neighbours of an output row from element o on, all inside it; bias: theirs (0
// without one).  ACT: the activation, or kActOf for p.act.
constexpr int kActOf = -1;
template <int ACT, bool STREAM = false, bool RES = true>
__device__ __forceinline__ void epilogue8(const MmParams& p, int64_t o, float (&v)[8],
                                          const float (&bias)[8], const Res8& res) {
  const int act = ACT == kActOf ? p.act : ACT;
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] += bias[j];
  if (p.pre) store8<STREAM>(p.pre, o, p.pre_bf16, v);
  if (act != SS_ACT_NONE) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = apply_act(act, v[j]);
  }
  if (RES && p.res) {
    if (p.res_bf16) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[2 * j] += __uint_as_float(res.w[j] << 16);
        v[2 * j + 1] += __uint_as_float(res.w[j] & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] += __uint_as_float(res.w[j]);
    }
  }
  store8<STREAM>(p.out, o, p.out_bf16, v);
}

}  // namespace ss
