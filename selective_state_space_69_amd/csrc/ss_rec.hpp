// What the kernels of the gated linear recurrence share: its coefficients, decays in
// coded form, and the joining of stretches of time across a wave.
//
// Decays in coded form.  A step h <- a h + b with a near 1 is remembered for 1 / (1 - a)
// steps, so the rounding of a itself would add up to 2^-24 / (1 - a) of the state; a
// small a must not carry an error of the old state's size either.  So a decay is held
// as one float c: a - 1 (negative) while a > 3/4, a itself (not negative) below, both
// with full relative accuracy, and
//     a h + b = c h + b + (c < 0 ? h : 0).
// a = 1 is coded as the smallest negative normal number, an a below the smallest
// positive one as that; 0 is a start, which drops even an h that is not finite.
//
// Layout.  A wave holds 64 channels, four neighbours per lane (16 lanes), by four
// stretches of time (its rows of 16 lanes) of S steps each; a workgroup's waves follow
// each other in time.  Every lane runs its stretch from a zero state, keeping its total
// log decay and end state; the stretches are joined in the wave by row swaps and across
// waves in LDS, and each lane runs its steps again from its true state.
#pragma once

#include <type_traits>

#include "ss_device.hpp"

namespace ss {

constexpr int kRecChans = 64;                    // channels of a workgroup
constexpr float kOne = -1.17549435e-38f;         // the code of a = 1

struct RecShape {
  int64_t B, L;
  int32_t D, groups;          // groups: of 64 channels
  int64_t chunk;              // steps of a chunk, one workgroup's
  int32_t nchunks;
  float decay;
};

__device__ __forceinline__ float sigmoid(float v) { return hw_rcp(1.0f + hw_exp2(-v * kLog2e)); }

// log2 decay per unit of sigmoid(r): -c softplus(lam) log2 e
__device__ __forceinline__ float rec_rate(float decay, float lam) {
  return -decay * softplus_log2(lam * kLog2e);
}

__device__ __forceinline__ float rec_code(float E) {       // of a = 1 + E
  const float near = __builtin_fminf(E, kOne), far = __builtin_fmaxf(1.0f + E, -kOne);
  return E > -0.25f ? near : far;
}
// of a total log decay; CUT: minus infinity is a start's
template <bool CUT> __device__ __forceinline__ float rec_code_log2(float l2) {
  const float c = rec_code(precise_expm1(l2));
  return CUT && l2 == -__builtin_inff() ? 0.0f : c;
}

// a h + b.  CUT: there may be starts
template <bool CUT>
__device__ __forceinline__ float rec_apply(float c, float h, float b) {
  const float rest = c < 0.0f ? h : 0.0f, v = __builtin_fmaf(c, h, b) + rest;
  return CUT && c == 0.0f ? b : v;
}

// Four neighbouring channels of a row, as stored, so that a prefetch is not waited for.
template <typename T> struct Quad { typename Raw4<T>::type v; };
template <typename T> __device__ __forceinline__ void unpack(const Quad<T>& q, float (&v)[4]) {
  const float4 f = unpack4(q.v);
  v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
}
// n of four floats (a (B, D) array or lam; the others 0)
__device__ __forceinline__ void load_f32(const float* p, int n, float (&v)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = j < n ? p[j] : 0.0f;
}
__device__ __forceinline__ void store_f32(float* p, int n, const float (&v)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (j < n) p[j] = v[j];
}

// x of the lower and of the upper of each pair of rows (16 lanes), or of the halves of
// the wave, in both
__device__ __forceinline__ void swap_rows(float x, float& lower, float& upper) {
#if defined(__HIP_DEVICE_COMPILE__)
  const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  lower = __uint_as_float(p[0]);
  upper = __uint_as_float(p[1]);
#endif
}
__device__ __forceinline__ void swap_halves(float x, float& lower, float& upper) {
#if defined(__HIP_DEVICE_COMPILE__)
  const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  lower = __uint_as_float(p[0]);
  upper = __uint_as_float(p[1]);
#endif
}

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kS = 4;                       // steps of a lane's stretch
constexpr int kWaveSteps = 4 * kS;

// Which stretch of which channels a lane has.
struct Place {
  int lane, wv, sub, n;      // sub: row of the wave; n: channels that exist (0..4)
  int32_t b, chunk;
  int32_t c;                 // first channel (0 where none exists)
  __device__ __forceinline__ Place(const RecShape& s) {
    lane = threadIdx.x & 63;
    wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    sub = lane >> 4;
    const uint32_t id = uint32_t(xcd_contiguous(blockIdx.x, gridDim.x));
    const uint32_t row = id / uint32_t(s.groups);
    const int32_t g = int32_t(id - row * uint32_t(s.groups));
    b = int32_t(row / uint32_t(s.nchunks));
    chunk = int32_t(row - uint32_t(b) * uint32_t(s.nchunks));
    const int32_t c0 = g * kRecChans + (lane & 15) * 4;
    n = s.D - c0 < 4 ? s.D - c0 : 4;
    if (n <= 0) n = 0;
    c = n ? c0 : 0;
  }
};

// One tensor as a workgroup walks it: `p` is the first row of a block, a lane's stretch
// starts `first` bytes behind it.  Accesses take a scalar base and 32-bit lane offsets.
// ANY: rows at any element address and quads that end behind their row, read element by
// element; what lies behind the tensor's last element then reads 0.
template <bool ANY> struct Stream {
  const char* p;
  uint32_t first, row;       // bytes; row: from one row to the next
  int64_t left;              // ANY: bytes from p to the tensor's end
  // size: of an element
  __device__ __forceinline__ void init(const void* base, int64_t ld, uint32_t size,
                                       const RecShape& s, int64_t row0, int off, const Place& at) {
    p = static_cast<const char*>(base) + row0 * ld * size;
    row = uint32_t(ld) * size;
    first = at.n ? uint32_t(off) * row + uint32_t(at.c) * size : kOutOfRange;
    if constexpr (ANY) left = ((s.B * s.L - 1 - row0) * ld + s.D) * size;
  }
  __device__ __forceinline__ void move(int rows) {
    p += int64_t(rows) * row;
    if constexpr (ANY) left -= int64_t(rows) * row;
  }
  __device__ __forceinline__ Rsrc rsrc() const {
    int n = 0x7fffffff;
    if constexpr (ANY) n = left < 0x7fffffff ? int(left) : 0x7fffffff;
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(p), short(0), n, 0x00020000);
  }
};

// The rows of a lane's stretch of one tensor; those from `valid` on hold anything.
template <typename T, bool ANY> struct Rows {
  Quad<T> q[kS];
  __device__ __forceinline__ void load(const Stream<ANY>& st, int valid) {
    const Rsrc v = st.rsrc();
#pragma unroll
    for (int s = 0; s < kS; ++s) {
      if constexpr (!ANY) {
        const uint32_t at = s < valid ? st.first : kOutOfRange, row = uint32_t(s) * st.row;
        if constexpr (sizeof(T) == 4)
          q[s] = __builtin_bit_cast(Quad<T>, __builtin_amdgcn_raw_buffer_load_b128(v, at, row, 0));
        else
          q[s] = __builtin_bit_cast(Quad<T>, __builtin_amdgcn_raw_buffer_load_b64(v, at, row, 0));
      } else {
        const uint32_t at = s < valid ? st.first + uint32_t(s) * st.row : kOutOfRange;
        if constexpr (sizeof(T) == 4) {
          uint32_t e[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            e[j] = __builtin_amdgcn_raw_buffer_load_b32(v, at + 4 * j, 0, 0);
          q[s] = __builtin_bit_cast(Quad<T>, u32x4{e[0], e[1], e[2], e[3]});
        } else {
          uint32_t e[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            e[j] = uint16_t(__builtin_amdgcn_raw_buffer_load_b16(v, at + 2 * j, 0, 0));
          q[s] = __builtin_bit_cast(Quad<T>, u32x2{e[0] | e[1] << 16, e[2] | e[3] << 16});
        }
      }
    }
  }
  // Hides where the values come from: what was computed from them in front of this is
  // computed again behind it, rather than held in registers.
  __device__ __forceinline__ void fresh() {
#if defined(__HIP_DEVICE_COMPILE__)
#pragma unroll
    for (int s = 0; s < kS; ++s) {
      asm volatile("" : "+v"(q[s].v.x), "+v"(q[s].v.y));
      if constexpr (sizeof(T) == 4) asm volatile("" : "+v"(q[s].v.z), "+v"(q[s].v.w));
    }
#endif
  }
};

// Row s of a lane's stretch of a dense output, n channels (s from `valid` on: none).
// ANY: element by element.
template <typename T, bool ANY>
__device__ __forceinline__ void put(const Stream<ANY>& st, int s, int valid, int n,
                                    const float (&f)[4]) {
  const Rsrc v = st.rsrc();
  if constexpr (ANY) {
    const uint32_t at = s < valid ? st.first + uint32_t(s) * st.row : kOutOfRange;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      buf_store<T>(v, j < n ? at + j * uint32_t(sizeof(T)) : kOutOfRange, 0, f[j]);
  } else {
    const uint32_t at = s < valid ? st.first : kOutOfRange, row = uint32_t(s) * st.row;
    if constexpr (sizeof(T) == 2)
      __builtin_amdgcn_raw_buffer_store_b64(u32x2{cvt_bf16x2(f[0], f[1]), cvt_bf16x2(f[2], f[3])},
                                            v, at, row, 0);
    else
      __builtin_amdgcn_raw_buffer_store_b128(
          u32x4{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                __float_as_uint(f[3])}, v, at, row, 0);
  }
}

// A chunk's steps, counted from its first, and what the masks say of a lane's.
struct Masks {
  int steps;               // of the chunk
  int len;                 // those at and behind it leave the state as it is
  Rsrc starts;
  template <bool MASK>
  __device__ __forceinline__ void init(const uint8_t* st, const int32_t* lengths, int32_t b,
                                       int64_t L, int64_t t0, int64_t chunk) {
    steps = int(L - t0 < chunk ? L - t0 : chunk);
    len = steps;
    if constexpr (MASK) {
      if (lengths) {
        const int64_t v = lengths[b] - t0;
        len = v < 0 ? 0 : v < steps ? int(v) : steps;
      }
      starts = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(st) + b * L + t0, short(0),
                                                 st ? steps : 0, 0x00020000);
    }
  }
  // the marks of a lane's steps, from step `at` on
  __device__ __forceinline__ void marks(int at, bool (&m)[kS]) const {
#pragma unroll
    for (int s = 0; s < kS; ++s)
      m[s] = __builtin_amdgcn_raw_buffer_load_b8(starts, uint32_t(at + s), 0, 0) != 0;
  }
};

// f(Z, MASK, ANY) as constants; rows at any address take the masked kernels
template <typename F> void rec_by_flags(bool z, bool mask, bool any, F&& f) {
  using Y = std::integral_constant<bool, true>;
  using N = std::integral_constant<bool, false>;
  if (z) {
    if (any) f(Y{}, Y{}, Y{});
    else if (mask) f(Y{}, Y{}, N{});
    else f(Y{}, N{}, N{});
  } else {
    if (any) f(N{}, Y{}, Y{});
    else if (mask) f(N{}, Y{}, N{});
    else f(N{}, N{}, N{});
  }
}

inline RecShape rec_shape(const ss_rec_desc_t& d, const RecPlan& pl) {
  return RecShape{d.batch, d.seqlen, int32_t(d.dim), int32_t((d.dim + kRecChans - 1) / kRecChans),
                  pl.chunk, int32_t(pl.nchunks), d.decay};
}
inline int64_t stride_of(int64_t stride, int64_t dim) { return stride ? stride : dim; }
// whether quads of bf16 rows are not 4-byte aligned
inline bool odd_rows(const void* p, int64_t ld, int32_t dtype) {
  return p && dtype == SS_BF16 && (ld % 2 != 0 || reinterpret_cast<uintptr_t>(p) % 4 != 0);
}

// Chunks' end states (from a zero start) to their start states, or in reverse the
// adjoints that leave them (with none entering) to those that enter.
void launch_rec_carry(const float* clog, float* carry, const float* first, int64_t batch,
                      int32_t D, int32_t nchunks, bool reverse, hipStream_t stream);

}  // namespace ss
