// What the kernels of the gated linear recurrence share: its coefficients, the rows of a
// workgroup, and the joining of stretches of time.
//
// Layout.  A workgroup holds kRecChans channels, two neighbours per lane; a wave's lanes
// hold kSubs stretches of time of S steps each, its waves follow each other in time.
// Every lane runs its stretch from a zero state; a stretch is then summed up by its decay P
// (the exponential of the sum of log decays) and its end state s, h <- P h + s.  Stretches are
// joined in the wave by row swaps and across waves in LDS, and each lane runs its steps again
// from its true state.
//
// Accuracy.  A state that a step hardly decays is remembered for 1 / (1 - a) steps, and a
// decay rounded to fp32 wherever it meets the state that is carried on would add up to 2^-24 /
// (1 - a) of it, every time to the same side where the gates repeat.  Decays of steps and
// stretches therefore stay within their wave.  A wave's and a chunk's are sums of logs, and
// are applied as a - 1 where they are near 1, h <- h + ((a - 1) h + s) (rec_decay_of,
// rec_apply).  The state's own rounding would add up the same way, half a step at every join:
// it is carried on as a sum of two numbers (Carry).  sqrt(1 - a^2) comes from a - 1 with full
// relative accuracy (a series near 0).  Inputs of one sign over 262144 steps, 1 - a from 1e-13
// to 5e-4: states and adjoints are 1.2e-6 of themselves off at most (9.3e-4 with fp32 decays
// all the way; 8 x 2048 x 2560 forward 118 -> 121 us, backward 242 -> 245).
#pragma once

#include <type_traits>

#include "ss_device.hpp"

namespace ss {

constexpr int kV = 2;                            // channels of a lane
constexpr int kRecLanes = 16;                    // lanes of one step's channels
constexpr int kRecChans = kV * kRecLanes;        // channels of a workgroup
constexpr int kSubs = 64 / kRecLanes;            // stretches of a wave
constexpr float kTiny = 1.17549435e-38f;         // smallest normal number

struct RecShape {
  int64_t B, L;
  int32_t D, groups;          // groups: of kRecChans channels
  int64_t chunk;              // steps of a chunk, one workgroup's
  int32_t nchunks;
  float decay;
};

__device__ __forceinline__ float sigmoid(float v) { return hw_rcp(1.0f + hw_exp2(-v * kLog2e)); }

// log2 decay per unit of sigmoid(r): -c softplus(lam) log2 e
__device__ __forceinline__ float rec_rate(float decay, float lam) {
  return -decay * softplus_log2(lam * kLog2e);
}

// A step's decay a, E = a - 1 and sqrt(1 - a^2) from its log2 decay.
struct Decay { float a, E, beta; };
__device__ __forceinline__ Decay rec_decay(float l2) {
  const float a = hw_exp2(l2), near = l2 * expm1_factor(l2), far = a - 1.0f;
  const float E = __builtin_unpredictable(l2 > -kSeries2) ? near : far;
  return Decay{a, E, __builtin_amdgcn_sqrtf(-E * (2.0f + E))};
}

// Steps.  CUT: there may be starts, whose decay is 0; every other one is at least kTiny, added
// so that a NaN stays one (a maximum drops it), and changes no decay above 2^-102: a start
// drops even a state that is not finite, and a gate that is NaN reaches all of its document,
// forward and backward, as it does without CUT.
template <bool CUT> __device__ __forceinline__ float step_decay(float a, bool cut) {
  return CUT ? (cut ? 0.0f : a + kTiny) : a;
}
// h decayed, and b added
template <bool CUT> __device__ __forceinline__ float step_apply(float a, float h, float b) {
  const float v = __builtin_fmaf(a, h, b);
  return CUT && a == 0.0f ? b : v;
}

// one decay after the other
template <bool CUT> __device__ __forceinline__ float step_both(float p, float q) {
  const float v = p * q, w = v + kTiny;
  return CUT ? (__builtin_fminf(p, q) == 0.0f ? 0.0f : w) : v;
}

// Stretches.  Their log2 decays are at most 0 and add up; that of one with a start is -infinity.
// (CUT: no other one is, nor a NaN, which the end state and the leaving adjoint carry on.)
constexpr float kCutLog = -__builtin_inff();
template <bool CUT> __device__ __forceinline__ float stretch_log(float l, bool cut) {
  const float v = __builtin_fmaxf(l, -1e30f);
  return CUT ? (cut ? kCutLog : v) : l;
}
// A decay as it is applied: a - 1, and then below 0, where a is near 1, else a (of CUT: 0 for
// a start alone).
constexpr float kNoDecay = -kTiny;
template <bool CUT> __device__ __forceinline__ float rec_decay_of(float l2) {
  const float near = __builtin_fmaf(l2, expm1_factor(l2), kNoDecay);
  float far = hw_exp2(l2);
  if (CUT) far += l2 == kCutLog ? 0.0f : kTiny;
  return __builtin_unpredictable(l2 > -kSeries2) ? near : far;
}
template <bool CUT> __device__ __forceinline__ float rec_apply(float q, float h0, float b) {
  const float h = CUT && q == 0.0f ? 0.0f : h0;
  return __builtin_fmaf(q, h, b) + (q < 0.0f ? h : 0.0f);
}
// A state (or adjoint) between blocks, base + rest: joins near 1 add to the rest, whose
// rounding is that of what a block adds; others start a new one.
struct Carry {
  float base, rest;
  __device__ __forceinline__ float value() const { return base + rest; }
  template <bool CUT> __device__ __forceinline__ void apply(float q, float b) {
    const bool near = q < 0.0f;
    const float v = value(), h = CUT && q == 0.0f ? 0.0f : v;
    rest = __builtin_fmaf(q, h, b) + (near ? rest : 0.0f);
    base = near ? base : 0.0f;
  }
  // base becomes the value, rest what that leaves
  __device__ __forceinline__ void settle() {
    const float v = value();
    rest -= v - base;
    base = v;
  }
};

// A lane's channels of a row, as stored, so that a prefetch is not waited for.
template <typename T> constexpr int kWords = kV * int(sizeof(T)) / 4;
template <typename T> struct Chans { uint32_t w[kWords<T>]; };
__device__ __forceinline__ void unpack(const Chans<float>& q, float (&v)[kV]) {
#pragma unroll
  for (int j = 0; j < kV; ++j) v[j] = __uint_as_float(q.w[j]);
}
__device__ __forceinline__ void unpack(const Chans<uint16_t>& q, float (&v)[kV]) {
#pragma unroll
  for (int j = 0; j < kV; ++j)
    v[j] = __uint_as_float(j & 1 ? q.w[j / 2] & 0xffff0000u : q.w[j / 2] << 16);
}
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
template <typename T>
__device__ __forceinline__ Chans<T> buf_chans(Rsrc v, uint32_t at, uint32_t row) {
  if constexpr (kWords<T> == 1)
    return __builtin_bit_cast(Chans<T>, __builtin_amdgcn_raw_buffer_load_b32(v, at, row, 0));
  else
    return __builtin_bit_cast(Chans<T>, __builtin_amdgcn_raw_buffer_load_b64(v, at, row, 0));
}
template <typename T>
__device__ __forceinline__ void buf_put(Rsrc v, uint32_t at, uint32_t row, const float (&f)[kV]) {
  Chans<T> q;
#pragma unroll
  for (int j = 0; j < kWords<T>; ++j)
    q.w[j] = sizeof(T) == 2 ? cvt_bf16x2(f[2 * j % kV], f[(2 * j + 1) % kV]) : __float_as_uint(f[j]);
  if constexpr (kWords<T> == 1)
    __builtin_amdgcn_raw_buffer_store_b32(q.w[0], v, at, row, 0);
  else
    __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, q), v, at, row, 0);
}
// A lane's n channels of a (D) row of floats; others repeat the first.
__device__ __forceinline__ void load_f32(const float* p, int n, float (&v)[kV]) {
#pragma unroll
  for (int j = 0; j < kV; ++j) v[j] = p[j < n ? j : 0];
}
__device__ __forceinline__ void store_f32(float* p, int n, const float (&v)[kV]) {
#pragma unroll
  for (int j = 0; j < kV; ++j)
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

// The stretches of a wave, joined: (P, s) of the lane's own on entry, of the whole wave on
// return; (Px, sx): of the stretches in front of the lane's.
template <bool CUT>
__device__ __forceinline__ void join_up(int sub, float& P, float& s, float& Px, float& sx) {
  float p0, p1, s0, s1;
  swap_rows(P, p0, p1);
  swap_rows(s, s0, s1);
  Px = sub & 1 ? p0 : 1.0f;
  sx = sub & 1 ? s0 : 0.0f;
  swap_halves(step_both<CUT>(p0, p1), p0, P);
  swap_halves(step_apply<CUT>(p1, s0, s1), s0, s);
  const float q = step_both<CUT>(p0, Px), t = step_apply<CUT>(Px, s0, sx);
  Px = sub & 2 ? q : Px;
  sx = sub & 2 ? t : sx;
  s = step_apply<CUT>(P, s0, s);
  P = step_both<CUT>(p0, P);
}
// Both walks of a backward pass: forward as above, and q, what leaves a stretch at its
// first step, joined from behind; (Py, qy): of the stretches behind the lane's.
template <bool CUT, bool UP>
__device__ __forceinline__ void join_both(int sub, float& P, float& s, float& q, float& Px,
                                          float& sx, float& Py, float& qy) {
  float p0, p1, q0, q1, r0, r1, u0, u1;
  swap_rows(P, p0, p1);
  swap_rows(q, q0, q1);
  Py = sub & 1 ? 1.0f : p1;
  qy = sub & 1 ? 0.0f : q1;
  swap_halves(step_both<CUT>(p0, p1), r0, r1);
  swap_halves(step_apply<CUT>(p0, q1, q0), u0, u1);
  q = step_apply<CUT>(r0, u1, u0);
  const float y = step_both<CUT>(Py, r1), v = step_apply<CUT>(Py, u1, qy);
  Py = sub & 2 ? Py : y;
  qy = sub & 2 ? qy : v;
  if constexpr (UP) {
    float s0, s1, t0, t1;
    swap_rows(s, s0, s1);
    Px = sub & 1 ? p0 : 1.0f;
    sx = sub & 1 ? s0 : 0.0f;
    swap_halves(step_apply<CUT>(p1, s0, s1), t0, t1);
    s = step_apply<CUT>(r1, t0, t1);
    const float x = step_both<CUT>(r0, Px), w = step_apply<CUT>(Px, t0, sx);
    Px = sub & 2 ? x : Px;
    sx = sub & 2 ? w : sx;
  }
  P = step_both<CUT>(r0, r1);
}
// Runs of chunks in the lanes of a wave, joined: (l, s) of the lane's own on entry, of the
// whole wave on return.  A run is long: its decay is applied as rec_apply does.
template <bool CUT> __device__ __forceinline__ void join_runs(float& l, float& s) {
  float l0, l1, d0, d1, s0, s1;
  swap_rows(l, l0, l1);
  swap_rows(rec_decay_of<CUT>(l), d0, d1);
  swap_rows(s, s0, s1);
  l = l0 + l1;
  s = rec_apply<CUT>(d1, s0, s1);
  swap_halves(l, l0, l1);
  swap_halves(rec_decay_of<CUT>(l), d0, d1);
  swap_halves(s, s0, s1);
  l = l0 + l1;
  s = rec_apply<CUT>(d1, s0, s1);
}
// The log decay of a wave's stretches, from the lane's own
__device__ __forceinline__ float wave_log(float l) {
  float a, b;
  swap_rows(l, a, b);
  swap_halves(a + b, a, b);
  return a + b;
}

// Which stretch of which channels a lane has.
struct Place {
  int lane, wv, sub, n;      // sub: stretch of the wave; n: channels that exist (0..kV)
  int32_t b, chunk;
  int32_t c;                 // first channel (0 where none exists)
  // back: the workgroups in reverse order
  __device__ __forceinline__ Place(const RecShape& s, bool back) {
    lane = threadIdx.x & 63;
    wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    sub = lane / kRecLanes;
    const uint32_t id0 = uint32_t(xcd_contiguous(blockIdx.x, gridDim.x));
    const uint32_t id = back ? gridDim.x - 1 - id0 : id0;
    const uint32_t row = id / uint32_t(s.groups);
    const int32_t g = int32_t(id - row * uint32_t(s.groups));
    b = int32_t(row / uint32_t(s.nchunks));
    chunk = int32_t(row - uint32_t(b) * uint32_t(s.nchunks));
    const int32_t c0 = g * kRecChans + lane % kRecLanes * kV;
    n = s.D - c0 < kV ? s.D - c0 : kV;
    if (n <= 0) n = 0;
    c = n ? c0 : 0;
  }
};

// The floats of a lane's channels in LDS.
struct alignas(4 * kV) Floats { float v[kV]; };
__device__ __forceinline__ void put_lds(float* p, const float (&v)[kV]) {
  Floats f;
#pragma unroll
  for (int j = 0; j < kV; ++j) f.v[j] = v[j];
  *reinterpret_cast<Floats*>(p) = f;
}
__device__ __forceinline__ Floats get_lds(const float* p) {
  return *reinterpret_cast<const Floats*>(p);
}

// A chunk's log decay, of a wave's stretches block after block: sum + rest, so that its rounding
// does not grow with the blocks.
struct LogSum {
  float sum = 0.0f, rest = 0.0f;
  __device__ __forceinline__ void add(float l) {
    const float v = sum + l;
    rest += l - (v - sum);
    sum = v;
  }
  __device__ __forceinline__ float value() const { return sum == kCutLog ? kCutLog : sum + rest; }
};

// What the chunks in front of one's own do to a state, folded by the whole workgroup:
// logs[k], end[k] (from a zero start), k < n, are `step` floats apart.  The lanes of a
// channel take equal runs of them, which are joined as stretches are, through tc and ts
// (kWaves rows each); H is advanced.
template <bool CUT, int kWaves>
__device__ __forceinline__ void fold_chunks(const float* logs, const float* end, int64_t step,
                                            int n, const Place& at, float (*tc)[kRecChans],
                                            float (*ts)[kRecChans], Carry (&H)[kV]) {
  const int units = kWaves * kSubs, per = (n + units - 1) / units;
  const int k0 = (at.wv * kSubs + at.sub) * per, k1 = k0 + per < n ? k0 + per : n;
  const int li = at.lane % kRecLanes * kV;
  float l[kV], s[kV];
#pragma unroll
  for (int j = 0; j < kV; ++j) l[j] = s[j] = 0.0f;
#pragma unroll 4
  for (int k = k0; k < k1; ++k) {
    float p[kV], e[kV];
    load_f32(logs + k * step, at.n, p);
    load_f32(end + k * step, at.n, e);
#pragma unroll
    for (int j = 0; j < kV; ++j) {
      s[j] = rec_apply<CUT>(rec_decay_of<CUT>(p[j]), s[j], e[j]);
      l[j] = l[j] + p[j];
    }
  }
#pragma unroll
  for (int j = 0; j < kV; ++j) {
    join_runs<CUT>(l[j], s[j]);
    l[j] = rec_decay_of<CUT>(l[j]);
  }
  if (at.sub == 0) {
    put_lds(&tc[at.wv][li], l);
    put_lds(&ts[at.wv][li], s);
  }
  __syncthreads();
#pragma unroll 2
  for (int w = 0; w < kWaves; ++w) {
    const Floats cv = get_lds(&tc[w][li]), sv = get_lds(&ts[w][li]);
#pragma unroll
    for (int j = 0; j < kV; ++j) H[j].template apply<CUT>(cv.v[j], sv.v[j]);
  }
#pragma unroll
  for (int j = 0; j < kV; ++j) H[j].settle();
}
// The waves' log decays of a chunk, added, in all of a channel's lanes.  box: kWaves rows that
// no wave reads any more.
template <int kWaves>
__device__ __forceinline__ void sum_logs(const Place& at, float (*box)[kRecChans],
                                         const LogSum (&sum)[kV], float (&l)[kV]) {
  const int li = at.lane % kRecLanes * kV;
#pragma unroll
  for (int j = 0; j < kV; ++j) l[j] = sum[j].value();
  __syncthreads();
  if (at.sub == 0) put_lds(&box[at.wv][li], l);
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kV; ++j) l[j] = 0.0f;
  for (int w = 0; w < kWaves; ++w) {
    const Floats v = get_lds(&box[w][li]);
#pragma unroll
    for (int j = 0; j < kV; ++j) l[j] = l[j] + v.v[j];
  }
}

// One tensor as a workgroup walks it: `p` is the first row of a block, a lane's stretch
// starts `first` bytes behind it.  Accesses take a scalar base and 32-bit lane offsets.
// ANY: rows at any element address and pairs that end behind their row, read element by
// element; what lies behind the tensor's last element then reads 0.
template <bool ANY> struct Stream {
  const char* p;
  uint32_t first, row;       // bytes; row: from one row to the next
  int64_t left;              // ANY: bytes from p to the tensor's end (negative behind it)
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
    if constexpr (ANY) n = left < 0 ? 0 : left < 0x7fffffff ? int(left) : 0x7fffffff;
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(p), short(0), n, 0x00020000);
  }
};

// The rows of a lane's stretch of one tensor; those from `valid` on hold anything.
template <typename T, int S, bool ANY> struct Rows {
  Chans<T> q[S];
  __device__ __forceinline__ void load(const Stream<ANY>& st, int valid) {
    const Rsrc v = st.rsrc();
#pragma unroll
    for (int s = 0; s < S; ++s) {
      if constexpr (!ANY) {
        q[s] = buf_chans<T>(v, s < valid ? st.first : kOutOfRange, uint32_t(s) * st.row);
      } else {
        const uint32_t at = s < valid ? st.first + uint32_t(s) * st.row : kOutOfRange;
        if constexpr (sizeof(T) == 4) {
#pragma unroll
          for (int j = 0; j < kV; ++j)
            q[s].w[j] = __builtin_amdgcn_raw_buffer_load_b32(v, at + 4 * j, 0, 0);
        } else {
#pragma unroll
          for (int j = 0; j < kV; j += 2) {
            const uint32_t e0 = uint16_t(__builtin_amdgcn_raw_buffer_load_b16(v, at + 2 * j, 0, 0));
            const uint32_t e1 =
                uint16_t(__builtin_amdgcn_raw_buffer_load_b16(v, at + 2 * j + 2, 0, 0));
            q[s].w[j / 2] = e0 | e1 << 16;
          }
        }
      }
    }
  }
  // Hides where the values come from: what was computed from them in front of this is
  // computed again behind it, rather than held in registers.
  __device__ __forceinline__ void fresh() {
#if defined(__HIP_DEVICE_COMPILE__)
#pragma unroll
    for (int s = 0; s < S; ++s) {
#pragma unroll
      for (int j = 0; j < kWords<T>; ++j) asm volatile("" : "+v"(q[s].w[j]));
    }
#endif
  }
};

// Row s of a lane's stretch of a dense output, n channels (s from `valid` on: none).
// ANY: element by element.
template <typename T, bool ANY>
__device__ __forceinline__ void put(const Stream<ANY>& st, int s, int valid, int n,
                                    const float (&f)[kV]) {
  const Rsrc v = st.rsrc();
  if constexpr (ANY) {
    const uint32_t at = s < valid ? st.first + uint32_t(s) * st.row : kOutOfRange;
#pragma unroll
    for (int j = 0; j < kV; ++j)
      buf_store<T>(v, j < n ? at + j * uint32_t(sizeof(T)) : kOutOfRange, 0, f[j]);
  } else {
    buf_put<T>(v, s < valid ? st.first : kOutOfRange, uint32_t(s) * st.row, f);
  }
}

// A chunk's steps, counted from its first, and what the masks say of a lane's.
struct Masks {
  int steps;               // of the chunk
  int len;                 // those at and behind it leave the state as it is, and are not read
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
  template <int S> __device__ __forceinline__ void marks(int at, bool (&m)[S]) const {
#pragma unroll
    for (int s = 0; s < S; ++s)
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
// whether pairs of bf16 rows are not 4-byte aligned
inline bool odd_rows(const void* p, int64_t ld, int32_t dtype) {
  return p && dtype == SS_BF16 && (ld % 2 != 0 || reinterpret_cast<uintptr_t>(p) % 4 != 0);
}

}  // namespace ss
