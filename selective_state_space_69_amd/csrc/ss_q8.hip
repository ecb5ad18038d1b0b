// Rows as 8-bit integers with one scale each, for gfx950.
//
// A row is read once: its elements stay in registers between the largest magnitude
// (taken on the bits, where NaN and infinity are above every number) and the quotients.
// 127 x / max is formed in 32 bits, with an error below 2^-15 (127 times three roundings
// of 2^-24); where that leaves the nearest whole number open (within 2^-13 of a tie, one
// value in 4096) 254 |x| is compared with (2 k + 1) max, both exact in 64 bits.  So the
// bits are those of the definition.  Memory bound.
#include "ss_device.hpp"

namespace ss {
namespace {

constexpr int kThreads = 256;
constexpr int64_t kMaxBlocks = int64_t(1) << 22;    // a grid's threads stay below 2^32

struct PackParams {
  const void* x;
  int8_t* q;
  float* s;
  int64_t rows, ldx, ldq;
  int32_t dim, span;       // span: bytes of a row of q that are written
};

// 8 neighbours from element c of n on, at any element address (0 past the end)
template <typename T> struct Eight {
  T e[8];
  __device__ __forceinline__ void load(const T* row, int c, int n) {
    struct __attribute__((packed, aligned(sizeof(T)))) Any { T e[8]; };
    if (c + 8 <= n) {
      const Any a = *reinterpret_cast<const Any*>(row + c);
#pragma unroll
      for (int j = 0; j < 8; ++j) e[j] = a.e[j];
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) e[j] = c + j < n ? row[c + j] : T(0);
    }
  }
  __device__ __forceinline__ uint32_t top() const {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t b = __float_as_uint(to_f32(e[j])) & 0x7fffffffu;
      m = b > m ? b : m;
    }
    return m;
  }
};

// scale: 127 / most, or 0 where that is too large for fp32 (then the quotient is formed
// in 64 bits)
__device__ __forceinline__ int nearest(float x, float scale, float most) {
  const float t = x * scale;
  int k = int(__builtin_rintf(t));
  const float f = __builtin_fabsf(t) - __builtin_floorf(__builtin_fabsf(t));
  if (__builtin_fabsf(f - 0.5f) < 0x1p-13f || scale == 0.0f) {
    const double a = 254.0 * __builtin_fabs(double(x)), m = double(most);
    // within one of the quotient's whole part: the comparisons settle it
    int n = int(scale == 0.0f ? a / (2.0 * m) : double(__builtin_fabsf(t)));
    if (a < 2.0 * n * m) --n;
    if (a >= 2.0 * (n + 1) * m) ++n;
    const double b = (2 * n + 1) * m;
    n += a > b || (a == b && (n & 1));
    k = x < 0.0f ? -n : n;
  }
  return k;
}

template <typename T>
__device__ __forceinline__ void store_eight(int8_t* row, int c, int span, const Eight<T>& v,
                                            float scale, float most, bool zero) {
  uint32_t w[2] = {0, 0};
  if (!zero) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      w[j / 4] |= uint32_t(nearest(to_f32(v.e[j]), scale, most) & 255) << (8 * (j % 4));
  }
  if (c + 8 <= span) {
    struct __attribute__((packed, aligned(1))) Any { uint32_t w[2]; };
    *reinterpret_cast<Any*>(row + c) = Any{{w[0], w[1]}};
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (c + j < span) row[c + j] = int8_t(w[j / 4] >> (8 * (j % 4)));
  }
}

// N vectors of 8 per thread, W waves to a row; N = 0: a row longer than registers hold
// is read twice.
template <typename T, int N, int W>
__global__ __launch_bounds__(kThreads) void pack_kernel(PackParams p) {
  __shared__ uint32_t tops[kThreads / 64];
  constexpr int kPer = 64 * W;                      // threads of a row
  constexpr int kRows = kThreads / kPer;
  const int tid = threadIdx.x % kPer;
  for (int64_t r0 = int64_t(blockIdx.x) * kRows; r0 < p.rows; r0 += int64_t(gridDim.x) * kRows) {
    const int64_t row = r0 + threadIdx.x / kPer;
    const bool here = row < p.rows;
    const T* x = static_cast<const T*>(p.x) + (here ? row : p.rows - 1) * p.ldx;
    Eight<T> v[N ? N : 1];
    uint32_t top = 0;
    if constexpr (N > 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i].load(x, (i * kPer + tid) * 8, p.dim);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const uint32_t m = v[i].top();
        top = m > top ? m : top;
      }
    } else {
      for (int c = tid * 8; c < p.dim; c += kPer * 8) {
        v[0].load(x, c, p.dim);
        const uint32_t m = v[0].top();
        top = m > top ? m : top;
      }
    }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) {
      const uint32_t o = uint32_t(__shfl_xor(int(top), d));
      top = o > top ? o : top;
    }
    if constexpr (W > 1) {
      __syncthreads();
      if ((threadIdx.x & 63) == 0) tops[threadIdx.x / 64] = top;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < W; ++w) top = tops[w] > top ? tops[w] : top;
    }
    const bool finite = top < 0x7f800000u, zero = !finite || top == 0;
    const float most = __uint_as_float(top);
    const float scale = most > 1e-35f ? 127.0f / most : 0.0f;
    if (!here) continue;
    int8_t* q = p.q + row * p.ldq;
    if (tid == 0) p.s[row] = finite ? most / 127.0f : __uint_as_float(0x7fc00000u);
    if constexpr (N > 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int c = (i * kPer + tid) * 8;
        if (c < p.span) store_eight(q, c, p.span, v[i], scale, most, zero);
      }
    } else {
      for (int c = tid * 8; c < p.span; c += kPer * 8) {
        v[0].load(x, c, p.dim);
        store_eight(q, c, p.span, v[0], scale, most, zero);
      }
    }
  }
}

template <typename T, int N>
void run_narrow(const PackParams& p, hipStream_t st) {
  const int64_t n = (p.rows + 3) / 4;
  pack_kernel<T, N, 1><<<unsigned(n < kMaxBlocks ? n : kMaxBlocks), kThreads, 0, st>>>(p);
}
template <typename T, int N>
void run_wide(const PackParams& p, hipStream_t st) {
  pack_kernel<T, N, 4><<<unsigned(p.rows < kMaxBlocks ? p.rows : kMaxBlocks), kThreads, 0, st>>>(p);
}
template <typename T>
void run(const PackParams& p, hipStream_t st) {
  // a wave to a row where the rows then still fill the GPU, else four
  if (p.span <= 4096 && p.rows >= 1024) {
    switch ((p.span + 511) / 512) {
      case 1: return run_narrow<T, 1>(p, st);
      case 2: return run_narrow<T, 2>(p, st);
      case 3: return run_narrow<T, 3>(p, st);
      case 4: return run_narrow<T, 4>(p, st);
      case 5: return run_narrow<T, 5>(p, st);
      case 6: return run_narrow<T, 6>(p, st);
      default: return run_narrow<T, 8>(p, st);
    }
  }
  if (p.span <= 2048) run_wide<T, 1>(p, st);
  else if (p.span <= 4096) run_wide<T, 2>(p, st);
  else if (p.span <= 8192) run_wide<T, 4>(p, st);
  else run_wide<T, 0>(p, st);
}

}  // namespace

int launch_q8_pack(const ss_q8_pack_desc_t& d, const void* x, int8_t* q, float* s, void* stream) {
  const int64_t ldq = d.q_stride ? d.q_stride : d.dim;
  const PackParams p{x, q, s, d.rows, d.x_stride ? d.x_stride : d.dim, ldq, int32_t(d.dim),
                     int32_t(ldq)};
  if (d.dtype == SS_BF16) run<uint16_t>(p, static_cast<hipStream_t>(stream));
  else run<float>(p, static_cast<hipStream_t>(stream));
  return int(hipGetLastError());
}

}  // namespace ss
