// Rows as 8-bit integers with one scale each, for gfx950.
//
// A row is read once: its elements stay in registers between the largest magnitude
// (taken on the bits, where NaN and infinity are above every number) and the quotients.
// 127 x / max is formed in 64 bits, with an error below 2^-51 of it; where that leaves
// the nearest whole number open (a tie, or nearly), 254 |x| is compared with (2 k + 1)
// max, both exact in 64 bits.  So the bits are those of the definition, whatever
// computes them.  Memory bound.
#include "ss_device.hpp"

namespace ss {
namespace {

constexpr int kThreads = 256;

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

__device__ __forceinline__ int nearest(float x, double scale, double most) {
  const double t = double(x) * scale, r = __builtin_rint(t);
  int k = int(r);
  if (__builtin_fabs(__builtin_fabs(t - r) - 0.5) < 1e-9) {
    const double m = __builtin_fabs(t);
    int f = int(m);                                 // between f and f + 1
    const double a = 254.0 * __builtin_fabs(double(x)), b = double(2 * f + 1) * most;
    f += a > b || (a == b && (f & 1));
    k = x < 0.0f ? -f : f;
  }
  return k;
}

template <typename T>
__device__ __forceinline__ void store_eight(int8_t* row, int c, int span, const Eight<T>& v,
                                            double scale, double most, bool zero) {
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
    const double scale = zero ? 0.0 : 127.0 / double(most);
    if (!here) continue;
    int8_t* q = p.q + row * p.ldq;
    if (tid == 0) p.s[row] = finite ? most / 127.0f : __uint_as_float(0x7fc00000u);
    if constexpr (N > 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int c = (i * kPer + tid) * 8;
        if (c < p.span) store_eight(q, c, p.span, v[i], scale, double(most), zero);
      }
    } else {
      for (int c = tid * 8; c < p.span; c += kPer * 8) {
        v[0].load(x, c, p.dim);
        store_eight(q, c, p.span, v[0], scale, double(most), zero);
      }
    }
  }
}

template <typename T>
void run(const PackParams& p, hipStream_t st) {
  // a wave to a row of up to 2048 bytes of q, if the rows then still fill the GPU
  const bool narrow = p.span <= 2048 && p.rows >= 4096;
  const int64_t per = narrow ? 4 : 1, blocks64 = (p.rows + per - 1) / per;
  const unsigned blocks = unsigned(blocks64 < (int64_t(1) << 22) ? blocks64 : int64_t(1) << 22);
  if (narrow) {
    if (p.span <= 512) pack_kernel<T, 1, 1><<<blocks, kThreads, 0, st>>>(p);
    else if (p.span <= 1024) pack_kernel<T, 2, 1><<<blocks, kThreads, 0, st>>>(p);
    else pack_kernel<T, 4, 1><<<blocks, kThreads, 0, st>>>(p);
  } else if (p.span <= 2048) {
    pack_kernel<T, 1, 4><<<blocks, kThreads, 0, st>>>(p);
  } else if (p.span <= 4096) {
    pack_kernel<T, 2, 4><<<blocks, kThreads, 0, st>>>(p);
  } else if (p.span <= 8192) {
    pack_kernel<T, 4, 4><<<blocks, kThreads, 0, st>>>(p);
  } else {
    pack_kernel<T, 0, 4><<<blocks, kThreads, 0, st>>>(p);
  }
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
