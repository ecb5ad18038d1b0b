// Rows as 8-bit integers with one scale each, for gfx950.
//
// A row is read once: its elements stay in registers between the largest magnitude
// (taken on the bits, where NaN and infinity are above every number) and the quotients.
// The bits are those of the definition.  127 x / max is rounded twice, with a factor 2^-22
// too small and one as much too large (the factor's own rounding is 2^-24).  Where both give
// the same, that is the nearest whole number; where not, a tie is near.  Of bf16 values only
// a true tie is: X, M of 8 bits, a quotient 127 X / M that is no tie is further than 2^-16 of
// itself from one, so the even one of both is right.  Of fp32 ones the sign of 254 |x| -
// (2 n + 1) max decides, taken exactly.  Memory bound.
#include "ss_device.hpp"

namespace ss {
namespace {

constexpr int kThreads = 256;
constexpr int64_t kWalking = 1024;                  // blocks that walk over the rows: four to a CU

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
    if constexpr (sizeof(T) == 2) {      // two values at a time
      typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
      u16x2 t{0, 0};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        t = __builtin_elementwise_max(t, u16x2{uint16_t(e[2 * j] & 0x7fff),
                                               uint16_t(e[2 * j + 1] & 0x7fff)});
      return uint32_t(t[0] > t[1] ? t[0] : t[1]) << 16;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t b = __float_as_uint(to_f32(e[j])) & 0x7fffffffu;
      m = b > m ? b : m;
    }
    return m;
  }
};

constexpr float kWhole = 12582912.0f;     // 1.5 2^23: sums with it are rounded to whole numbers
// The whole number nearest to 127 x / most in the low byte, for rows whose products and
// reciprocal stay inside fp32; scale: 127 / most.
__device__ __forceinline__ uint32_t nearest(float x, float scale, float most) {
  const float a = __builtin_fabsf(x), n = __builtin_floorf(a * scale), o = __builtin_fmaf(2.0f, n, 1.0f);
  const float q = o * most;
  // exact where the products are near each other
  const float d = __builtin_fmaf(254.0f, a, -q) - __builtin_fmaf(o, most, -q);
  // n + 1/2, moved by a quarter to the side that d shows; a tie goes to even with the sum
  const float side = __builtin_amdgcn_fmed3f(d * (scale * 0x1p40f), -0.25f, 0.25f);
  return __float_as_uint(__builtin_copysignf(n + 0.5f + side, x) + kWhole);
}
// the same for any row, in 64 bits
__device__ __forceinline__ uint32_t nearest64(float x, float most) {
  const double a = 254.0 * __builtin_fabs(double(x)), m = double(most);
  int n = int(a / (2.0 * m));                    // within one of the quotient's whole part
  if (a < 2.0 * n * m) --n;
  if (a >= 2.0 * (n + 1) * m) ++n;
  const double b = (2 * n + 1) * m;
  n += a > b || (a == b && (n & 1));
  return uint32_t(x < 0.0f ? -n : n);
}

// scale: 127 / most, 0 where fp32 cannot hold what nearest() forms
template <typename T>
__device__ __forceinline__ void store_eight(int8_t* row, int c, int span, const Eight<T>& v,
                                            float scale, float most, bool zero) {
  uint32_t b[8], differ = 0;
  const float under = scale * (1.0f - 0x1p-22f), over = scale * (1.0f + 0x1p-22f);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float x = to_f32(v.e[j]);
    const uint32_t u = __float_as_uint(__builtin_fmaf(x, under, kWhole));
    const uint32_t o = __float_as_uint(__builtin_fmaf(x, over, kWhole));
    b[j] = u & 1 ? o : u;
    if constexpr (sizeof(T) == 4) differ |= u ^ o;
  }
  if (sizeof(T) == 4 && differ && !zero) {
#pragma unroll
    for (int j = 0; j < 8; ++j) b[j] = nearest(to_f32(v.e[j]), scale, most);
  }
  if (scale == 0.0f && !zero) {
#pragma unroll
    for (int j = 0; j < 8; ++j) b[j] = nearest64(to_f32(v.e[j]), most);
  }
  uint32_t w[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const uint32_t lo = __builtin_amdgcn_perm(b[4 * j + 1], b[4 * j], 0x0c0c0400u);
    const uint32_t hi = __builtin_amdgcn_perm(b[4 * j + 3], b[4 * j + 2], 0x04000c0cu);
    w[j] = zero ? 0u : lo | hi;
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
  const int64_t first = int64_t(blockIdx.x) * kRows + threadIdx.x / kPer;
  const int64_t step = int64_t(gridDim.x) * kRows;
  // (rows past the last repeat it)
  auto row_of = [&](int64_t row) {
    return static_cast<const T*>(p.x) + (row < p.rows ? row : p.rows - 1) * p.ldx;
  };
  Eight<T> v[N ? N : 1], next[N ? N : 1];
  auto load = [&](Eight<T> (&d)[N ? N : 1], int64_t row) {
    const T* x = row_of(row);
#pragma unroll
    for (int i = 0; i < N; ++i) d[i].load(x, (i * kPer + tid) * 8, p.dim);
  };
  load(v, first);
  const int64_t turns = (p.rows - int64_t(blockIdx.x) * kRows + step - 1) / step;
  int64_t row = first;
  for (int64_t turn = 0; turn < turns; ++turn, row += step) {
    if (turn + 1 < turns) load(next, row + step);        // arrives under this row's work
    uint32_t top = 0;
    if constexpr (N > 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const uint32_t m = v[i].top();
        top = m > top ? m : top;
      }
    } else {
      const T* x = row_of(row);
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
    const float scale = most > 0x1p-60f && most < 0x1p115f ? 127.0f / most : 0.0f;
    if (row < p.rows) {
      int8_t* q = p.q + row * p.ldq;
      if (tid == 0) p.s[row] = finite ? most / 127.0f : __uint_as_float(0x7fc00000u);
      if constexpr (N > 0) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const int c = (i * kPer + tid) * 8;
          if (c < p.span) store_eight(q, c, p.span, v[i], scale, most, zero);
        }
      } else {
        const T* x = row_of(row);
        for (int c = tid * 8; c < p.span; c += kPer * 8) {
          v[0].load(x, c, p.dim);
          store_eight(q, c, p.span, v[0], scale, most, zero);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = next[i];
  }
}

template <typename T, int N>
void run_narrow(const PackParams& p, hipStream_t st) {
  const int64_t n = (p.rows + 3) / 4;
  pack_kernel<T, N, 1><<<unsigned(n < kWalking ? n : kWalking), kThreads, 0, st>>>(p);
}
template <typename T, int N>
void run_wide(const PackParams& p, hipStream_t st) {
  pack_kernel<T, N, 4><<<unsigned(p.rows < kWalking ? p.rows : kWalking), kThreads, 0, st>>>(p);
}
template <typename T>
void run(const PackParams& p, hipStream_t st) {
  // A wave to a row where the rows then still fill the GPU, else four, and each walks over
  // rows with the next one's loads out before this one's quotients.  bf16, us, one wave / four:
  // 16384 x 2560 24.4 / 32.5 (5.2 TB/s), 3001 x 1537 6.1 / 13.7, 16384 x 768 11 / 41,
  // 1100 x 2560 4.9 / 4.5, 500 x 2560 3.6 / 3.6.
  if (p.span <= 4096 && p.rows >= 2048) {
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
