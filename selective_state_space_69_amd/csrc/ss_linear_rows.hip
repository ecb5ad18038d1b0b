// Linear projection of a few rows (decoding: M <= 32 tokens) for gfx950.
//
// y = act(x w^T + b) + residual reads w once and does little with it, so the
// kernel streams w: a workgroup takes 16 rows of w (output columns), its 8 waves
// interleave over the contraction, 32 bf16 (16 fp32) of each row at a time, and
// every lane's 16-byte loads go straight from memory to the registers that the
// MFMA reads (no LDS on the way in).  w is the A side (16 rows), x the B side (16
// rows per fragment, rows past M repeat the last one and are not stored), so one
// pass serves up to 32 tokens.  The waves' partial tiles are added in wave order
// through LDS and the epilogue runs on the sums: one launch, no workspace.
//
// Bound by memory and a launch's ramp: 8 rows, 2560 -> 10240 bf16 take 13.6 us (3.9
// TB/s of w; 15.4 us with w always out of cache).  4 or 16 waves, twice the loads in
// flight, whole lines per wave or streamed loads were no faster (15.4 to 17.6).
#include "ss_linear_mm.hpp"

namespace ss {
namespace {

constexpr int kWaves = 8;
constexpr int kUnroll = 5;      // loads of w in flight per wave

template <typename T>
__device__ __forceinline__ f32x4 mma16(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (sizeof(T) == 2) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a[i]), __uint_as_float(b[i]), c, 0,
                                               0, 0);
    return c;
  }
}

// 16 bytes of a row from element t of n; VEC: n and the row's alignment allow
// whole 16-byte units
template <typename T, bool VEC>
__device__ __forceinline__ u32x4 load_unit(const T* row, int t, int n) {
  constexpr int E = 16 / int(sizeof(T));
  if constexpr (VEC) {
    return t < n ? *reinterpret_cast<const u32x4*>(row + t) : u32x4{0, 0, 0, 0};
  } else {
    struct Elems { T e[E]; } v;
#pragma unroll
    for (int j = 0; j < E; ++j) v.e[j] = t + j < n ? row[t + j] : T(0);
    return __builtin_bit_cast(u32x4, v);
  }
}

// MB: fragments of x, 16 rows each
template <typename T, int MB, bool VEC>
__global__ __launch_bounds__(kWaves * kWave) void rows_kernel(MmParams p) {
  __shared__ float part[kWaves][MB][16][17];
  constexpr int E = 16 / int(sizeof(T));
  constexpr int kSpan = 4 * E;              // t per wave and step
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int m = lane & 15, g = lane >> 4;
  const int s0 = int(blockIdx.x) * 16;
  const int K = int(p.nT);
  const T* w = static_cast<const T*>(p.S) + int64_t(s0 + m < p.nS ? s0 + m : p.nS - 1) * p.lds;
  const T* x[MB];
  f32x4 acc[MB];
#pragma unroll
  for (int b = 0; b < MB; ++b) {
    const int64_t r = b * 16 + m;
    x[b] = static_cast<const T*>(p.R) + (r < p.nR ? r : p.nR - 1) * p.ldr;
    acc[b] = f32x4{0, 0, 0, 0};
  }
  for (int t0 = wv * kSpan + g * E; t0 - g * E < K; t0 += kUnroll * kWaves * kSpan) {
    u32x4 a[kUnroll], v[kUnroll][MB];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) a[u] = load_unit<T, VEC>(w, t0 + u * kWaves * kSpan, K);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
#pragma unroll
      for (int b = 0; b < MB; ++b) v[u][b] = load_unit<T, VEC>(x[b], t0 + u * kWaves * kSpan, K);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
#pragma unroll
      for (int b = 0; b < MB; ++b) acc[b] = mma16<T>(a[u], v[u][b], acc[b]);
  }
  // lane: columns s0 + 4 g .. + 3 of row m
#pragma unroll
  for (int b = 0; b < MB; ++b)
#pragma unroll
    for (int j = 0; j < 4; ++j) part[wv][b][m][4 * g + j] = acc[b][j];
  __syncthreads();
  for (int i = threadIdx.x; i < MB * 256; i += kWaves * kWave) {
    const int b = i >> 8, row = (i >> 4) & 15, s = i & 15;
    const int64_t r = b * 16 + row;
    if (r >= p.nR || s0 + s >= p.nS) continue;
    float f = 0.0f;
#pragma unroll
    for (int k = 0; k < kWaves; ++k) f += part[k][b][row][s];
    epilogue1(p, p.act, r, s0 + s, f);
  }
}

template <typename T>
void run(const MmParams& p, bool vec, hipStream_t st) {
  const unsigned blocks = unsigned((p.nS + 15) / 16), threads = kWaves * kWave;
  if (p.nR <= 16) {
    if (vec) rows_kernel<T, 1, true><<<blocks, threads, 0, st>>>(p);
    else rows_kernel<T, 1, false><<<blocks, threads, 0, st>>>(p);
  } else {
    if (vec) rows_kernel<T, 2, true><<<blocks, threads, 0, st>>>(p);
    else rows_kernel<T, 2, false><<<blocks, threads, 0, st>>>(p);
  }
}

}  // namespace

void launch_rows(const MmParams& p, bool bf16, bool vec, hipStream_t st) {
  if (bf16) run<uint16_t>(p, vec, st);
  else run<float>(p, vec, st);
}

}  // namespace ss
