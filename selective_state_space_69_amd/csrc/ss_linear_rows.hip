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
//
// Gated products: the 16 rows of w are 8 of each half, so that a workgroup has both
// factors of 8 outputs.  8-bit integers: 64 of the contraction per MFMA; rows that are not
// whole 16-byte units are read from any address, their last unit byte by byte.  8 rows: 2560 ->
// 2 x 6912 bf16 17.4 us (4.1 TB/s of w), 2560 -> 10240 in bytes 8.2 us (3.2).
#include "ss_linear_mm.hpp"

namespace ss {
namespace {

constexpr int kWaves = 8;
constexpr int kUnroll = 5;      // loads of w in flight per wave

// 16 bytes of a row from element t of n; VEC: n and the row's alignment allow
// whole 16-byte units
template <typename T, bool VEC>
__device__ __forceinline__ u32x4 load_unit(const T* row, int t, int n) {
  constexpr int E = 16 / int(sizeof(T));
  if constexpr (VEC) {
    return t < n ? *reinterpret_cast<const u32x4*>(row + t) : u32x4{0, 0, 0, 0};
  } else if constexpr (sizeof(T) == 1) {
    struct __attribute__((packed, aligned(1))) Bytes { u32x4 v; };
    if (t + E <= n) return reinterpret_cast<const Bytes*>(row + t)->v;
    struct { T e[E]; } v;
#pragma unroll
    for (int j = 0; j < E; ++j) v.e[j] = t + j < n ? row[t + j] : T(0);
    return __builtin_bit_cast(u32x4, v);
  } else {
    struct Elems { T e[E]; } v;
#pragma unroll
    for (int j = 0; j < E; ++j) v.e[j] = t + j < n ? row[t + j] : T(0);
    return __builtin_bit_cast(u32x4, v);
  }
}

// MB: fragments of x, 16 rows each
template <typename T, int MB, bool VEC, int KIND>
__global__ __launch_bounds__(kWaves * kWave) void rows_kernel(MmParams p) {
  using Acc = std::conditional_t<KIND == kInt8, i32x4, f32x4>;
  using Sum = std::conditional_t<KIND == kInt8, int32_t, float>;
  __shared__ Sum part[kWaves][MB][16][17];
  constexpr int E = 16 / int(sizeof(T));
  constexpr int kSpan = 4 * E;              // t per wave and step
  constexpr int kCols = KIND == kGlu ? 8 : 16;
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int m = lane & 15, g = lane >> 4;
  const int s0 = int(blockIdx.x) * kCols;
  const int K = int(p.nT);
  int64_t col = s0 + m % kCols < p.nS ? s0 + m % kCols : p.nS - 1;
  if (KIND == kGlu && m >= kCols) col += p.nS;
  const T* w = static_cast<const T*>(p.S) + col * p.lds;
  const T* x[MB];
  Acc acc[MB];
#pragma unroll
  for (int b = 0; b < MB; ++b) {
    const int64_t r = b * 16 + m;
    x[b] = static_cast<const T*>(p.R) + (r < p.nR ? r : p.nR - 1) * p.ldr;
    acc[b] = Acc{0, 0, 0, 0};
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
      for (int b = 0; b < MB; ++b) acc[b] = mfma<T>(a[u], v[u][b], acc[b]);
  }
  // lane: rows s0 + 4 g .. + 3 of w, row m of x
#pragma unroll
  for (int b = 0; b < MB; ++b)
#pragma unroll
    for (int j = 0; j < 4; ++j) part[wv][b][m][4 * g + j] = acc[b][j];
  __syncthreads();
  for (int i = threadIdx.x; i < MB * 16 * kCols; i += kWaves * kWave) {
    const int b = i / (16 * kCols), row = i / kCols % 16, s = i % kCols;
    const int64_t r = b * 16 + row;
    if (r >= p.nR || s0 + s >= p.nS) continue;
    Sum f = 0, up = 0;
#pragma unroll
    for (int k = 0; k < kWaves; ++k) {
      f += part[k][b][row][s];
      if (KIND == kGlu) up += part[k][b][row][8 + s];
    }
    if constexpr (KIND == kGlu) glu1(p, p.act, r, s0 + s, f, up);
    else if constexpr (KIND == kInt8)
      epilogue1(p, p.act, r, s0 + s, scaled(f, RowScale(p.row_scale[r]), p.col_scale[s0 + s]));
    else epilogue1(p, p.act, r, s0 + s, f);
  }
}

template <typename T, int KIND>
void run(const MmParams& p, bool vec, hipStream_t st) {
  constexpr int kCols = KIND == kGlu ? 8 : 16;
  const unsigned blocks = unsigned((p.nS + kCols - 1) / kCols), threads = kWaves * kWave;
  if (p.nR <= 16) {
    if (vec) rows_kernel<T, 1, true, KIND><<<blocks, threads, 0, st>>>(p);
    else rows_kernel<T, 1, false, KIND><<<blocks, threads, 0, st>>>(p);
  } else {
    if (vec) rows_kernel<T, 2, true, KIND><<<blocks, threads, 0, st>>>(p);
    else rows_kernel<T, 2, false, KIND><<<blocks, threads, 0, st>>>(p);
  }
}

}  // namespace

void launch_rows(const MmParams& p, bool bf16, bool vec, hipStream_t st) {
  if (bf16) run<uint16_t, kMm>(p, vec, st);
  else run<float, kMm>(p, vec, st);
}
void launch_rows_glu(const MmParams& p, bool bf16, bool vec, hipStream_t st) {
  if (bf16) run<uint16_t, kGlu>(p, vec, st);
  else run<float, kGlu>(p, vec, st);
}
void launch_rows_q8(const MmParams& p, bool vec, hipStream_t st) { run<uint8_t, kInt8>(p, vec, st); }

}  // namespace ss
