// Linear projections for gfx950: the plan, what prepares the products' operands
// (aligned copies of rows that 16-byte loads cannot read in place, the backward's
// pre-activation gradient), the join of split contractions, and the launchers.
#include "ss_linear_mm.hpp"

namespace ss {
namespace {

constexpr int kThreads = 256;
constexpr int64_t kMaxBlocks = int64_t(1) << 22;    // a grid's threads stay below 2^32

// Sum of the splits' partials, in order, and the epilogue.
__global__ __launch_bounds__(kThreads) void join_kernel(MmParams p) {
  const int64_t units = (p.nS + 7) / 8;
  const int64_t total = p.nR * units;
  for (int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x; i < total;
       i += int64_t(gridDim.x) * kThreads) {
    const int64_t r = i / units;
    const int32_t s = int32_t(i - r * units) * 8;
    const float* src = p.part + r * p.nS + s;
    const int64_t step = p.nR * p.nS;
    if (s + 8 <= p.nS) {
      float v[8] = {0, 0, 0, 0, 0, 0, 0, 0}, bias[8] = {0, 0, 0, 0, 0, 0, 0, 0};
      const Res8 res = fetch_res8(p, r * p.nS + s, true);
      if (p.bias) load8(p.bias + s, bias);
      for (int k = 0; k < p.splits; ++k) {
        float f[8];
        load8(src + k * step, f);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += f[j];
      }
      epilogue8<kActOf>(p, r * p.nS + s, v, bias, res);
    } else {
      for (int j = 0; s + j < p.nS; ++j) {
        float v = 0.0f;
        for (int k = 0; k < p.splits; ++k) v += src[k * step + j];
        epilogue1(p, p.act, r, s + j, v);
      }
    }
  }
}

// Sum of the splits' partials of both gated products, in order, and their epilogue.
__global__ __launch_bounds__(kThreads) void join_glu_kernel(MmParams p) {
  const int64_t total = p.nR * p.nS, step = 2 * total;
  for (int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x; i < total;
       i += int64_t(gridDim.x) * kThreads) {
    const int64_t r = i / p.nS;
    const int32_t c = int32_t(i - r * p.nS);
    const float* src = p.part + 2 * r * p.nS + c;
    float gate = 0.0f, up = 0.0f;
    for (int k = 0; k < p.splits; ++k) {
      gate += src[k * step];
      up += src[k * step + p.nS];
    }
    glu1(p, p.act, r, c, gate, up);
  }
}
// Sum of the splits' whole numbers, their scales and the epilogue.
__global__ __launch_bounds__(kThreads) void join_q8_kernel(MmParams p) {
  const int64_t total = p.nR * p.nS;
  const int32_t* part = reinterpret_cast<const int32_t*>(p.part);
  for (int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x; i < total;
       i += int64_t(gridDim.x) * kThreads) {
    const int64_t r = i / p.nS;
    const int32_t c = int32_t(i - r * p.nS);
    int32_t sum = 0;
    for (int k = 0; k < p.splits; ++k) sum += part[k * total + i];
    epilogue1(p, p.act, r, c, scaled(sum, RowScale(p.row_scale[r]), p.col_scale[c]));
  }
}

// Rows of one or two tensors (blockIdx.y) at a 16-byte aligned stride, zero past
// their end: one 16-byte unit of the copy per thread.  T: bf16 or bytes.
struct PadJob {
  const void* src;
  void* dst;
  int64_t ld_src, rows;
  int32_t cols, units;     // units of a row of the copy
};
struct PadParams {
  PadJob job[2];
};
template <typename T>
__global__ __launch_bounds__(kThreads) void pad_kernel(PadParams q) {
  constexpr int E = 16 / int(sizeof(T));
  const PadJob p = q.job[blockIdx.y];
  const int64_t total = p.rows * p.units;
  for (int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x; i < total;
       i += int64_t(gridDim.x) * kThreads) {
    const int64_t r = total <= INT32_MAX ? int64_t(uint32_t(i) / uint32_t(p.units)) : i / p.units;
    const int c = int(i - r * p.units) * E;
    const T* src = static_cast<const T*>(p.src) + r * p.ld_src + c;
    struct __attribute__((packed, aligned(sizeof(T)))) Elems { T e[E]; } v;
    if (c + E <= p.cols) {
      v = *reinterpret_cast<const Elems*>(src);      // 16 bytes at any element address
    } else {
#pragma unroll
      for (int j = 0; j < E; ++j) v.e[j] = c + j < p.cols ? src[j] : T(0);
    }
    reinterpret_cast<u32x4*>(p.dst)[i] = __builtin_bit_cast(u32x4, v);
  }
}

// dpre = dy act'(pre) in the operand type (when asked for), in rows of ld elements
// that are zero past N, and its column sums before that rounding.  A block takes
// 64 V columns (V neighbours per lane; 8 where N is a whole number of 16-byte units, of
// which bf16 ones are loaded as two halves) and a chunk of rows, a wave every fourth row
// of it, four at a time; the waves' sums are added in order into one partial row per
// block.  A lane adds runs of 64 rows, then the runs, so that a column sum's rounding does
// not grow with the rows that the column blocks leave to a chunk (2^20 rows of one value,
// 2049 columns, 8192 rows to a lane: 6.5e-5 off in one chain, 1.0e-6 so; no slower).
// What bf16 operands see of a dpre that is not bf16 goes by the gradients' type.  bf16
// gradients: bf16(dpre), a second half step beside their own (errors of 2.3e-3 instead
// of 1.7e-3 of a gradient, 2-norms).  fp32 gradients: sum2, each value as hi = bf16(v)
// and lo = bf16(v - hi), 8 hi, then their 8 lo, exact to 2^-16 (2.5e-6; 1.7e-3 with hi
// alone) for twice the products' MFMAs (bf16 4096 x 768 x 1536 with fp32 dy: 41 -> 60
// us, 16384 x 2560 x 5120 768 -> 1434).
struct DpreParams {
  const void* dy;
  const void* pre;
  void* d;            // or null
  float* part;        // (gridDim.y, N) or null
  int64_t M, rows;    // rows per block
  int32_t N, ld, act, sum2;
};
// what bf16(v) leaves of v (0, not infinity less infinity, of what it makes infinite)
__device__ __forceinline__ float rest_of(float v) {
  const uint32_t hi = cvt_bf16x2(0.0f, v) & 0xffff0000u;
  return (hi & 0x7f800000u) == 0x7f800000u ? 0.0f : v - __uint_as_float(hi);
}
template <typename T, int V>
__device__ __forceinline__ void load_cols(const T* p, int c, int n, float (&v)[V]) {
  if constexpr (V == 8) {
    // c and n are multiples of 8
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float4 f = c < n ? unpack4(load_raw4(p + c + 4 * h)) : make_float4(0, 0, 0, 0);
      v[4 * h] = f.x; v[4 * h + 1] = f.y; v[4 * h + 2] = f.z; v[4 * h + 3] = f.w;
    }
  } else {
    v[0] = c < n ? to_f32(p[c]) : 0.0f;
  }
}
template <typename Dy, typename T, int V, int ACT>
__global__ __launch_bounds__(kThreads) void dpre_kernel(DpreParams p) {
  __shared__ float part[4][64 * V];
  constexpr int kRows = 4;
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int c = (int(blockIdx.x) * 64 + lane) * V;
  const int64_t m0 = int64_t(blockIdx.y) * p.rows;
  const int64_t m1 = m0 + p.rows < p.M ? m0 + p.rows : p.M;
  constexpr int kRun = 64 / kRows;      // turns of a run
  float sum[V], run[V];
#pragma unroll
  for (int j = 0; j < V; ++j) sum[j] = run[j] = 0.0f;
  int turn = 0;
  for (int64_t m = m0 + wv; m < m1; m += 4 * kRows) {
    if (++turn > kRun) {
      turn = 1;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        sum[j] += run[j];
        run[j] = 0.0f;
      }
    }
    float v[kRows][V], q[kRows][V];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int64_t r = m + 4 * i < m1 ? m + 4 * i : m1 - 1;
      load_cols<Dy, V>(static_cast<const Dy*>(p.dy) + r * p.N, c, p.N, v[i]);
      if constexpr (ACT != SS_ACT_NONE)
        load_cols<T, V>(static_cast<const T*>(p.pre) + r * p.N, c, p.N, q[i]);
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int64_t r = m + 4 * i;
      if (r >= m1) break;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        if constexpr (ACT != SS_ACT_NONE) v[i][j] *= act_grad(ACT, q[i][j]);
        run[j] += v[i][j];
      }
      if (!p.d) continue;
      if (sizeof(T) == 2 && p.sum2) {
        if (2 * c >= p.ld) continue;
        uint16_t* d = static_cast<uint16_t*>(p.d) + r * p.ld + (c >> 3) * 16 + (c & 7);
        float lo[V];
#pragma unroll
        for (int j = 0; j < V; ++j) lo[j] = rest_of(v[i][j]);
        if constexpr (V == 8) {
          store8(d, 0, true, v[i]);
          store8(d, 8, true, lo);
        } else {
          store_out<uint16_t>(d, v[i][0]);
          store_out<uint16_t>(d + 8, lo[0]);
        }
      } else if (c < p.ld) {
        T* d = static_cast<T*>(p.d) + r * p.ld + c;
        if constexpr (V == 8) store8(d, 0, sizeof(T) == 2, v[i]);
        else store_out<T>(d, c < p.N ? v[i][0] : 0.0f);
      }
    }
  }
  if (!p.part) return;
#pragma unroll
  for (int j = 0; j < V; ++j) part[wv][lane * V + j] = sum[j] + run[j];
  __syncthreads();
  for (int i = threadIdx.x; i < 64 * V; i += kThreads) {
    const int col = int(blockIdx.x) * 64 * V + i;
    if (col < p.N)
      p.part[int64_t(blockIdx.y) * p.N + col] =
          (part[0][i] + part[1][i]) + (part[2][i] + part[3][i]);
  }
}

// Both halves of a gated dpre, d = [dy up act'(gate), dy act(gate)], in rows of ld
// elements that are zero past 2 F, and their column sums: as dpre_kernel, a lane taking V
// columns of each half.  V is 8 where F is a whole number of 16-byte units.  The products of
// bf16 operands see of d what they see of a dpre: with bf16 gradients bf16(d), half a step
// beside their own (16384 x 2560 -> 6912: 2.4e-3 off for 1.7e-3, 2000 us), with fp32 ones d to
// 2^-16 (2e-6; 3960 us).
struct DgluParams {
  const void* dy;     // (M, F)
  const void* pre;    // (M, 2 F)
  void* d;            // or null
  float* part;        // (gridDim.y, 2 F) or null
  int64_t M, rows;    // rows per block
  int32_t F, ld, sum2;
};
template <typename T, int V>
__device__ __forceinline__ void put_cols(const DgluParams& p, int64_t r, int32_t c,
                                         const float (&v)[V]) {
  if (sizeof(T) == 2 && p.sum2) {
    uint16_t* d = static_cast<uint16_t*>(p.d) + r * p.ld + (c >> 3) * 16 + (c & 7);
    float lo[V];
#pragma unroll
    for (int j = 0; j < V; ++j) lo[j] = rest_of(v[j]);
    if constexpr (V == 8) {
      store8(d, 0, true, v);
      store8(d, 8, true, lo);
    } else {
      store_out<uint16_t>(d, v[0]);
      store_out<uint16_t>(d + 8, lo[0]);
    }
  } else {
    T* d = static_cast<T*>(p.d) + r * p.ld + c;
    if constexpr (V == 8) store8(d, 0, sizeof(T) == 2, v);
    else store_out<T>(d, v[0]);
  }
}
// SUMS: with the column sums, for which a block walks its rows, two at a time; without
// them it takes four rows, one a wave (bf16 16384 x 6912: 349 us walking, 198 so, 5.7 TB/s).
constexpr int64_t kDgluRows = 4;
template <typename Dy, typename T, int V, int ACT, bool SUMS>
__global__ __launch_bounds__(kThreads) void dglu_kernel(DgluParams p) {
  __shared__ float part[SUMS ? 4 : 1][2][64 * V];
  constexpr int kRows = SUMS ? 2 : 1;
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int c = (int(blockIdx.x) * 64 + lane) * V;
  const int64_t m0 = int64_t(blockIdx.y) * p.rows;
  const int64_t m1 = m0 + p.rows < p.M ? m0 + p.rows : p.M;
  constexpr int kRun = 64 / kRows;      // turns of a run
  float sum[2][V], run[2][V];
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int j = 0; j < V; ++j) sum[k][j] = run[k][j] = 0.0f;
  int turn = 0;
  for (int64_t m = m0 + wv; m < m1; m += 4 * kRows) {
    if (SUMS && ++turn > kRun) {
      turn = 1;
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int j = 0; j < V; ++j) {
          sum[k][j] += run[k][j];
          run[k][j] = 0.0f;
        }
    }
    float v[kRows][V], gate[kRows][V], up[kRows][V];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int64_t r = m + 4 * i < m1 ? m + 4 * i : m1 - 1;
      const T* pre = static_cast<const T*>(p.pre) + 2 * r * p.F;
      load_cols<Dy, V>(static_cast<const Dy*>(p.dy) + r * p.F, c, p.F, v[i]);
      load_cols<T, V>(pre, c, p.F, gate[i]);
      load_cols<T, V>(pre + p.F, c, p.F, up[i]);
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int64_t r = m + 4 * i;
      if (r >= m1) break;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float g = gate[i][j], dy = v[i][j];
        gate[i][j] = dy * up[i][j] * act_grad(ACT, g);
        up[i][j] = dy * apply_act(ACT, g);
        if constexpr (SUMS) {
          run[0][j] += gate[i][j];
          run[1][j] += up[i][j];
        }
      }
      if (!p.d) continue;
      if (c < p.F) {
        put_cols<T, V>(p, r, c, gate[i]);
        put_cols<T, V>(p, r, p.F + c, up[i]);
      } else if (V == 1 && 2 * p.F + (c - p.F) < p.ld / (p.sum2 ? 2 : 1)) {
        const float zero[V] = {};
        put_cols<T, V>(p, r, p.F + c, zero);
      }
    }
  }
  if constexpr (!SUMS) return;
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int j = 0; j < V; ++j) part[wv][k][lane * V + j] = sum[k][j] + run[k][j];
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * 64 * V; i += kThreads) {
    const int k = i / (64 * V), n = i % (64 * V), col = int(blockIdx.x) * 64 * V + n;
    if (col < p.F)
      p.part[(int64_t(blockIdx.y) * 2 + k) * p.F + col] =
          (part[0][k][n] + part[1][k][n]) + (part[2][k][n] + part[3][k][n]);
  }
}

size_t align256(size_t x) { return (x + 255) / 256 * 256; }
bool ptr16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }
int unit_of(const ss_linear_desc_t& d) { return d.in_dtype == SS_BF16 ? 8 : 4; }
int64_t pad_to_unit(const ss_linear_desc_t& d, int64_t n) {
  const int e = unit_of(d);
  return (n + e - 1) / e * e;
}

// How a product is tiled.  bf16: 128 x 128 tiles while all of them fit on the 256 CUs
// at once, two to a CU (or one, of two wave groups that share its stages), and where
// 256 x 256 ones would be mostly empty.  Beyond that, 256 x 256 tiles against 128 x
// 128 ones four to a CU with one buffer each, whichever ends first: a large tile
// takes 0.75 to 1.45 us per stage of 128 bytes (the more CUs are busy the lower is the
// clock) and 6.5 us around them with nothing beside it, a small one 0.46 and 0.9 us of
// its CU, whose other tiles cover its waits.  Measured, large and single-buffered
// tiles (bf16 out, us of a call among 150 in a row, both kinds in turn):
//   contraction            160            320            640           1280
//   16384 x 5120      64.3   51.0    79.1   73.0   113.3  116.2   185.9  205.7
//   with softplus     83.6   65.6    99.3   85.5   132.8  128.2   201.9  216.9
//   4096 x 5120       24.7   16.0    29.9   20.9    42.5   34.5    66.3   60.1
// (small and double-buffered against large, contraction 2560: 2048 x 4096, 512 small
// tiles, 45.9 and 53.6).
// fp32: 64 x 64, of which five fit.  Where the tiles of a long contraction leave CUs
// empty it is split.  The model below picks the groups and the number of parts: a
// stage of 128 bytes takes 0.7 us with one group of waves on a CU and 0.9 us for two
// (fp32: 0.5 us for each, not below 0.7), two groups meet for 1 us, and a split
// product pays for the join kernel and for its partial sums' way to memory and back.
// Measured, one group and two:
//   768 x 1536 over 5003 (72 tiles, 79 stages), three parts   31.3   28.7 us
//     (one group in one part 50.9, two 34.6, five 28.7, eight 36.6)
//   5003 x 768 over 1536 (240 tiles, 24 stages), one part     22.5   19.8
//     (one group in two parts 28.2)
//   2048 x 1536 over 768 (192 tiles, 12 stages), one part     13.9   11.3
//   512 x 5120 over 2560 (160 tiles, 40 stages), one part     33.3   27.5
struct Tiling {
  MmTile tile;
  int32_t tiles_r, tiles_s, splits;
  int64_t t_split;
  double us;       // the model's time
};
constexpr double kLaunchUs = 6.0;       // a product's launch, first copies and epilogue
double stage_us(bool bf16, int64_t items) {
  const int64_t per_cu = (items + 255) / 256;
  return bf16 ? (per_cu > 1 ? 0.9 : 0.7) : (per_cu > 1 ? 0.5 * double(per_cu) : 0.7);
}
// a large tile, of a launch that fills the GPU
double big_us(int64_t stages) { return 1.45 * double(stages) + 6.5; }
// the join of k parts, their sums written and read
double join_us(int64_t nR, int64_t nS, int64_t k) {
  return k > 1 ? 6.0 + double(k) * double(nR) * double(nS) * 8.0 / 4.0e6 : 0.0;
}
// What one product offers to choose from: its small tiles, its stages, how many
// items fit on the GPU at once.
struct Small {
  bool bf16;
  int64_t nR, nS, nT, step, tiles_r, tiles_s, tiles, stages, fit;
  // size: bytes of an element of the contraction, for bf16 as the sum of two 4
  Small(bool fp32, int size, int64_t r, int64_t s, int64_t t) : bf16(!fp32), nR(r), nS(s), nT(t) {
    const int64_t side = bf16 ? 128 : 64;
    step = 128 / size;
    fit = bf16 ? 512 : 1024;
    tiles_r = (nR + side - 1) / side;
    tiles_s = (nS + side - 1) / side;
    tiles = tiles_r * tiles_s;
    stages = (nT + step - 1) / step;
  }
  int64_t per_part(int64_t k) const { return (stages + k - 1) / k; }
  // k parts; those that hold no stage are dropped
  Tiling tiling(MmTile tile, int64_t k, double us) const {
    const int64_t len = per_part(k) * step;
    return Tiling{tile, int32_t(tiles_r), int32_t(tiles_s), int32_t((nT + len - 1) / len), len, us};
  }
};
Tiling tiling(const Small& p) {
  const int64_t nR = p.nR, nS = p.nS, nT = p.nT;
  const int64_t r256 = (nR + 255) / 256, s256 = (nS + 255) / 256;
  if (p.bf16 && p.tiles > 512 && p.tiles * 100 > 282 * r256 * s256) {
    const int64_t rounds = (r256 * s256 + 255) / 256, per_cu = (p.tiles + 255) / 256;
    const double fill = double(r256 * s256) / double(256 * rounds);
    const double big = kLaunchUs + double(rounds) * ((0.75 + 0.7 * fill) * double(p.stages) + 6.5);
    const double single = kLaunchUs + double(per_cu) * (0.46 * double(p.stages) + 0.9);
    if (single < big) return p.tiling(MmTile::kSmallSingle, 1, single);
    return Tiling{MmTile::kBig, int32_t(r256), int32_t(s256), 1, nT, big};
  }
  Tiling best{};
  for (int64_t k = 1; k <= 64 && (k == 1 || (k * p.tiles <= p.fit && k * 2 <= p.stages)); ++k) {
    const double rest = kLaunchUs + join_us(nR, nS, k);
    double us = double(p.per_part(k)) * stage_us(p.bf16, k * p.tiles) + rest;
    MmTile tile = p.bf16 ? MmTile::kSmall : MmTile::kSmallF32;
    if (p.bf16 && k * p.tiles <= 256) {
      const double two = double(p.per_part(2 * k)) * 0.9 + 1.0 + rest;
      if (two < us) {
        us = two;
        tile = MmTile::kSmallPair;
      }
    }
    if (k == 1 || us < best.us) best = p.tiling(tile, k, us);
  }
  return best;
}
// a forward's tiles (n: its columns, both halves of gated ones)
Tiling tiling_fwd(const ss_linear_desc_t& d, int64_t n) {
  const bool fp32 = d.in_dtype == SS_F32;
  return tiling(Small(fp32, fp32 ? 4 : 2, d.rows, n, d.in_dim));
}
// The tiles of a backward pass.  One launch computes dx and dw where the model finds
// that faster than one after the other: small tiles that all fit on the GPU at once
// (bf16 5003 x 768 x 1536, whole call: 48 us, both 37), or 256 x 256 ones, where the
// workgroups that dw's last round does not reach go on with dx's tiles, the others
// taking `few` of those each.
struct Backward {
  Tiling dx, dw;
  bool both;
  int behind, few;
};
Backward tilings_bwd(const ss_linear_desc_t& d, bool sum2) {
  const bool fp32 = d.in_dtype == SS_F32;
  const int size = fp32 || sum2 ? 4 : 2;
  const Small a(fp32, size, d.rows, d.in_dim, d.out_dim), b(fp32, size, d.out_dim, d.in_dim, d.rows);
  Backward t{tiling(a), tiling(b), false, 0, 0};
  auto longer = [](int64_t u, int64_t v) { return u > v ? u : v; };
  if (t.dx.tile == MmTile::kBig && t.dw.tile == MmTile::kBig) {
    const double ux = big_us(a.stages), uw = big_us(b.stages);
    const int64_t nx = int64_t(t.dx.tiles_r) * t.dx.tiles_s;
    const int64_t nw = int64_t(t.dw.tiles_r) * t.dw.tiles_s;
    const int64_t behind = nw % 256, rest = 256 - behind;
    double best = 2.0 * kLaunchUs + double((nx + 255) / 256) * ux + double((nw + 255) / 256) * uw;
    for (int64_t few = 0; few <= nx / 256 && (few == 0 || behind); ++few) {
      const int64_t most = few + (nx - few * 256 + rest - 1) / rest;
      const double late = uw + double(few) * ux, early = double(most) * ux;
      const double us = kLaunchUs + double(nw / 256) * uw +
                        (behind && late > early ? late : early);
      if (us < best) {
        best = us;
        t.both = true;
        t.behind = int(behind);
        t.few = int(few);
      }
    }
    return t;
  }
  double best = t.dx.us + t.dw.us;
  for (int64_t i = 1; i <= 16 && i * 2 <= a.stages + 1; ++i)
    for (int64_t j = 1; j <= 64 && j * 2 <= b.stages + 1; ++j) {
      const int64_t items = i * a.tiles + j * b.tiles;
      if (items > a.fit) break;
      const double rest = kLaunchUs + join_us(a.nR, a.nS, i) + join_us(b.nR, b.nS, j);
      const int64_t one = longer(a.per_part(i), b.per_part(j));
      const int64_t two = longer(a.per_part(2 * i), b.per_part(2 * j));
      const double us[2] = {double(one) * stage_us(a.bf16, items) + rest,
                            double(two) * 0.9 + 1.0 + rest};
      const int pair = a.bf16 && items <= 256 && us[1] < us[0];
      if (us[pair] < best) {
        best = us[pair];
        const MmTile tile = pair ? MmTile::kSmallPair
                                 : a.bf16 ? MmTile::kSmall : MmTile::kSmallF32;
        t.both = true;
        t.dx = a.tiling(tile, i, best);
        t.dw = b.tiling(tile, j, best);
      }
    }
  return t;
}

size_t part_bytes(const Tiling& t, int64_t nR, int64_t nS) {
  return t.splits > 1 ? align256(size_t(t.splits) * size_t(nR) * size_t(nS) * 4) : 0;
}

MmParams tiled(MmParams p, const Tiling& t, char* part) {
  p.tiles_r = t.tiles_r;
  p.tiles_s = t.tiles_s;
  p.splits = t.splits;
  p.t_split = t.t_split;
  p.part = reinterpret_cast<float*>(part);
  return p;
}
void join(const MmParams& p, hipStream_t stream) {
  if (p.splits == 1) return;
  const int64_t n = (p.nR * ((p.nS + 7) / 8) + kThreads - 1) / kThreads;
  join_kernel<<<unsigned(n < kMaxBlocks ? n : kMaxBlocks), kThreads, 0, stream>>>(p);
}
void run_mm(MmParams p, const Tiling& t, bool rt, bool st, bool sum2, char* part,
            hipStream_t stream) {
  p = tiled(p, t, part);
  launch_mm(p, t.tile, rt, st, sum2, stream);
  join(p, stream);
}

// The operands of a call that 16-byte units cannot read in place: bf16 ones are copied
// to rows of pad_to_unit(cols) elements by one launch, for fp32 ones the products are
// told to read single elements.
struct Operands {
  int esize;         // bytes of an element
  PadParams pad{};
  int n = 0;
  bool any = false;
  // rows x cols of src, rows *ld elements apart: where the products read it
  const void* take(const void* src, int64_t* ld, int64_t rows, int64_t cols, char* dst) {
    const int e = 16 / esize;
    if (ptr16(src) && *ld % e == 0 && cols % e == 0) return src;
    if (esize == 4) {
      any = true;
      return src;
    }
    const int64_t units = (cols + e - 1) / e;
    pad.job[n++] = PadJob{src, dst, *ld, rows, int32_t(cols), int32_t(units)};
    *ld = units * e;
    return dst;
  }
  MmTile tile(MmTile t) const { return any && t == MmTile::kSmallF32 ? MmTile::kSmallF32Any : t; }
  void launch(hipStream_t st) {
    if (n == 0) return;
    int64_t blocks = 1;
    for (int i = 0; i < n; ++i) {
      const int64_t b = (pad.job[i].rows * pad.job[i].units + kThreads - 1) / kThreads;
      if (b > blocks) blocks = b;
    }
    const dim3 grid(unsigned(blocks < kMaxBlocks ? blocks : kMaxBlocks), unsigned(n));
    if (esize == 1) pad_kernel<uint8_t><<<grid, kThreads, 0, st>>>(pad);
    else pad_kernel<uint16_t><<<grid, kThreads, 0, st>>>(pad);
  }
};

template <typename Dy, typename T, int V>
void dpre_act(const DpreParams& p, dim3 grid, hipStream_t st) {
  switch (p.act) {
    case SS_ACT_SILU: dpre_kernel<Dy, T, V, SS_ACT_SILU><<<grid, kThreads, 0, st>>>(p); break;
    case SS_ACT_GELU: dpre_kernel<Dy, T, V, SS_ACT_GELU><<<grid, kThreads, 0, st>>>(p); break;
    case SS_ACT_SOFTPLUS:
      dpre_kernel<Dy, T, V, SS_ACT_SOFTPLUS><<<grid, kThreads, 0, st>>>(p);
      break;
    default: dpre_kernel<Dy, T, V, SS_ACT_NONE><<<grid, kThreads, 0, st>>>(p);
  }
}
template <int V>
void dpre_types(const ss_linear_desc_t& d, const DpreParams& p, dim3 grid, hipStream_t st) {
  const bool yb = d.out_dtype == SS_BF16, tb = d.in_dtype == SS_BF16;
  if (yb && tb) dpre_act<uint16_t, uint16_t, V>(p, grid, st);
  else if (yb) dpre_act<uint16_t, float, V>(p, grid, st);
  else if (tb) dpre_act<float, uint16_t, V>(p, grid, st);
  else dpre_act<float, float, V>(p, grid, st);
}
// columns of a lane that makes dpre, of rows (or halves of rows) of n
int dpre_vec(int64_t n) { return n % 8 == 0 ? 8 : 1; }

}  // namespace

// gated: out_dim counts both halves, and the kernel that makes dpre takes a column of
// each at once
static LinearPlan plan_bwd_fwd(const ss_linear_desc_t& d, int op, bool gated) {
  LinearPlan pl;
  const size_t esize = d.in_dtype == SS_BF16 ? 2 : 4;
  const size_t x_bytes = align256(size_t(d.rows) * size_t(pad_to_unit(d, d.in_dim)) * esize);
  const size_t w_bytes = align256(size_t(d.out_dim) * size_t(pad_to_unit(d, d.in_dim)) * esize);
  // rows with a stride may start anywhere: reserve a copy
  const bool bf16 = d.in_dtype == SS_BF16;
  const bool pad_k = bf16 && d.in_dim % 8 != 0, pad_x = pad_k || (bf16 && d.x_stride != 0);
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += bytes;
    return at;
  };
  if (op == SS_LINEAR_FWD) {
    if (d.rows <= kRowsMax) return pl;
    if (pad_x) pl.off_x = take(x_bytes);
    if (pad_k) pl.off_w = take(w_bytes);
    pl.off_part =
        take(part_bytes(tiling_fwd(d, d.out_dim), d.rows, d.out_dim));
    pl.bytes = off;
    return pl;
  }
  pl.need_dpre = d.act != SS_ACT_NONE || d.out_dtype != d.in_dtype ||
                 (bf16 && d.out_dim % 8 != 0);
  pl.sum2 = bf16 && d.grad_dtype == SS_F32 &&
            (d.act != SS_ACT_NONE || d.out_dtype != SS_BF16);
  pl.ld_dpre = pad_to_unit(d, d.out_dim) * (pl.sum2 ? 2 : 1);
  // about 1024 blocks over the columns and row chunks, at least 16 rows each; gated ones of
  // single columns, whose lanes load an element at a time, 8192 in at most 1024 chunks
  // (dbias of bf16 16384 x 1004: 46 us, with 1024 blocks 73)
  const int64_t width = gated ? d.out_dim / 2 : d.out_dim, span = 64 * dpre_vec(width);
  const int64_t cols = (width + span - 1) / span;
  const int64_t blocks = gated && span == 64 ? 8192 : 1024;
  int64_t chunks = (blocks + cols - 1) / cols;
  int64_t most = (d.rows + 15) / 16;
  if (most > 1024) most = 1024;
  if (chunks > most) chunks = most;
  pl.chunk_rows = (d.rows + chunks - 1) / chunks;
  pl.chunks = (d.rows + pl.chunk_rows - 1) / pl.chunk_rows;
  if (pl.need_dpre)
    pl.off_dpre = take(align256(size_t(d.rows) * size_t(pl.ld_dpre) * esize));
  if (op == SS_LINEAR_BWD_CKPT || pad_x) pl.off_x = take(x_bytes);
  if (pad_k) pl.off_w = take(w_bytes);
  pl.off_sums = take(align256(size_t(pl.chunks) * size_t(d.out_dim) * 4));
  // dx's and dw's parts: one after the other in one place, or side by side
  const Backward t = tilings_bwd(d, pl.sum2);
  const size_t a = part_bytes(t.dx, d.rows, d.in_dim), b = part_bytes(t.dw, d.out_dim, d.in_dim);
  pl.off_part_dw = t.both ? a : 0;
  pl.off_part = take(t.both ? a + b : a > b ? a : b);
  pl.bytes = off;
  return pl;
}

LinearPlan plan_linear(const ss_linear_desc_t& d, int op) { return plan_bwd_fwd(d, op, false); }

int launch_linear_fwd(const ss_linear_desc_t& d, const void* x, const void* w, const float* bias,
                      const void* residual, void* y, void* pre, char* ws, void* stream) {
  hipStream_t st = static_cast<hipStream_t>(stream);
  MmParams p{};
  p.ldr = d.x_stride ? d.x_stride : d.in_dim;
  p.lds = d.in_dim;
  p.nR = d.rows;
  p.nS = int32_t(d.out_dim);
  p.nT = d.in_dim;
  p.bias = bias;
  p.res = residual;
  p.out = y;
  p.pre = pre;
  p.act = d.act;
  p.out_bf16 = d.out_dtype == SS_BF16;
  p.res_bf16 = d.res_dtype == SS_BF16;
  p.pre_bf16 = d.in_dtype == SS_BF16;
  if (d.rows <= kRowsMax) {
    const int e = unit_of(d);
    p.R = x;
    p.S = w;
    launch_rows(p, d.in_dtype == SS_BF16, ptr16(x) && p.ldr % e == 0 && p.nT % e == 0, st);
    return int(hipGetLastError());
  }
  const LinearPlan pl = plan_linear(d, SS_LINEAR_FWD);
  Operands ops{d.in_dtype == SS_BF16 ? 2 : 4};
  p.R = ops.take(x, &p.ldr, d.rows, d.in_dim, ws + pl.off_x);
  p.S = ops.take(w, &p.lds, d.out_dim, d.in_dim, ws + pl.off_w);
  ops.launch(st);
  Tiling t = tiling_fwd(d, d.out_dim);
  t.tile = ops.tile(t.tile);
  run_mm(p, t, true, true, false, ws + pl.off_part, st);
  return int(hipGetLastError());
}

// dx and dw of a dpre (rows of pl.ld_dpre, or d.out_dim, elements); odd: fp32 rows of it
// that 16-byte units cannot read.
static int backward_products(const ss_linear_desc_t& d, const LinearPlan& pl, const void* dpre,
                             bool odd, const void* x, const int8_t* q, const uint8_t* e,
                             const void* w, void* dx, void* dw, char* ws, void* stream) {
  MmParams p{};
  hipStream_t st = static_cast<hipStream_t>(stream);
  p.R = dpre;
  p.ldr = pl.need_dpre ? pl.ld_dpre : d.out_dim;
  p.nS = int32_t(d.in_dim);
  p.act = SS_ACT_NONE;
  p.out_bf16 = d.grad_dtype == SS_BF16;
  Operands ops{d.in_dtype == SS_BF16 ? 2 : 4};
  MmParams px = p, pw = p;
  px.lds = d.in_dim;
  pw.lds = d.x_stride ? d.x_stride : d.in_dim;
  if (dx) {
    px.S = ops.take(w, &px.lds, d.out_dim, d.in_dim, ws + pl.off_w);
    px.nR = d.rows;
    px.nT = d.out_dim;
    px.out = dx;
  }
  if (dw) {
    if (q) {
      ss_ckpt_desc_t c{};
      c.rows = d.rows;
      c.dim = d.in_dim;
      c.x_stride = pw.lds = pad_to_unit(d, d.in_dim);
      c.dtype = d.in_dtype;
      pw.S = ws + pl.off_x;
      const int rc = launch_ckpt_unpack(c, q, e, ws + pl.off_x, stream);
      if (rc) return rc;
    } else {
      pw.S = ops.take(x, &pw.lds, d.rows, d.in_dim, ws + pl.off_x);
    }
    pw.nR = d.out_dim;
    pw.nT = d.rows;
    pw.out = dw;
  }
  ops.launch(st);
  char* const part = ws + pl.off_part;
  // one gradient alone is computed as it is beside the other: the same sums
  if (odd) ops.any = true;
  Backward t = tilings_bwd(d, pl.sum2);
  t.dx.tile = ops.tile(t.dx.tile);
  t.dw.tile = ops.tile(t.dw.tile);
  char* const part_dw = part + pl.off_part_dw;
  if (t.both && dx && dw) {
    px = tiled(px, t.dx, part);
    pw = tiled(pw, t.dw, part_dw);
    launch_mm_both(px, pw, t.dx.tile, t.behind, t.few, pl.sum2, st);
    join(px, st);
    join(pw, st);
  } else {
    if (dx) run_mm(px, t.dx, true, false, pl.sum2, part, st);
    if (dw) run_mm(pw, t.dw, false, false, pl.sum2, part_dw, st);
  }
  return int(hipGetLastError());
}

int launch_linear_bwd(const ss_linear_desc_t& d, const LinearPlan& pl, const void* x,
                      const int8_t* q, const uint8_t* e, const void* w, const void* pre,
                      const void* dy, void* dx, void* dw, float* dbias, char* ws, void* stream) {
  hipStream_t st = static_cast<hipStream_t>(stream);
  const bool dpre = pl.need_dpre && (dx || dw);
  if (dbias || dpre) {
    DpreParams p{dy, pre, dpre ? ws + pl.off_dpre : nullptr,
                 dbias ? reinterpret_cast<float*>(ws + pl.off_sums) : nullptr, d.rows,
                 pl.chunk_rows, int32_t(d.out_dim), int32_t(pl.ld_dpre), d.act, pl.sum2};
    const int v = dpre_vec(d.out_dim);
    const int64_t cols = pad_to_unit(d, d.out_dim);
    const dim3 grid(unsigned((cols + 64 * v - 1) / (64 * v)), unsigned(pl.chunks));
    if (v == 8) dpre_types<8>(d, p, grid, st);
    else dpre_types<1>(d, p, grid, st);
    if (dbias)
      launch_column_sums(p.part, dbias, nullptr, nullptr, pl.chunks, int32_t(d.out_dim), stream);
  }
  return backward_products(d, pl, dpre ? static_cast<const void*>(ws + pl.off_dpre) : dy,
                           !dpre && d.out_dim % unit_of(d) != 0, x, q, e, w, dx, dw, ws, stream);
}

// Gated products: the projection's plan and launches with twice the columns.
static ss_linear_desc_t both_halves(const ss_glu_desc_t& d) {
  ss_linear_desc_t l{};
  l.rows = d.rows;
  l.in_dim = d.in_dim;
  l.out_dim = 2 * d.out_dim;
  l.x_stride = d.x_stride;
  l.in_dtype = d.in_dtype;
  l.out_dtype = d.out_dtype;
  l.grad_dtype = d.grad_dtype;
  l.act = SS_ACT_SILU;       // dpre is never dy itself
  return l;
}
LinearPlan plan_glu(const ss_glu_desc_t& d, int op) {
  const ss_linear_desc_t l = both_halves(d);
  LinearPlan pl = plan_bwd_fwd(l, op == SS_GLU_FWD ? SS_LINEAR_FWD : SS_LINEAR_BWD, true);
  return pl;
}

int launch_glu_fwd(const ss_glu_desc_t& d, const LinearPlan& pl, const void* x, const void* w,
                   const float* bias, void* y, void* pre, char* ws, void* stream) {
  hipStream_t st = static_cast<hipStream_t>(stream);
  const ss_linear_desc_t l = both_halves(d);
  MmParams p{};
  p.ldr = d.x_stride ? d.x_stride : d.in_dim;
  p.lds = d.in_dim;
  p.nR = d.rows;
  p.nS = int32_t(d.out_dim);
  p.nT = d.in_dim;
  p.bias = bias;
  p.out = y;
  p.pre = pre;
  p.act = d.act;
  p.out_bf16 = d.out_dtype == SS_BF16;
  p.pre_bf16 = d.in_dtype == SS_BF16;
  if (d.rows <= kRowsMax) {
    const int e = unit_of(l);
    p.R = x;
    p.S = w;
    launch_rows_glu(p, d.in_dtype == SS_BF16, ptr16(x) && p.ldr % e == 0 && p.nT % e == 0, st);
    return int(hipGetLastError());
  }
  Operands ops{d.in_dtype == SS_BF16 ? 2 : 4};
  p.R = ops.take(x, &p.ldr, d.rows, d.in_dim, ws + pl.off_x);
  p.S = ops.take(w, &p.lds, 2 * d.out_dim, d.in_dim, ws + pl.off_w);
  ops.launch(st);
  const Tiling t = tiling_fwd(l, l.out_dim);
  p = tiled(p, t, ws + pl.off_part);
  launch_mm_glu(p, ops.tile(t.tile), st);
  if (p.splits > 1) {
    const int64_t n = (p.nR * p.nS + kThreads - 1) / kThreads;
    join_glu_kernel<<<unsigned(n < kMaxBlocks ? n : kMaxBlocks), kThreads, 0, st>>>(p);
  }
  return int(hipGetLastError());
}

template <typename Dy, typename T, int V, int ACT>
static void dglu_sums(const DgluParams& p, dim3 grid, hipStream_t st) {
  if (p.part) dglu_kernel<Dy, T, V, ACT, true><<<grid, kThreads, 0, st>>>(p);
  else dglu_kernel<Dy, T, V, ACT, false><<<grid, kThreads, 0, st>>>(p);
}
template <typename Dy, typename T, int V>
static void dglu_act(const DgluParams& p, int act, dim3 grid, hipStream_t st) {
  switch (act) {
    case SS_ACT_SILU: dglu_sums<Dy, T, V, SS_ACT_SILU>(p, grid, st); break;
    case SS_ACT_GELU: dglu_sums<Dy, T, V, SS_ACT_GELU>(p, grid, st); break;
    default: dglu_sums<Dy, T, V, SS_ACT_NONE>(p, grid, st);
  }
}
template <int V>
static void dglu_types(const ss_glu_desc_t& d, const DgluParams& p, dim3 grid, hipStream_t st) {
  const bool yb = d.out_dtype == SS_BF16, tb = d.in_dtype == SS_BF16;
  if (yb && tb) dglu_act<uint16_t, uint16_t, V>(p, d.act, grid, st);
  else if (yb) dglu_act<uint16_t, float, V>(p, d.act, grid, st);
  else if (tb) dglu_act<float, uint16_t, V>(p, d.act, grid, st);
  else dglu_act<float, float, V>(p, d.act, grid, st);
}

int launch_glu_bwd(const ss_glu_desc_t& d, const LinearPlan& pl, const void* x, const void* w,
                   const void* pre, const void* dy, void* dx, void* dw, float* dbias, char* ws,
                   void* stream) {
  hipStream_t st = static_cast<hipStream_t>(stream);
  const ss_linear_desc_t l = both_halves(d);
  const bool dpre = dx || dw;
  const int v = dpre_vec(d.out_dim);
  // with single columns, lanes past F clear the rows' last unit
  const int64_t cols = v == 8 ? d.out_dim : d.out_dim + pad_to_unit(l, l.out_dim) - l.out_dim;
  const int64_t across = (cols + 64 * v - 1) / (64 * v);
  // without column sums a block has no reason to walk but the grid's limits
  const int64_t most = kMaxBlocks / across < 32768 ? kMaxBlocks / across : 32768;
  const int64_t turns = (d.rows + kDgluRows * most - 1) / (kDgluRows * most);
  const int64_t rows = dbias ? pl.chunk_rows : kDgluRows * turns;
  const DgluParams p{dy, pre, dpre ? ws + pl.off_dpre : nullptr,
                     dbias ? reinterpret_cast<float*>(ws + pl.off_sums) : nullptr, d.rows, rows,
                     int32_t(d.out_dim), int32_t(pl.ld_dpre), pl.sum2};
  const dim3 grid(unsigned(across), unsigned((d.rows + rows - 1) / rows));
  if (v == 8) dglu_types<8>(d, p, grid, st);
  else dglu_types<1>(d, p, grid, st);
  if (dbias)
    launch_column_sums(p.part, dbias, nullptr, nullptr, pl.chunks, int32_t(l.out_dim), stream);
  if (!dpre) return int(hipGetLastError());
  return backward_products(l, pl, ws + pl.off_dpre, false, x, nullptr, nullptr, w, dx, dw, ws,
                           stream);
}

// 8-bit integers: tiles, stages and splits as for bf16, at 128 of the contraction a stage.
static Tiling tiling_q8(const ss_q8_desc_t& d) {
  return tiling(Small(false, 1, d.rows, d.out_dim, d.in_dim));
}
Q8Plan plan_q8(const ss_q8_desc_t& d) {
  Q8Plan pl;
  if (d.rows <= kRowsMax) return pl;
  auto take = [&](size_t bytes) {
    const size_t at = pl.bytes;
    pl.bytes += align256(bytes);
    return at;
  };
  const int64_t units = (d.in_dim + 15) / 16 * 16;
  if (d.in_dim % 16 != 0 || d.x_stride != 0) pl.off_x = take(size_t(d.rows) * size_t(units));
  if (d.in_dim % 16 != 0 || d.w_stride != 0) pl.off_w = take(size_t(d.out_dim) * size_t(units));
  pl.off_part = take(part_bytes(tiling_q8(d), d.rows, d.out_dim));
  return pl;
}
int launch_q8_linear(const ss_q8_desc_t& d, const Q8Plan& pl, const int8_t* xq, const float* xs,
                     const int8_t* wq, const float* wsc, const float* bias, const void* residual,
                     void* y, char* ws, void* stream) {
  hipStream_t st = static_cast<hipStream_t>(stream);
  MmParams p{};
  p.ldr = d.x_stride ? d.x_stride : d.in_dim;
  p.lds = d.w_stride ? d.w_stride : d.in_dim;
  p.nR = d.rows;
  p.nS = int32_t(d.out_dim);
  p.nT = d.in_dim;
  p.bias = bias;
  p.res = residual;
  p.out = y;
  p.act = d.act;
  p.out_bf16 = d.out_dtype == SS_BF16;
  p.res_bf16 = d.res_dtype == SS_BF16;
  p.row_scale = xs;
  p.col_scale = wsc;
  if (d.rows <= kRowsMax) {
    p.R = xq;
    p.S = wq;
    launch_rows_q8(p, ptr16(xq) && ptr16(wq) && p.ldr % 16 == 0 && p.lds % 16 == 0 &&
                          p.nT % 16 == 0, st);
    return int(hipGetLastError());
  }
  const Tiling t = tiling_q8(d);
  Operands ops{1};
  // Rows whose units are aligned are read in place.  What lies behind an odd contraction's
  // end, in the row's last unit, is cleared in small tiles' registers, and meets the zeros of
  // w's copy in large ones.
  if (ptr16(xq) && p.ldr % 16 == 0) p.R = xq;
  else p.R = ops.take(xq, &p.ldr, d.rows, d.in_dim, ws + pl.off_x);
  if (t.tile != MmTile::kBig && ptr16(wq) && p.lds % 16 == 0) p.S = wq;
  else p.S = ops.take(wq, &p.lds, d.out_dim, d.in_dim, ws + pl.off_w);
  ops.launch(st);
  p = tiled(p, t, ws + pl.off_part);
  launch_mm_q8(p, t.tile, st);
  if (p.splits > 1) {
    const int64_t n = (p.nR * p.nS + kThreads - 1) / kThreads;
    join_q8_kernel<<<unsigned(n < kMaxBlocks ? n : kMaxBlocks), kThreads, 0, st>>>(p);
  }
  return int(hipGetLastError());
}

}  // namespace ss
