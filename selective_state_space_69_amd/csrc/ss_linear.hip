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

// bf16 rows of one or two tensors (blockIdx.y) at a 16-byte aligned stride, zero past
// their end: one 16-byte unit of the copy per thread.
struct PadJob {
  const void* src;
  void* dst;
  int64_t ld_src, rows;
  int32_t cols, units;     // units of a row of the copy
};
struct PadParams {
  PadJob job[2];
};
__global__ __launch_bounds__(kThreads) void pad_kernel(PadParams q) {
  constexpr int E = 8;
  const PadJob p = q.job[blockIdx.y];
  const int64_t total = p.rows * p.units;
  for (int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x; i < total;
       i += int64_t(gridDim.x) * kThreads) {
    const int64_t r = total <= INT32_MAX ? int64_t(uint32_t(i) / uint32_t(p.units)) : i / p.units;
    const int c = int(i - r * p.units) * E;
    const uint16_t* src = static_cast<const uint16_t*>(p.src) + r * p.ld_src + c;
    struct __attribute__((packed, aligned(2))) Elems { uint16_t e[E]; } v;
    if (c + E <= p.cols) {
      v = *reinterpret_cast<const Elems*>(src);      // 16 bytes at any element address
    } else {
#pragma unroll
      for (int j = 0; j < E; ++j) v.e[j] = c + j < p.cols ? src[j] : uint16_t(0);
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
  Small(const ss_linear_desc_t& d, int64_t r, int64_t s, int64_t t, bool sum2)
      : nR(r), nS(s), nT(t) {
    bf16 = d.in_dtype == SS_BF16;
    const int64_t side = bf16 ? 128 : 64;
    step = bf16 && !sum2 ? 64 : 32;
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
Tiling tiling(const ss_linear_desc_t& d, int64_t nR, int64_t nS, int64_t nT, bool sum2) {
  const int64_t r256 = (nR + 255) / 256, s256 = (nS + 255) / 256;
  const Small p(d, nR, nS, nT, sum2);
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
  const Small a(d, d.rows, d.in_dim, d.out_dim, sum2), b(d, d.out_dim, d.in_dim, d.rows, sum2);
  Backward t{tiling(d, a.nR, a.nS, a.nT, sum2), tiling(d, b.nR, b.nS, b.nT, sum2), false, 0, 0};
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
  const ss_linear_desc_t& d;
  PadParams pad{};
  int n = 0;
  bool any = false;
  // rows x cols of src, rows *ld elements apart: where the products read it
  const void* take(const void* src, int64_t* ld, int64_t rows, int64_t cols, char* dst) {
    const int e = unit_of(d);
    if (ptr16(src) && *ld % e == 0 && cols % e == 0) return src;
    if (d.in_dtype == SS_F32) {
      any = true;
      return src;
    }
    pad.job[n++] = PadJob{src, dst, *ld, rows, int32_t(cols), int32_t(pad_to_unit(d, cols) / e)};
    *ld = pad_to_unit(d, cols);
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
    pad_kernel<<<grid, kThreads, 0, st>>>(pad);
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
int dpre_vec(const ss_linear_desc_t& d) { return d.out_dim % 8 == 0 ? 8 : 1; }

}  // namespace

LinearPlan plan_linear(const ss_linear_desc_t& d, int op) {
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
        take(part_bytes(tiling(d, d.rows, d.out_dim, d.in_dim, false), d.rows, d.out_dim));
    pl.bytes = off;
    return pl;
  }
  pl.need_dpre = d.act != SS_ACT_NONE || d.out_dtype != d.in_dtype ||
                 (bf16 && d.out_dim % 8 != 0);
  pl.sum2 = bf16 && d.grad_dtype == SS_F32 &&
            (d.act != SS_ACT_NONE || d.out_dtype != SS_BF16);
  pl.ld_dpre = pad_to_unit(d, d.out_dim) * (pl.sum2 ? 2 : 1);
  // about 1024 blocks over the columns and row chunks, at least 16 rows each
  const int64_t span = 64 * dpre_vec(d), cols = (d.out_dim + span - 1) / span;
  int64_t chunks = (1024 + cols - 1) / cols;
  const int64_t most = (d.rows + 15) / 16;
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
  Operands ops{d};
  p.R = ops.take(x, &p.ldr, d.rows, d.in_dim, ws + pl.off_x);
  p.S = ops.take(w, &p.lds, d.out_dim, d.in_dim, ws + pl.off_w);
  ops.launch(st);
  Tiling t = tiling(d, p.nR, p.nS, p.nT, false);
  t.tile = ops.tile(t.tile);
  run_mm(p, t, true, true, false, ws + pl.off_part, st);
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
    const int v = dpre_vec(d);
    const int64_t cols = pad_to_unit(d, d.out_dim);
    const dim3 grid(unsigned((cols + 64 * v - 1) / (64 * v)), unsigned(pl.chunks));
    if (v == 8) dpre_types<8>(d, p, grid, st);
    else dpre_types<1>(d, p, grid, st);
    if (dbias)
      launch_column_sums(p.part, dbias, nullptr, nullptr, pl.chunks, int32_t(d.out_dim), stream);
  }
  MmParams p{};
  p.R = dpre ? static_cast<const void*>(ws + pl.off_dpre) : dy;
  p.ldr = pl.need_dpre ? pl.ld_dpre : d.out_dim;
  p.nS = int32_t(d.in_dim);
  p.act = SS_ACT_NONE;
  p.out_bf16 = d.grad_dtype == SS_BF16;
  Operands ops{d};
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
  if (!dpre && d.out_dim % unit_of(d) != 0) ops.any = true;     // dy in place (fp32)
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

}  // namespace ss
