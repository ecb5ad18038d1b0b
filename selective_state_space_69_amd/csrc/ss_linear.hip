// Linear projections for gfx950: the general product, the backward's
// pre-activation gradient, the join of split contractions, and the launchers.
//
// The general kernel serves every type, alignment and size: 128 x 128 output
// tiles, 4 waves of 64 x 64, both operands staged through registers into LDS as
// rows of t (128 bytes: 64 bf16 or 32 fp32), whatever their order in memory, and
// multiplied by v_mfma_f32_16x16x32_bf16 or v_mfma_f32_16x16x4_f32.  A lane
// supplies 16 bytes of t at a time to either; the four fp32 products of those 16
// bytes number t as 4 g + i (g = lane / 16) on both sides alike.
#include "ss_linear_mm.hpp"

namespace ss {
namespace {

constexpr int kTile = 128;
constexpr int kThreads = 256;
constexpr int kRowBytes = 128;                      // bytes of t per LDS row
constexpr int64_t kMaxBlocks = int64_t(1) << 22;    // a grid's threads stay below 2^32

template <typename T> constexpr int kStep = kRowBytes / int(sizeof(T));   // t per stage

// 16-byte unit c (0..7) of LDS row i; units are permuted within a row so that
// the 16 rows of a fragment read touch all banks evenly
__device__ __forceinline__ int lds_unit(int i, int c) { return i * 8 + (c ^ (i & 7)); }

// One thread's share of an operand tile: 4 units of 16 bytes, held in registers
// between the global read and the LDS write.
template <typename T, bool TCONTIG>
struct Stage {
  static constexpr int E = 16 / int(sizeof(T));    // elements per unit
  u32x4 u[4];

  // rows i0.. of n, contraction t0.. up to t1
  __device__ __forceinline__ void load(const T* p, int64_t ld, bool vec, int64_t i0, int64_t n,
                                       int64_t t0, int64_t t1) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int id = int(threadIdx.x) + k * kThreads;
      int64_t a, b, an, bn;      // a: storage row, b: first element of the unit in it
      if constexpr (TCONTIG) {
        a = i0 + id / 8;
        b = t0 + (id % 8) * E;
        an = n;
        bn = t1;
      } else {
        constexpr int per = kTile / E;
        a = t0 + id / per;
        b = i0 + (id % per) * E;
        an = t1;
        bn = n;
      }
      u[k] = u32x4{0, 0, 0, 0};
      if (a >= an || b >= bn) continue;
      const T* src = p + a * ld + b;
      if (vec && b + E <= bn) {
        u[k] = *reinterpret_cast<const u32x4*>(src);
      } else {
        T e[E];
#pragma unroll
        for (int j = 0; j < E; ++j) e[j] = b + j < bn ? src[j] : T(0);
        u[k] = __builtin_bit_cast(u32x4, e);
      }
    }
  }

  __device__ __forceinline__ void write(u32x4* lds) const {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int id = int(threadIdx.x) + k * kThreads;
      if constexpr (TCONTIG) {
        lds[lds_unit(id / 8, id % 8)] = u[k];
      } else {
        constexpr int per = kTile / E;
        const int t = id / per, i = (id % per) * E;
        struct Elems { T e[E]; };
        const Elems v = __builtin_bit_cast(Elems, u[k]);
#pragma unroll
        for (int j = 0; j < E; ++j)
          reinterpret_cast<T*>(&lds[lds_unit(i + j, t / E)])[t % E] = v.e[j];
      }
    }
  }
};

template <typename T>
__device__ __forceinline__ f32x4 mma(u32x4 a, u32x4 b, f32x4 c) {
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

template <typename T, bool RT, bool ST>
__global__ __launch_bounds__(kThreads) void mm_kernel(MmParams p) {
  __shared__ u32x4 lr[kTile * 8], ls[kTile * 8];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int wr = (wv & 1) * 64, wsn = (wv >> 1) * 64;      // the wave's corner of the tile
  const int m = lane & 15, g = lane >> 4;
  const int64_t items = int64_t(p.tiles_r) * p.tiles_s * p.splits;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int64_t tiles = int64_t(p.tiles_r) * p.tiles_s;
    const int split = int(it / tiles);
    int64_t tr;
    int ts;
    tile_of(p, xcd_contiguous(it - split * tiles, tiles), &tr, &ts);
    const int64_t r0 = tr * kTile;
    const int64_t s0 = int64_t(ts) * kTile;
    const int64_t t0 = split * p.t_split;
    const int64_t t1 = t0 + p.t_split < p.nT ? t0 + p.t_split : p.nT;
    f32x4 acc[4][4];      // [s][r]
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
    Stage<T, RT> sr;
    Stage<T, ST> ss_;
    sr.load(static_cast<const T*>(p.R), p.ldr, p.vec_r, r0, p.nR, t0, t1);
    ss_.load(static_cast<const T*>(p.S), p.lds, p.vec_s, s0, p.nS, t0, t1);
    for (int64_t t = t0; t < t1; t += kStep<T>) {
      __syncthreads();                 // the previous stage has been read
      sr.write(lr);
      ss_.write(ls);
      __syncthreads();
      if (t + kStep<T> < t1) {
        sr.load(static_cast<const T*>(p.R), p.ldr, p.vec_r, r0, p.nR, t + kStep<T>, t1);
        ss_.load(static_cast<const T*>(p.S), p.lds, p.vec_s, s0, p.nS, t + kStep<T>, t1);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        u32x4 a[4], b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          a[i] = ls[lds_unit(wsn + 16 * i + m, 4 * h + g)];
          b[i] = lr[lds_unit(wr + 16 * i + m, 4 * h + g)];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][j] = mma<T>(a[i], b[j], acc[i][j]);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float v[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
        const int64_t r = r0 + wr + 16 * j + m;
        const int32_t s = int32_t(s0) + wsn + 16 * i + 4 * g;
        if (p.splits > 1) store_partial4(p, split, r, s, v);
        else epilogue4(p, r, s, v);
      }
  }
}

// Sum of the splits' partials, in order, and the epilogue.
__global__ __launch_bounds__(kThreads) void join_kernel(MmParams p) {
  const int64_t quads = (p.nS + 3) / 4;
  const int64_t total = p.nR * quads;
  for (int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x; i < total;
       i += int64_t(gridDim.x) * kThreads) {
    const int64_t r = i / quads;
    const int32_t s = int32_t(i - r * quads) * 4;
    float v[4] = {0, 0, 0, 0};
    for (int k = 0; k < p.splits; ++k) {
      const float* src = p.part + (int64_t(k) * p.nR + r) * p.nS + s;
      if ((p.nS & 3) == 0) {
        const float4 f = *reinterpret_cast<const float4*>(src);
        v[0] += f.x; v[1] += f.y; v[2] += f.z; v[3] += f.w;
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (s + j < p.nS) v[j] += src[j];
      }
    }
    epilogue4(p, r, s, v);
  }
}

// dpre = dy act'(pre) in the operand type (when asked for) and its column sums
// before that rounding: 64 columns x 4 waves per block, a wave takes every
// fourth row of the block's rows, the four sums are added in wave order into
// one partial row per block.
struct DpreParams {
  const void* dy;
  const void* pre;
  void* d;            // or null
  float* part;        // (gridDim.y, N) or null
  int64_t M, rows;    // rows per block
  int32_t N, act;
};
template <typename Dy, typename T>
__global__ __launch_bounds__(kThreads) void dpre_kernel(DpreParams p) {
  __shared__ float part[4][64];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int64_t c = int64_t(blockIdx.x) * 64 + lane;
  const int64_t m0 = int64_t(blockIdx.y) * p.rows;
  const int64_t m1 = m0 + p.rows < p.M ? m0 + p.rows : p.M;
  float sum = 0.0f;
  if (c < p.N) {
    for (int64_t m = m0 + wv; m < m1; m += 4) {
      float v = to_f32(static_cast<const Dy*>(p.dy)[m * p.N + c]);
      if (p.act != SS_ACT_NONE)
        v *= act_grad(p.act, to_f32(static_cast<const T*>(p.pre)[m * p.N + c]));
      if (p.d) store_out<T>(static_cast<T*>(p.d) + m * p.N + c, v);
      sum += v;
    }
  }
  if (!p.part) return;
  part[wv][lane] = sum;
  __syncthreads();
  if (wv == 0 && c < p.N)
    p.part[int64_t(blockIdx.y) * p.N + c] =
        (part[0][lane] + part[1][lane]) + (part[2][lane] + part[3][lane]);
}

__global__ __launch_bounds__(kThreads) void column_sum_kernel(const float* src, float* dst,
                                                              int64_t nparts, int32_t N) {
  __shared__ float part[4][64];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int64_t c = int64_t(blockIdx.x) * 64 + lane;
  float acc = 0.0f;
  if (c < N) {
#pragma unroll 8
    for (int64_t i = wv; i < nparts; i += 4) acc += src[i * N + c];
  }
  part[wv][lane] = acc;
  __syncthreads();
  if (wv == 0 && c < N)
    dst[c] = (part[0][lane] + part[1][lane]) + (part[2][lane] + part[3][lane]);
}

size_t align256(size_t x) { return (x + 255) / 256 * 256; }
bool ptr16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// Splits of the contraction over 128 x 128 tiles: enough work items for two
// rounds of the 256 CUs, each at least 4 stages long.
void plan_splits(int64_t nR, int64_t nS, int64_t nT, int step, int32_t* splits, int64_t* t_split) {
  const int64_t tiles = ((nR + kTile - 1) / kTile) * ((nS + kTile - 1) / kTile);
  int64_t k = tiles >= 256 ? 1 : (512 + tiles - 1) / tiles;
  const int64_t most = nT / (4 * step);
  if (k > most) k = most;
  if (k > 64) k = 64;
  if (k < 1) k = 1;
  int64_t len = (nT + k - 1) / k;
  len = (len + step - 1) / step * step;
  *t_split = len;
  *splits = int32_t((nT + len - 1) / len);
}

int step_of(const ss_linear_desc_t& d) {
  return d.in_dtype == SS_BF16 ? kStep<uint16_t> : kStep<float>;
}

size_t part_bytes(int64_t nR, int64_t nS, int64_t nT, int step) {
  int32_t splits;
  int64_t len;
  plan_splits(nR, nS, nT, step, &splits, &len);
  return splits > 1 ? align256(size_t(splits) * size_t(nR) * size_t(nS) * 4) : 0;
}

template <bool RT, bool ST>
void run_mm(MmParams p, int32_t in_dtype, hipStream_t st) {
  const int step = in_dtype == SS_BF16 ? kStep<uint16_t> : kStep<float>;
  const int e = in_dtype == SS_BF16 ? 8 : 4;
  plan_splits(p.nR, p.nS, p.nT, step, &p.splits, &p.t_split);
  p.tiles_r = int32_t((p.nR + kTile - 1) / kTile);
  p.tiles_s = (p.nS + kTile - 1) / kTile;
  p.vec_r = ptr16(p.R) && p.ldr % e == 0;
  p.vec_s = ptr16(p.S) && p.lds % e == 0;
  const int64_t items = int64_t(p.tiles_r) * p.tiles_s * p.splits;
  const unsigned blocks = unsigned(items < kMaxBlocks ? items : kMaxBlocks);
  if (in_dtype == SS_BF16 && items <= kMaxBlocks &&
      mm_operand_ok(p.R, p.ldr, RT ? p.nT : p.nR) && mm_operand_ok(p.S, p.lds, ST ? p.nT : p.nS)) {
    const int64_t tiles = (p.nR + 255) / 256 * ((p.nS + 255) / 256);
    const bool big = tiles >= 128;
    if (big) {
      p.tiles_r = int32_t((p.nR + 255) / 256);
      p.tiles_s = (p.nS + 255) / 256;
      p.splits = 1;
    }
    launch_mm(p, big, RT, ST, st);
  } else if (in_dtype == SS_BF16) {
    mm_kernel<uint16_t, RT, ST><<<blocks, kThreads, 0, st>>>(p);
  } else {
    mm_kernel<float, RT, ST><<<blocks, kThreads, 0, st>>>(p);
  }
  if (p.splits > 1) {
    const int64_t n = (p.nR * ((p.nS + 3) / 4) + kThreads - 1) / kThreads;
    join_kernel<<<unsigned(n < kMaxBlocks ? n : kMaxBlocks), kThreads, 0, st>>>(p);
  }
}

}  // namespace

LinearPlan plan_linear(const ss_linear_desc_t& d, int op) {
  LinearPlan pl;
  const int step = step_of(d);
  const size_t esize = d.in_dtype == SS_BF16 ? 2 : 4;
  if (op == SS_LINEAR_FWD) {
    pl.bytes = part_bytes(d.rows, d.out_dim, d.in_dim, step);
    return pl;
  }
  pl.need_dpre = d.act != SS_ACT_NONE || d.out_dtype != d.in_dtype;
  // about 1024 blocks over the columns and row chunks, at least 16 rows each
  const int64_t cols = (d.out_dim + 63) / 64;
  int64_t chunks = (1024 + cols - 1) / cols;
  const int64_t most = (d.rows + 15) / 16;
  if (chunks > most) chunks = most;
  pl.chunk_rows = (d.rows + chunks - 1) / chunks;
  pl.chunks = (d.rows + pl.chunk_rows - 1) / pl.chunk_rows;
  size_t off = 0;
  if (pl.need_dpre) {
    pl.off_dpre = off;
    off += align256(size_t(d.rows) * size_t(d.out_dim) * esize);
  }
  if (op == SS_LINEAR_BWD_CKPT) {
    pl.off_x = off;
    off += align256(size_t(d.rows) * size_t(d.in_dim) * esize);
  }
  pl.off_sums = off;
  off += align256(size_t(pl.chunks) * size_t(d.out_dim) * 4);
  pl.off_part = off;
  const size_t a = part_bytes(d.rows, d.in_dim, d.out_dim, step);
  const size_t b = part_bytes(d.out_dim, d.in_dim, d.rows, step);
  off += a > b ? a : b;
  pl.bytes = off;
  return pl;
}

int launch_linear_fwd(const ss_linear_desc_t& d, const void* x, const void* w, const float* bias,
                      const void* residual, void* y, void* pre, char* ws, void* stream) {
  MmParams p{};
  p.R = x;
  p.S = w;
  p.ldr = d.x_stride ? d.x_stride : d.in_dim;
  p.lds = d.in_dim;
  p.nR = d.rows;
  p.nS = int32_t(d.out_dim);
  p.nT = d.in_dim;
  p.bias = bias;
  p.res = residual;
  p.out = y;
  p.pre = pre;
  p.part = reinterpret_cast<float*>(ws);
  p.act = d.act;
  p.out_bf16 = d.out_dtype == SS_BF16;
  p.res_bf16 = d.res_dtype == SS_BF16;
  p.pre_bf16 = d.in_dtype == SS_BF16;
  run_mm<true, true>(p, d.in_dtype, static_cast<hipStream_t>(stream));
  return int(hipGetLastError());
}

int launch_linear_bwd(const ss_linear_desc_t& d, const LinearPlan& pl, const void* x,
                      const int8_t* q, const uint8_t* e, const void* w, const void* pre,
                      const void* dy, void* dx, void* dw, float* dbias, char* ws, void* stream) {
  hipStream_t st = static_cast<hipStream_t>(stream);
  const void* g = pl.need_dpre ? static_cast<const void*>(ws + pl.off_dpre) : dy;
  if (dbias || (pl.need_dpre && (dx || dw))) {
    DpreParams p{dy, pre, pl.need_dpre && (dx || dw) ? ws + pl.off_dpre : nullptr,
                 dbias ? reinterpret_cast<float*>(ws + pl.off_sums) : nullptr, d.rows,
                 pl.chunk_rows, int32_t(d.out_dim), d.act};
    const dim3 grid(unsigned((d.out_dim + 63) / 64), unsigned(pl.chunks));
    const bool yb = d.out_dtype == SS_BF16, tb = d.in_dtype == SS_BF16;
    if (yb && tb) dpre_kernel<uint16_t, uint16_t><<<grid, kThreads, 0, st>>>(p);
    else if (yb) dpre_kernel<uint16_t, float><<<grid, kThreads, 0, st>>>(p);
    else if (tb) dpre_kernel<float, uint16_t><<<grid, kThreads, 0, st>>>(p);
    else dpre_kernel<float, float><<<grid, kThreads, 0, st>>>(p);
    if (dbias)
      column_sum_kernel<<<grid.x, kThreads, 0, st>>>(p.part, dbias, pl.chunks,
                                                     int32_t(d.out_dim));
  }
  MmParams p{};
  p.R = g;
  p.ldr = d.out_dim;
  p.nS = int32_t(d.in_dim);
  p.part = reinterpret_cast<float*>(ws + pl.off_part);
  p.act = SS_ACT_NONE;
  p.out_bf16 = d.grad_dtype == SS_BF16;
  if (dx) {
    p.S = w;
    p.lds = d.in_dim;
    p.nR = d.rows;
    p.nT = d.out_dim;
    p.out = dx;
    run_mm<true, false>(p, d.in_dtype, st);
  }
  if (dw) {
    if (q) {
      ss_ckpt_desc_t c{};
      c.rows = d.rows;
      c.dim = d.in_dim;
      c.dtype = d.in_dtype;
      const int rc = launch_ckpt_unpack(c, q, e, ws + pl.off_x, stream);
      if (rc) return rc;
      x = ws + pl.off_x;
    }
    p.S = x;
    p.lds = q || !d.x_stride ? d.in_dim : d.x_stride;
    p.nR = d.out_dim;
    p.nT = d.rows;
    p.out = dw;
    run_mm<false, false>(p, d.in_dtype, st);
  }
  return int(hipGetLastError());
}

}  // namespace ss
