// Layer norm with the residual add, forward and backward, for gfx950 (the norm
// in front of a Mamba block: Gu & Dao wiki note, "Mamba architecture").
//
//   s = x + residual, mean = sum s / D, rstd = 1 / sqrt(sum (s - mean)^2 / D + eps),
//   y = (s - mean) rstd w + b
//   g = dy w, xh = (s - mean) rstd:
//   dx = rstd (g - mean(g) - xh mean(g xh)) + dsum,  dw = sum_rows dy xh,  db = sum_rows dy
//
// Both passes stream: a row is read once into registers (8 channels per thread
// and vector, 16-byte loads), its sums are taken there and it is written once.
// The variance is a second sum over the registers, about the mean, so rows far
// from zero lose nothing; the rest of the mean that fp32 summation left in them
// is summed along with it and taken out too (a row of one value gives y = b).  A row belongs to the fewest waves that hold it with
// one vector per thread (D <= 8192; four vectors beyond).
#include "ss_device.hpp"

namespace ss {
namespace {

constexpr int kVec = 8;           // channels per thread and vector
constexpr int kMaxWaves = 16;
constexpr int64_t kMaxRowBlocks = int64_t(1) << 20;   // a grid's threads stay below 2^32

// Sum over the wave's 64 lanes, in a fixed order, in every lane: row_shr 1, 2,
// 4, 8 leave each 16-lane row's sum in its last lane, the two row broadcasts
// carry it on to lane 63.
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_add(float v) {
  const int s = __builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, ROWS, 0xf, true);
  return v + __int_as_float(s);
}
__device__ __forceinline__ float wave_sum(float v) {
  v = dpp_add<0x111, 0xf>(v);
  v = dpp_add<0x112, 0xf>(v);
  v = dpp_add<0x114, 0xf>(v);
  v = dpp_add<0x118, 0xf>(v);
  v = dpp_add<0x142, 0xa>(v);
  v = dpp_add<0x143, 0xc>(v);
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

// 8 channels of a row in fp32.  VEC: 8 neighbours from column c, by 16-byte
// loads; else 8 columns c, c + step, ... of which only those below D exist.
template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T* row, int c, int step, int D, float (&v)[kVec]) {
  if constexpr (VEC) {
    if (c < D) {
      if constexpr (sizeof(T) == 2) {
        const uint4 r = *reinterpret_cast<const uint4*>(row + c);
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[2 * i] = __uint_as_float(w[i] << 16);
          v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
      } else {
        const float4 a = *reinterpret_cast<const float4*>(row + c);
        const float4 b = *reinterpret_cast<const float4*>(row + c + 4);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < kVec; ++j) v[j] = 0.0f;
    }
  } else {
#pragma unroll
    for (int j = 0; j < kVec; ++j) v[j] = c + j * step < D ? to_f32(row[c + j * step]) : 0.0f;
  }
}

template <typename T, bool VEC>
__device__ __forceinline__ void store8(T* row, int c, int step, int D, const float (&v)[kVec]) {
  if constexpr (VEC) {
    if (c < D) {
      if constexpr (sizeof(T) == 2) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          w[i] = uint32_t(f32_to_bf16(v[2 * i])) | (uint32_t(f32_to_bf16(v[2 * i + 1])) << 16);
        *reinterpret_cast<uint4*>(row + c) = make_uint4(w[0], w[1], w[2], w[3]);
      } else {
        *reinterpret_cast<float4*>(row + c) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4*>(row + c + 4) = make_float4(v[4], v[5], v[6], v[7]);
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < kVec; ++j)
      if (c + j * step < D) store_out<T>(row + c + j * step, v[j]);
  }
}

// A thread's place in its row: tpr threads per row, vector k of thread t starts
// at column (k tpr + t) 8 (VEC) or t + k 8 tpr with steps of tpr.
struct Place {
  int tid, tpr, wave, nwaves;
  int64_t row;        // first row
  int64_t row_step;
};
__device__ __forceinline__ Place place(int nwaves) {
  Place a;
  a.nwaves = nwaves;
  a.tpr = nwaves * kWave;
  const int sub = nwaves == 1 ? int(threadIdx.x) / kWave : 0;   // rows side by side in a block
  a.tid = int(threadIdx.x) - sub * a.tpr;
  a.wave = a.tid / kWave;
  const int rows = nwaves == 1 ? int(blockDim.x) / kWave : 1;
  a.row = int64_t(blockIdx.x) * rows + sub;
  a.row_step = int64_t(gridDim.x) * rows;
  return a;
}
template <bool VEC>
__device__ __forceinline__ int col0(const Place& a, int k) {
  return VEC ? (k * a.tpr + a.tid) * kVec : k * kVec * a.tpr + a.tid;
}

// Sums of v[0..N) over a row's threads; every thread gets them.  buf: floats that
// no wave still reads from an earlier use (callers alternate).
template <int N>
__device__ __forceinline__ void row_sum(const Place& a, float (&v)[N], float (&buf)[N][kMaxWaves]) {
#pragma unroll
  for (int n = 0; n < N; ++n) v[n] = wave_sum(v[n]);
  if (a.nwaves == 1) return;
  if ((threadIdx.x & 63) == 0) {
#pragma unroll
    for (int n = 0; n < N; ++n) buf[n][a.wave] = v[n];
  }
  __syncthreads();
#pragma unroll
  for (int n = 0; n < N; ++n) v[n] = 0.0f;
  for (int i = 0; i < a.nwaves; ++i)
#pragma unroll
    for (int n = 0; n < N; ++n) v[n] += buf[n][i];
}

struct NormFwdParams {
  const void* x;
  const void* res;
  const float* w;
  const float* b;
  void* y;
  void* sum;
  float* mean;
  float* rstd;
  int64_t rows, xs;
  int D, nwaves;
  float eps, inv_d;
};

template <typename In, typename Res, typename Out, bool VEC, int VPT>
__global__ __launch_bounds__(1024) void norm_fwd_kernel(NormFwdParams p) {
  __shared__ float buf1[1][kMaxWaves], buf2[2][kMaxWaves];
  const Place a = place(p.nwaves);
  // one row per block, or one per wave without barriers: a row is uniform over
  // everything that meets at row_sum's barrier
  for (int64_t row = a.row; row < p.rows; row += a.row_step) {
    const int64_t o = row * p.D;
    float s[VPT][kVec];
    float t[1] = {0.0f};
#pragma unroll
    for (int k = 0; k < VPT; ++k)
      load8<In, VEC>(static_cast<const In*>(p.x) + row * p.xs, col0<VEC>(a, k), a.tpr, p.D, s[k]);
    if (p.res) {
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        float r[kVec];
        load8<Res, VEC>(static_cast<const Res*>(p.res) + o, col0<VEC>(a, k), a.tpr, p.D, r);
#pragma unroll
        for (int j = 0; j < kVec; ++j) s[k][j] += r[j];
      }
    }
#pragma unroll
    for (int k = 0; k < VPT; ++k)
#pragma unroll
      for (int j = 0; j < kVec; ++j) t[0] += s[k][j];
    if (p.sum) {
#pragma unroll
      for (int k = 0; k < VPT; ++k)
        store8<Res, VEC>(static_cast<Res*>(p.sum) + o, col0<VEC>(a, k), a.tpr, p.D, s[k]);
    }
    row_sum(a, t, buf1);
    const float mean = t[0] * p.inv_d;
    float c[2] = {0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < VPT; ++k)
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        const bool on = col0<VEC>(a, k) + (VEC ? 0 : j * a.tpr) < p.D;
        s[k][j] = on ? s[k][j] - mean : 0.0f;
        c[0] += s[k][j];
        c[1] = __builtin_fmaf(s[k][j], s[k][j], c[1]);
      }
    row_sum(a, c, buf2);
    const float rest = c[0] * p.inv_d;
    const float var = __builtin_fmaf(c[1], p.inv_d, -rest * rest);
    // var is never below 0 but for rounding; NaN passes
    const float rstd = 1.0f / __builtin_sqrtf((var < 0.0f ? 0.0f : var) + p.eps);
    if (p.mean && a.tid == 0) {
      p.mean[row] = mean + rest;
      p.rstd[row] = rstd;
    }
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int col = col0<VEC>(a, k);
      float f[kVec];
#pragma unroll
      for (int j = 0; j < kVec; ++j) s[k][j] = (s[k][j] - rest) * rstd;
      if (p.w) {
        load8<float, VEC>(p.w, col, a.tpr, p.D, f);
#pragma unroll
        for (int j = 0; j < kVec; ++j) s[k][j] *= f[j];
      }
      if (p.b) {
        load8<float, VEC>(p.b, col, a.tpr, p.D, f);
#pragma unroll
        for (int j = 0; j < kVec; ++j) s[k][j] += f[j];
      }
      store8<Out, VEC>(static_cast<Out*>(p.y) + o, col, a.tpr, p.D, s[k]);
    }
  }
}

struct NormBwdParams {
  const void* s;
  const float* w;
  const float* mean;
  const float* rstd;
  const void* dy;
  const void* dsum;
  void* dx;
  float* pw;      // (partials, D) dweight sums of a block's rows, or null
  float* pb;
  int64_t rows, xs;
  int D, nwaves;
  float inv_d;
};

// ACC: also sum dy xh and dy over the block's rows, in registers, one partial
// row per walker (block, or wave where a row is one wave's).
template <typename In, typename Res, typename Out, bool VEC, int VPT, bool ACC>
__global__ __launch_bounds__(1024) void norm_bwd_kernel(NormBwdParams p) {
  __shared__ float buf[2][2][kMaxWaves];
  const Place a = place(p.nwaves);
  float aw[ACC ? VPT : 1][kVec], ab[ACC ? VPT : 1][kVec];
  if constexpr (ACC) {
#pragma unroll
    for (int k = 0; k < VPT; ++k)
#pragma unroll
      for (int j = 0; j < kVec; ++j) aw[k][j] = ab[k][j] = 0.0f;
  }
  int par = 0;
  for (int64_t row = a.row; row < p.rows; row += a.row_step, par ^= 1) {
    const int64_t o = row * p.D;
    float xh[VPT][kVec], g[VPT][kVec];
    const float mean = p.mean[row], rstd = p.rstd[row];
    float t1 = 0.0f, t2 = 0.0f;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int c = col0<VEC>(a, k);
      load8<In, VEC>(static_cast<const In*>(p.s) + row * p.xs, c, a.tpr, p.D, xh[k]);
      load8<Out, VEC>(static_cast<const Out*>(p.dy) + o, c, a.tpr, p.D, g[k]);
    }
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      float w[kVec];
      if (p.w) load8<float, VEC>(p.w, col0<VEC>(a, k), a.tpr, p.D, w);
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        const bool on = col0<VEC>(a, k) + (VEC ? 0 : j * a.tpr) < p.D;
        xh[k][j] = on ? (xh[k][j] - mean) * rstd : 0.0f;
        if constexpr (ACC) {
          aw[k][j] = __builtin_fmaf(g[k][j], xh[k][j], aw[k][j]);
          ab[k][j] += g[k][j];
        }
        if (p.w) g[k][j] *= w[j];
        t1 += g[k][j];
        t2 = __builtin_fmaf(g[k][j], xh[k][j], t2);
      }
    }
    float t[2] = {t1, t2};
    row_sum(a, t, buf[par]);
    const float m1 = t[0] * p.inv_d, m2 = t[1] * p.inv_d;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int c = col0<VEC>(a, k);
#pragma unroll
      for (int j = 0; j < kVec; ++j) g[k][j] = rstd * (g[k][j] - m1 - xh[k][j] * m2);
      if (p.dsum) {
        float r[kVec];
        load8<Res, VEC>(static_cast<const Res*>(p.dsum) + o, c, a.tpr, p.D, r);
#pragma unroll
        for (int j = 0; j < kVec; ++j) g[k][j] += r[j];
      }
      store8<Res, VEC>(static_cast<Res*>(p.dx) + o, c, a.tpr, p.D, g[k]);
    }
  }
  if constexpr (ACC) {
    // a.row numbers the walkers 0 .. a.row_step - 1: each writes its partial row
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int c = col0<VEC>(a, k);
      store8<float, VEC>(p.pw + a.row * p.D, c, a.tpr, p.D, aw[k]);
      store8<float, VEC>(p.pb + a.row * p.D, c, a.tpr, p.D, ab[k]);
    }
  }
}

// Partial dweight and dbias of a wide row (D > 8192): a block of 256 columns
// walks every nparts-th row.
template <typename In, typename Out>
__global__ __launch_bounds__(256) void norm_wgrad_kernel(NormBwdParams p) {
  const int c = int(blockIdx.x) * 256 + int(threadIdx.x);
  if (c >= p.D) return;
  float aw = 0.0f, ab = 0.0f;
  for (int64_t row = blockIdx.y; row < p.rows; row += gridDim.y) {
    const float g = to_f32(static_cast<const Out*>(p.dy)[row * p.D + c]);
    const float s = to_f32(static_cast<const In*>(p.s)[row * p.xs + c]);
    aw = __builtin_fmaf(g, (s - p.mean[row]) * p.rstd[row], aw);
    ab += g;
  }
  p.pw[int64_t(blockIdx.y) * p.D + c] = aw;
  p.pb[int64_t(blockIdx.y) * p.D + c] = ab;
}

// dweight, dbias from the partial rows: 64 columns per block, 4 waves take every
// fourth partial row each, their sums are added in wave order.
__global__ __launch_bounds__(256) void norm_reduce_kernel(const float* pw, const float* pb,
                                                          float* dw, float* db, int nparts,
                                                          int D) {
  __shared__ float part[4][64];
  const float* src = blockIdx.y == 0 ? pw : pb;
  float* dst = blockIdx.y == 0 ? dw : db;
  if (!dst) return;
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int c = int(blockIdx.x) * 64 + lane;
  float acc = 0.0f;
  if (c < D) {
#pragma unroll 8
    for (int i = wv; i < nparts; i += 4) acc += src[int64_t(i) * D + c];
  }
  part[wv][lane] = acc;
  __syncthreads();
  if (wv == 0 && c < D) dst[c] = (part[0][lane] + part[1][lane]) + (part[2][lane] + part[3][lane]);
}

// waves per row and vectors per thread
void row_shape(int64_t D, int* nwaves, int* vpt) {
  const int64_t vecs = (D + kVec - 1) / kVec;
  *vpt = vecs <= kMaxWaves * kWave ? 1 : 4;
  *nwaves = int((vecs + *vpt * kWave - 1) / (*vpt * kWave));
}

bool vec_ok(const ss_norm_desc_t& d, const void* x) {
  const int64_t xs = d.x_stride ? d.x_stride : d.dim;
  return d.dim % kVec == 0 && xs % kVec == 0 && reinterpret_cast<uintptr_t>(x) % 16 == 0;
}

template <typename In, typename Res, typename Out>
void fwd_types(const NormFwdParams& p, bool vec, int vpt, int threads, int64_t blocks,
               hipStream_t st) {
  const dim3 g{unsigned(blocks)}, b{unsigned(threads)};
  if (vec && vpt == 1) norm_fwd_kernel<In, Res, Out, true, 1><<<g, b, 0, st>>>(p);
  else if (vec) norm_fwd_kernel<In, Res, Out, true, 4><<<g, b, 0, st>>>(p);
  else if (vpt == 1) norm_fwd_kernel<In, Res, Out, false, 1><<<g, b, 0, st>>>(p);
  else norm_fwd_kernel<In, Res, Out, false, 4><<<g, b, 0, st>>>(p);
}

template <typename In, typename Res, typename Out>
void bwd_types(const NormBwdParams& p, bool vec, int vpt, bool acc, int threads, int64_t blocks,
               hipStream_t st) {
  const dim3 g{unsigned(blocks)}, b{unsigned(threads)};
  if (vpt == 1) {
    if (vec && acc) norm_bwd_kernel<In, Res, Out, true, 1, true><<<g, b, 0, st>>>(p);
    else if (vec) norm_bwd_kernel<In, Res, Out, true, 1, false><<<g, b, 0, st>>>(p);
    else if (acc) norm_bwd_kernel<In, Res, Out, false, 1, true><<<g, b, 0, st>>>(p);
    else norm_bwd_kernel<In, Res, Out, false, 1, false><<<g, b, 0, st>>>(p);
  } else if (vec) {
    norm_bwd_kernel<In, Res, Out, true, 4, false><<<g, b, 0, st>>>(p);
  } else {
    norm_bwd_kernel<In, Res, Out, false, 4, false><<<g, b, 0, st>>>(p);
  }
}

// f(In, Res, Out) with the element types of three dtypes
template <typename F>
void by_types(int32_t in, int32_t res, int32_t out, F&& f) {
  auto third = [&](auto a, auto b) {
    if (out == SS_BF16) f(a, b, uint16_t{});
    else f(a, b, float{});
  };
  auto second = [&](auto a) {
    if (res == SS_BF16) third(a, uint16_t{});
    else third(a, float{});
  };
  if (in == SS_BF16) second(uint16_t{});
  else second(float{});
}

}  // namespace

NormPlan plan_norm(const ss_norm_desc_t& d) {
  NormPlan pl;
  row_shape(d.dim, &pl.nwaves, &pl.vpt);
  const int64_t rows_per_block = pl.nwaves == 1 ? 4 : 1;
  const int64_t row_blocks = (d.rows + rows_per_block - 1) / rows_per_block;
  if (pl.vpt == 1) {
    pl.blocks = row_blocks < 1024 ? row_blocks : 1024;
    pl.nparts = int(pl.blocks * rows_per_block);
  } else {
    pl.blocks = row_blocks < 1024 ? row_blocks : 1024;
    pl.nparts = int(d.rows < 64 ? d.rows : 64);
  }
  const size_t part = (size_t(pl.nparts) * size_t(d.dim) * 4 + 255) / 256 * 256;
  pl.off_w = 0;
  pl.off_b = part;
  pl.bytes = 2 * part;
  return pl;
}

int launch_norm_fwd(const ss_norm_desc_t& d, const void* x, const void* residual,
                    const float* weight, const float* bias, void* y, void* sum, float* mean,
                    float* rstd, void* stream) {
  const NormPlan pl = plan_norm(d);
  const int rpb = pl.nwaves == 1 ? 4 : 1;
  NormFwdParams p{x, residual, weight, bias, y, sum, mean, rstd, d.rows,
                  d.x_stride ? d.x_stride : d.dim, int(d.dim), pl.nwaves, d.eps,
                  1.0f / float(d.dim)};
  const int threads = rpb * pl.nwaves * kWave;
  int64_t blocks = (d.rows + rpb - 1) / rpb;
  if (blocks > kMaxRowBlocks) blocks = kMaxRowBlocks;
  by_types(d.in_dtype, d.res_dtype, d.out_dtype, [&](auto a, auto b, auto c) {
    fwd_types<decltype(a), decltype(b), decltype(c)>(p, vec_ok(d, x), pl.vpt, threads, blocks,
                                                     static_cast<hipStream_t>(stream));
  });
  return int(hipGetLastError());
}

int launch_norm_bwd(const ss_norm_desc_t& d, const NormPlan& pl, const void* s,
                    const float* weight, const float* mean, const float* rstd, const void* dy,
                    const void* dsum, void* dx, float* dweight, float* dbias, char* ws,
                    void* stream) {
  hipStream_t st = static_cast<hipStream_t>(stream);
  const int rpb = pl.nwaves == 1 ? 4 : 1;
  const bool grads = dweight || dbias;
  NormBwdParams p{s, weight, mean, rstd, dy, dsum, dx,
                  grads ? reinterpret_cast<float*>(ws + pl.off_w) : nullptr,
                  grads ? reinterpret_cast<float*>(ws + pl.off_b) : nullptr, d.rows,
                  d.x_stride ? d.x_stride : d.dim, int(d.dim), pl.nwaves, 1.0f / float(d.dim)};
  const int threads = rpb * pl.nwaves * kWave;
  const bool acc = grads && pl.vpt == 1;
  by_types(d.in_dtype, d.res_dtype, d.out_dtype, [&](auto a, auto b, auto c) {
    bwd_types<decltype(a), decltype(b), decltype(c)>(p, vec_ok(d, s), pl.vpt, acc, threads,
                                                     pl.blocks, st);
    if (grads && !acc)
      norm_wgrad_kernel<decltype(a), decltype(c)>
          <<<dim3(unsigned((d.dim + 255) / 256), unsigned(pl.nparts)), 256, 0, st>>>(p);
  });
  if (grads)
    norm_reduce_kernel<<<dim3(unsigned((d.dim + 63) / 64), 2), 256, 0, st>>>(
        p.pw, p.pb, dweight, dbias, pl.nparts, int(d.dim));
  return int(hipGetLastError());
}

}  // namespace ss
