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
// is summed along with it and taken out too (a row of one value gives y = b).  A
// row belongs to the fewest waves that hold it with one vector per thread (D <=
// 8192; four vectors beyond).  Both are bound by memory: at 16384 x 2560 (bf16 x,
// fp32 residual stream) the forward moves 5.2 TB/s (96 us), the backward 5.3 (111
// us, the sums of dw and db included); a large copy reaches 5.1.
#include "ss_device.hpp"

namespace ss {
namespace {

constexpr int kVec = 8;           // channels per thread and vector
constexpr int kMaxWaves = 16;
constexpr int kGroupWaves = 8;    // a block takes several narrow rows, up to so many waves
// dw and db: a thread adds runs of so many rows, then the runs, so that their rounding
// does not grow with the rows (2^19 rows of one value, D = 4096: 1.0e-5 off in one chain
// of 1024 rows, 8.9e-7 so; no slower)
constexpr int kRun = 64;
constexpr int64_t kCUs = 256;
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

// 8 neighbouring channels of a row from column c, in fp32 (0 past D).  Rows need
// only their element's alignment: 16-byte accesses at any element address are
// ordinary ones here.  TAIL: D is not a multiple of 8, and one thread's vector ends
// past the row: it is stored element by element, and loaded as the row's last eight,
// shifted into place where it is widened (element by element the load would have to
// be waited for on the spot, with everything prefetched behind it).
struct __attribute__((packed, aligned(2))) Raw8h { uint32_t w[4]; };
struct __attribute__((packed, aligned(4))) Raw8f { float v[8]; };

template <typename T> struct Raw8;
template <> struct Raw8<uint16_t> { using type = Raw8h; };
template <> struct Raw8<float> { using type = Raw8f; };

// loaded in the storage form, widened where it is used, so that a prefetch does
// not make the wave wait
template <bool TAIL, typename T>
__device__ __forceinline__ typename Raw8<T>::type load_raw8(const T* row, int c, int D) {
  using R = typename Raw8<T>::type;
  R r{};
  if (!TAIL || D >= kVec) {
    const int at = TAIL && c + kVec > D ? D - kVec : c;
    if (c < D) r = *reinterpret_cast<const R*>(row + at);
  } else {
    struct Elems { T e[kVec]; } v;
#pragma unroll
    for (int j = 0; j < kVec; ++j) v.e[j] = c + j < D ? row[c + j] : T(0);
    r = __builtin_bit_cast(R, v);
  }
  return r;
}
__device__ __forceinline__ void widen8(const Raw8h& r, float (&v)[kVec]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(r.w[i] << 16);
    v[2 * i + 1] = __uint_as_float(r.w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void widen8(const Raw8f& r, float (&v)[kVec]) {
#pragma unroll
  for (int j = 0; j < kVec; ++j) v[j] = r.v[j];
}
// the vector at column c, 0 past D
template <bool TAIL, typename R>
__device__ __forceinline__ void widen8(const R& r, int c, int D, float (&v)[kVec]) {
  widen8(r, v);
  if constexpr (TAIL) {
    const int by = D >= kVec && c < D && c + kVec > D ? c + kVec - D : 0;
#pragma unroll
    for (int s = 4; s > 0; s /= 2)
#pragma unroll
      for (int j = 0; j < kVec; ++j) v[j] = by & s ? (j + s < kVec ? v[j + s] : 0.0f) : v[j];
  }
}
template <bool TAIL, typename T>
__device__ __forceinline__ void load8(const T* row, int c, int D, float (&v)[kVec]) {
  widen8<TAIL>(load_raw8<TAIL>(row, c, D), c, D, v);
}

template <bool TAIL, typename T>
__device__ __forceinline__ void store8(T* row, int c, int D, const float (&v)[kVec]) {
  if (c + kVec <= D) {
    if constexpr (sizeof(T) == 2) {
      Raw8h r;
#pragma unroll
      for (int i = 0; i < 4; ++i) r.w[i] = cvt_bf16x2(v[2 * i], v[2 * i + 1]);
      *reinterpret_cast<Raw8h*>(row + c) = r;
    } else {
      Raw8f r;
#pragma unroll
      for (int j = 0; j < kVec; ++j) r.v[j] = v[j];
      *reinterpret_cast<Raw8f*>(row + c) = r;
    }
  } else if (TAIL) {
#pragma unroll
    for (int j = 0; j < kVec; ++j)
      if (c + j < D) store_out<T>(row + c + j, v[j]);
  }
}

// A thread's place in its row: tpr threads per row, vector k of thread t starts
// at column (k tpr + t) 8.
struct Place {
  int tid, tpr, wave, nwaves;
  int sub, groups;    // the block's rows side by side
  int64_t row;        // first row
  int64_t row_step;
};
__device__ __forceinline__ Place place(int nwaves) {
  Place a;
  a.nwaves = nwaves;
  a.tpr = nwaves * kWave;
  a.groups = int(blockDim.x) / a.tpr;
  a.sub = int(threadIdx.x) / a.tpr;
  a.tid = int(threadIdx.x) - a.sub * a.tpr;
  a.wave = a.tid / kWave;
  a.row = int64_t(blockIdx.x) * a.groups + a.sub;
  a.row_step = int64_t(gridDim.x) * a.groups;
  return a;
}
__device__ __forceinline__ int col0(const Place& a, int k) { return (k * a.tpr + a.tid) * kVec; }

// Sums of v[0..N) over a row's threads; every thread gets them.  Every thread of
// the block calls it.  buf: floats that no wave still reads from an earlier use
// (callers alternate).
template <int N>
__device__ __forceinline__ void row_sum(const Place& a, float (&v)[N], float (&buf)[N][kMaxWaves]) {
#pragma unroll
  for (int n = 0; n < N; ++n) v[n] = wave_sum(v[n]);
  if (a.nwaves == 1) return;
  const int w0 = a.sub * a.nwaves;
  if ((threadIdx.x & 63) == 0) {
#pragma unroll
    for (int n = 0; n < N; ++n) buf[n][w0 + a.wave] = v[n];
  }
  __syncthreads();
#pragma unroll
  for (int n = 0; n < N; ++n) v[n] = 0.0f;
  for (int i = 0; i < a.nwaves; ++i)
#pragma unroll
    for (int n = 0; n < N; ++n) v[n] += buf[n][w0 + i];
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

template <typename In, typename Res, typename Out, int VPT, bool TAIL>
__global__ __launch_bounds__(1024) void norm_fwd_kernel(NormFwdParams p) {
  __shared__ float buf1[1][kMaxWaves], buf2[2][kMaxWaves];
  const Place a = place(p.nwaves);
  // the block's groups walk together (row_sum has a barrier); a group past the last
  // row repeats it and stores nothing
  for (int64_t first = a.row - a.sub; first < p.rows; first += a.row_step) {
    const bool live = first + a.sub < p.rows;
    const int64_t row = live ? first + a.sub : p.rows - 1;
    const int64_t o = row * p.D;
    float s[VPT][kVec];
    float t[1] = {0.0f};
#pragma unroll
    for (int k = 0; k < VPT; ++k)
      load8<TAIL>(static_cast<const In*>(p.x) + row * p.xs, col0(a, k), p.D, s[k]);
    if (p.res) {
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        float r[kVec];
        load8<TAIL>(static_cast<const Res*>(p.res) + o, col0(a, k), p.D, r);
#pragma unroll
        for (int j = 0; j < kVec; ++j) s[k][j] += r[j];
      }
    }
#pragma unroll
    for (int k = 0; k < VPT; ++k)
#pragma unroll
      for (int j = 0; j < kVec; ++j) t[0] += s[k][j];
    if (p.sum && live) {
#pragma unroll
      for (int k = 0; k < VPT; ++k)
        store8<TAIL>(static_cast<Res*>(p.sum) + o, col0(a, k), p.D, s[k]);
    }
    row_sum(a, t, buf1);
    const float mean = t[0] * p.inv_d;
    float c[2] = {0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < VPT; ++k)
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        const bool on = col0(a, k) + j < p.D;
        s[k][j] = on ? s[k][j] - mean : 0.0f;
        c[0] += s[k][j];
        c[1] = __builtin_fmaf(s[k][j], s[k][j], c[1]);
      }
    row_sum(a, c, buf2);
    const float rest = c[0] * p.inv_d;
    const float var = __builtin_fmaf(c[1], p.inv_d, -rest * rest);
    // var is never below 0 but for rounding; NaN passes
    const float rstd = 1.0f / __builtin_sqrtf((var < 0.0f ? 0.0f : var) + p.eps);
    if (p.mean && live && a.tid == 0) {
      p.mean[row] = mean + rest;
      p.rstd[row] = rstd;
    }
    if (!live) continue;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int col = col0(a, k);
      float f[kVec];
#pragma unroll
      for (int j = 0; j < kVec; ++j) s[k][j] = (s[k][j] - rest) * rstd;
      if (p.w) {
        load8<TAIL>(p.w, col, p.D, f);
#pragma unroll
        for (int j = 0; j < kVec; ++j) s[k][j] *= f[j];
      }
      if (p.b) {
        load8<TAIL>(p.b, col, p.D, f);
#pragma unroll
        for (int j = 0; j < kVec; ++j) s[k][j] += f[j];
      }
      store8<TAIL>(static_cast<Out*>(p.y) + o, col, p.D, s[k]);
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

// ACC (one vector per thread): also sum dy xh and dy over the block's rows, in
// registers, one partial row per block.
template <typename In, typename Res, typename Out, int VPT, bool TAIL, bool ACC>
__global__ __launch_bounds__(1024) void norm_bwd_kernel(NormBwdParams p) {
  __shared__ float buf[2][2][kMaxWaves];
  __shared__ float acc_buf[ACC ? kGroupWaves * kWave * kVec : 1];
  const Place a = place(p.nwaves);
  // aw, ab: sums of a run of kRun rows; sw, sb: of the runs
  float aw[ACC ? VPT : 1][kVec], ab[ACC ? VPT : 1][kVec];
  float sw[ACC ? VPT : 1][kVec], sb[ACC ? VPT : 1][kVec];
  auto end_run = [&]() {
#pragma unroll
    for (int k = 0; k < VPT; ++k)
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        sw[k][j] += aw[k][j];
        sb[k][j] += ab[k][j];
        aw[k][j] = ab[k][j] = 0.0f;
      }
  };
  int run = 0;
  if constexpr (ACC) {
#pragma unroll
    for (int k = 0; k < VPT; ++k)
#pragma unroll
      for (int j = 0; j < kVec; ++j) aw[k][j] = ab[k][j] = sw[k][j] = sb[k][j] = 0.0f;
  }
  constexpr bool kAhead = VPT == 1;
  // the next row's s, dy and dsum are on their way while this one is summed (with
  // one vector per thread; four would spill)
  typename Raw8<In>::type rs[VPT];
  typename Raw8<Out>::type rg[VPT];
  typename Raw8<Res>::type rd[kAhead ? VPT : 1];
  float rm = 0.0f, rr = 0.0f;
  auto fetch = [&](int64_t row) {
    rm = p.mean[row];
    rr = p.rstd[row];
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int c = col0(a, k);
      rs[k] = load_raw8<TAIL>(static_cast<const In*>(p.s) + row * p.xs, c, p.D);
      rg[k] = load_raw8<TAIL>(static_cast<const Out*>(p.dy) + row * p.D, c, p.D);
      if (kAhead && p.dsum)
        rd[k] = load_raw8<TAIL>(static_cast<const Res*>(p.dsum) + row * p.D, c, p.D);
    }
  };
  auto clear = [&]() {
    rm = rr = 0.0f;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      rs[k] = {};
      rg[k] = {};
      if (kAhead) rd[k] = {};
    }
  };
  if (kAhead && a.row < p.rows) fetch(a.row);
  int par = 0;
  // the block's groups walk together (row_sum has a barrier); a group past the last
  // row carries zeros
  for (int64_t first = a.row - a.sub; first < p.rows; first += a.row_step, par ^= 1) {
    const int64_t row = first + a.sub;
    const bool live = row < p.rows;
    if constexpr (ACC) {
      if (++run > kRun) {
        run = 1;
        end_run();
      }
    }
    if (!live) clear();
    else if (!kAhead) fetch(row);
    float xh[VPT][kVec], g[VPT][kVec], d[kAhead ? VPT : 1][kVec];
    const float mean = rm, rstd = rr;
    float t[2] = {0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int c = col0(a, k);
      widen8<TAIL>(rs[k], c, p.D, xh[k]);
      widen8<TAIL>(rg[k], c, p.D, g[k]);
      if (kAhead && p.dsum) widen8<TAIL>(rd[k], c, p.D, d[k]);
    }
    if (kAhead && row + a.row_step < p.rows) fetch(row + a.row_step);
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      float w[kVec];
      if (p.w) load8<TAIL>(p.w, col0(a, k), p.D, w);
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        const bool on = col0(a, k) + j < p.D;
        xh[k][j] = on ? (xh[k][j] - mean) * rstd : 0.0f;
        if constexpr (ACC) {
          aw[k][j] = __builtin_fmaf(g[k][j], xh[k][j], aw[k][j]);
          ab[k][j] += g[k][j];
        }
        if (p.w) g[k][j] *= w[j];
        t[0] += g[k][j];
        t[1] = __builtin_fmaf(g[k][j], xh[k][j], t[1]);
      }
    }
    row_sum(a, t, buf[par]);
    const float m1 = t[0] * p.inv_d, m2 = t[1] * p.inv_d;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      if (!kAhead && p.dsum && live)
        load8<TAIL>(static_cast<const Res*>(p.dsum) + row * p.D, col0(a, k), p.D, d[0]);
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        g[k][j] = rstd * (g[k][j] - m1 - xh[k][j] * m2);
        if (p.dsum) g[k][j] += d[kAhead ? k : 0][j];
      }
      if (live) store8<TAIL>(static_cast<Res*>(p.dx) + row * p.D, col0(a, k), p.D, g[k]);
    }
  }
  if constexpr (ACC) {
    end_run();
    // the groups' sums are added in group order through LDS: one partial row per block
    if (a.groups > 1) {
      auto add = [&](float (&v)[kVec]) {
        __syncthreads();
        float* mine = acc_buf + (a.sub * a.tpr + a.tid) * kVec;
#pragma unroll
        for (int j = 0; j < kVec; ++j) mine[j] = v[j];
        __syncthreads();
        if (a.sub == 0) {
          for (int i = 1; i < a.groups; ++i)
#pragma unroll
            for (int j = 0; j < kVec; ++j) v[j] += acc_buf[(i * a.tpr + a.tid) * kVec + j];
        }
      };
      add(sw[0]);
      add(sb[0]);
      if (a.sub != 0) return;
    }
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      store8<TAIL>(p.pw + int64_t(blockIdx.x) * p.D, col0(a, k), p.D, sw[k]);
      store8<TAIL>(p.pb + int64_t(blockIdx.x) * p.D, col0(a, k), p.D, sb[k]);
    }
  }
}

// Partial dweight and dbias of a wide row (D > 8192): a block of 256 columns
// walks every nparts-th row.
template <typename In, typename Out>
__global__ __launch_bounds__(256) void norm_wgrad_kernel(NormBwdParams p) {
  const int c = int(blockIdx.x) * 256 + int(threadIdx.x);
  if (c >= p.D) return;
  float aw = 0.0f, ab = 0.0f, sw = 0.0f, sb = 0.0f;
  int run = 0;
  for (int64_t row = blockIdx.y; row < p.rows; row += gridDim.y) {
    if (++run > kRun) {
      run = 1;
      sw += aw;
      sb += ab;
      aw = ab = 0.0f;
    }
    const float g = to_f32(static_cast<const Out*>(p.dy)[row * p.D + c]);
    const float s = to_f32(static_cast<const In*>(p.s)[row * p.xs + c]);
    aw = __builtin_fmaf(g, (s - p.mean[row]) * p.rstd[row], aw);
    ab += g;
  }
  p.pw[int64_t(blockIdx.y) * p.D + c] = sw + aw;
  p.pb[int64_t(blockIdx.y) * p.D + c] = sb + ab;
}

// Column sums of partial rows: 64 columns per block, 16 waves take every 16th row
// each, their sums are added in wave order.  blockIdx.y picks one of two arrays.
constexpr int kSumWaves = 16;
struct SumParams {
  const float* src[2];
  float* dst[2];
  int64_t nparts;
  int32_t N;
};
__global__ __launch_bounds__(kSumWaves * kWave) void column_sum_kernel(SumParams p) {
  __shared__ float part[kSumWaves][64];
  const float* src = p.src[blockIdx.y];
  float* dst = p.dst[blockIdx.y];
  if (!dst) return;
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int c = int(blockIdx.x) * 64 + lane;
  float acc = 0.0f;
  if (c < p.N) {
#pragma unroll 8
    for (int64_t i = wv; i < p.nparts; i += kSumWaves) acc += src[i * p.N + c];
  }
  part[wv][lane] = acc;
  __syncthreads();
  if (wv == 0 && c < p.N) {
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < kSumWaves; ++i) t += part[i][lane];
    dst[c] = t;
  }
}

// waves per row and vectors per thread
void row_shape(int64_t D, int* nwaves, int* vpt) {
  const int64_t vecs = (D + kVec - 1) / kVec;
  *vpt = vecs <= kMaxWaves * kWave ? 1 : 4;
  *nwaves = int((vecs + *vpt * kWave - 1) / (*vpt * kWave));
}
int row_groups(int nwaves) { return nwaves < kGroupWaves ? kGroupWaves / nwaves : 1; }

template <typename In, typename Res, typename Out>
void fwd_types(const NormFwdParams& p, int vpt, int threads, int64_t blocks, hipStream_t st) {
  const dim3 g{unsigned(blocks)}, b{unsigned(threads)};
  const bool tail = p.D % kVec != 0;
  if (vpt == 1 && !tail) norm_fwd_kernel<In, Res, Out, 1, false><<<g, b, 0, st>>>(p);
  else if (vpt == 1) norm_fwd_kernel<In, Res, Out, 1, true><<<g, b, 0, st>>>(p);
  else norm_fwd_kernel<In, Res, Out, 4, true><<<g, b, 0, st>>>(p);
}

template <typename In, typename Res, typename Out>
void bwd_types(const NormBwdParams& p, int vpt, bool acc, int threads, int64_t blocks,
               hipStream_t st) {
  const dim3 g{unsigned(blocks)}, b{unsigned(threads)};
  const bool tail = p.D % kVec != 0;
  if (vpt != 1) norm_bwd_kernel<In, Res, Out, 4, true, false><<<g, b, 0, st>>>(p);
  else if (!acc) norm_bwd_kernel<In, Res, Out, 1, true, false><<<g, b, 0, st>>>(p);
  else if (tail) norm_bwd_kernel<In, Res, Out, 1, true, true><<<g, b, 0, st>>>(p);
  else norm_bwd_kernel<In, Res, Out, 1, false, true><<<g, b, 0, st>>>(p);
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

void launch_column_sums(const float* src0, float* dst0, const float* src1, float* dst1,
                        int64_t nparts, int32_t N, void* stream) {
  const SumParams p{{src0, src1}, {dst0, dst1}, nparts, N};
  column_sum_kernel<<<dim3(unsigned((N + 63) / 64), dst1 ? 2 : 1), kSumWaves * kWave, 0,
                      static_cast<hipStream_t>(stream)>>>(p);
}

NormPlan plan_norm(const ss_norm_desc_t& d) {
  NormPlan pl;
  row_shape(d.dim, &pl.nwaves, &pl.vpt);
  pl.groups = row_groups(pl.nwaves);
  const int64_t row_blocks = (d.rows + pl.groups - 1) / pl.groups;
  // The backward's blocks walk the rows, two to a CU: with the next row prefetched
  // that keeps memory busy, and each block writes one partial row (16384 x 2560: 152
  // us with one block per CU, 115 with two, 137 with three, 141 with four).
  pl.blocks = row_blocks < 2 * kCUs ? row_blocks : 2 * kCUs;
  pl.nparts = int(pl.vpt == 1 ? pl.blocks : (d.rows < 64 ? d.rows : 64));
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
  NormFwdParams p{x, residual, weight, bias, y, sum, mean, rstd, d.rows,
                  d.x_stride ? d.x_stride : d.dim, int(d.dim), pl.nwaves, d.eps,
                  1.0f / float(d.dim)};
  const int threads = pl.groups * pl.nwaves * kWave;
  int64_t blocks = (d.rows + pl.groups - 1) / pl.groups;
  if (blocks > kMaxRowBlocks) blocks = kMaxRowBlocks;
  by_types(d.in_dtype, d.res_dtype, d.out_dtype, [&](auto a, auto b, auto c) {
    fwd_types<decltype(a), decltype(b), decltype(c)>(p, pl.vpt, threads, blocks,
                                                     static_cast<hipStream_t>(stream));
  });
  return int(hipGetLastError());
}

int launch_norm_bwd(const ss_norm_desc_t& d, const NormPlan& pl, const void* s,
                    const float* weight, const float* mean, const float* rstd, const void* dy,
                    const void* dsum, void* dx, float* dweight, float* dbias, char* ws,
                    void* stream) {
  hipStream_t st = static_cast<hipStream_t>(stream);
  const bool grads = dweight || dbias;
  NormBwdParams p{s, weight, mean, rstd, dy, dsum, dx,
                  grads ? reinterpret_cast<float*>(ws + pl.off_w) : nullptr,
                  grads ? reinterpret_cast<float*>(ws + pl.off_b) : nullptr, d.rows,
                  d.x_stride ? d.x_stride : d.dim, int(d.dim), pl.nwaves, 1.0f / float(d.dim)};
  const int threads = pl.groups * pl.nwaves * kWave;
  const bool acc = grads && pl.vpt == 1;
  by_types(d.in_dtype, d.res_dtype, d.out_dtype, [&](auto a, auto b, auto c) {
    bwd_types<decltype(a), decltype(b), decltype(c)>(p, pl.vpt, acc, threads,
                                                     pl.blocks, st);
    if (grads && !acc)
      norm_wgrad_kernel<decltype(a), decltype(c)>
          <<<dim3(unsigned((d.dim + 255) / 256), unsigned(pl.nparts)), 256, 0, st>>>(p);
  });
  if (grads) launch_column_sums(p.pw, dweight, p.pb, dbias, pl.nparts, int32_t(d.dim), stream);
  return int(hipGetLastError());
}

}  // namespace ss
