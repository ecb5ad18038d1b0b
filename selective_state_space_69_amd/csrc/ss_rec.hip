// Gated linear recurrence for gfx950: forward, decode step, plan.
// Layout and accuracy: ss_rec.hpp.
//
// The forward moves each tensor once and is bound by memory.  A workgroup takes 32
// channels of one batch row and walks its time in blocks, the rows of the next two being
// loaded while the present one is computed; one barrier per block joins the waves.  Few
// channels (one long sequence) would leave the GPU empty: their time is cut into chunks,
// whose decays and end states a first pass over the inputs provides; every chunk folds
// those in front of it.
//
// Measured (bf16): 8 x 2048 x 2560 with a gate 121 us, 3.47 TB/s of the least traffic (which
// is what the counters see) against a copy's 5.1; the vector ALU is busy 67% of it.  What holds
// it back is how the rows lie: 335 MB as 7 x 2048 x 2336 take 79 us, as 8 x 2048 x 2048, rows
// 4096 bytes apart, 102.  A batch row's workgroups on one XCD matter most (in plain order 155
// us, when the kernel took 118).  1 x 262144 x 256: 251 us, of them 113 the sums' pass.
#include "ss_rec.hpp"

namespace ss {
namespace {

constexpr int kS = 4;                       // steps of a lane's stretch
constexpr int kWaveSteps = kSubs * kS;
constexpr int kWaves = 8;
constexpr int kBlock = kWaves * kWaveSteps;
// Steps of a lane, waves (bf16 8 x 2048 x 2560 with a gate, us; measured with decays joined as
// fp32 numbers, which takes 3 less than now): 4, 8 117; 4, 4 146; 8, 4 145 (more loads than the
// counter of those in flight holds); 4, 16 139.  Rows 5120 bytes apart are the slow ones of
// these: 8 x 2048 x 2592 takes 110, 107, 112 and 124.
static_assert(SS_REC_CHUNK % kWaveSteps == 0 && kBlock % SS_REC_CHUNK == 0,
              "states are kept at a wave's first step");

struct FwdParams {
  RecShape s;
  const void *x, *r, *i, *z;
  int64_t ldx, ldr, ldi, ldz;
  const float *lam, *h0;
  const uint8_t* starts;
  const int32_t* lengths;
  void* y;
  float *h_last, *states;
  float *clog, *cend;        // (B, nchunks, D) chunks' log decays and end states from a zero start
  float* first;              // SUM: (B, D), h0 as the outputs' pass reads it (h_last may take
                             // its place before every chunk has)
};

// Z: with a gate.  MASK: starts or lengths given.  SUM: only the chunks' carries.
// No branch skips a load or a store: the compiler then knows how many are in flight, and
// waits for the oldest alone.
template <typename T, typename Out, bool Z, bool MASK, bool ANY, bool SUM>
__global__ __launch_bounds__(kWaves * 64, sizeof(T) == 2 && !ANY ? 4 : 2)
void rec_fwd_kernel(FwdParams p) {
#if defined(__HIP_DEVICE_COMPILE__)
  __shared__ float tc[2][kWaves][kRecChans], ts[2][kWaves][kRecChans];
  const Place at(p.s, !SUM && p.s.nchunks > 1);
  const int32_t D = p.s.D;
  const int64_t L = p.s.L, row0 = int64_t(at.b) * L;
  const int64_t t0 = at.chunk * p.s.chunk;
  Masks masks;
  masks.init<MASK>(p.starts, p.lengths, at.b, L, t0, p.s.chunk);
  const int64_t crow = int64_t(at.b * p.s.nchunks + at.chunk) * D + at.c;
  float k[kV], start_state[kV] = {};
  load_f32(p.lam + at.c, at.n, k);
#pragma unroll
  for (int j = 0; j < kV; ++j) k[j] = rec_rate(p.s.decay, k[j]);
  if (!SUM && p.h0) load_f32(p.h0 + int64_t(at.b) * D + at.c, at.n, start_state);
  Carry H[kV];
#pragma unroll
  for (int j = 0; j < kV; ++j) H[j] = Carry{start_state[j], 0.0f};
  [[maybe_unused]] LogSum chunk_log[kV];
  const int off = at.wv * kWaveSteps + at.sub * kS;      // of the lane's stretch in a block
  const int li = at.lane % kRecLanes * kV;

  Stream<ANY> px, pr, pi, pz, py;
  px.init(p.x, p.ldx, sizeof(T), p.s, row0 + t0, off, at);
  pr.init(p.r, p.ldr, sizeof(T), p.s, row0 + t0, off, at);
  pi.init(p.i, p.ldi, sizeof(T), p.s, row0 + t0, off, at);
  if constexpr (Z && !SUM) pz.init(p.z, p.ldz, sizeof(T), p.s, row0 + t0, off, at);
  if constexpr (!SUM) py.init(p.y, D, sizeof(Out), p.s, row0 + t0, off, at);
  // two blocks in turn: each one's rows are loaded as soon as those before are used up
  struct Block { Rows<T, kS, ANY> x, r, i, z; } even, odd;
  auto load = [&](Block& b, int valid) {       // x, r, i
    b.x.load(px, valid);
    b.r.load(pr, valid);
    b.i.load(pi, valid);
    px.move(kBlock);
    pr.move(kBlock);
    pi.move(kBlock);
    __builtin_amdgcn_sched_barrier(0);       // loads stay in the order of their use
  };
  auto load_z = [&](Block& b, int valid) {
    if constexpr (Z && !SUM) {
      b.z.load(pz, valid);
      pz.move(kBlock);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  load(even, masks.len - off);
  load_z(even, masks.len - off);
  load(odd, masks.len - off - kBlock);
  load_z(odd, masks.len - off - kBlock);
  if (!SUM && at.chunk > 0) {
    const int64_t first = int64_t(at.b) * p.s.nchunks * D + at.c;
    fold_chunks<MASK, kWaves>(p.clog + first, p.cend + first, D, at.chunk, at, tc[1], ts[1], H);
  }
  auto run = [&](Block& in_, int tb, int buf) {
    // steps of the lane's stretch inside the chunk; before the length, this time and the next
    const int now = masks.steps - tb - off, live = masks.len - tb - off, next = live - 2 * kBlock;
    auto& x = in_.x;
    auto& r = in_.r;
    auto& i = in_.i;
    auto& z = in_.z;
    bool start[kS] = {};
    if constexpr (MASK) masks.marks(tb + off, start);
    float c[kS][kV], g[kS][kV], l[kV] = {}, s[kV] = {};
    bool cuts = false;
#pragma unroll
    for (int e = 0; e < kS; ++e) {
      float xv[kV], rv[kV], iv[kV];
      unpack(x.q[e], xv);
      unpack(r.q[e], rv);
      unpack(i.q[e], iv);
#pragma unroll
      for (int j = 0; j < kV; ++j) {
        const bool in = e < live;
        float l2 = k[j] * sigmoid(rv[j]);
        l2 = in ? l2 : 0.0f;
        const Decay d = rec_decay(l2);
        const float add = d.beta * sigmoid(iv[j]) * xv[j];
        const bool cut = MASK && start[e] && in;
        c[e][j] = step_decay<MASK>(d.a, cut);
        g[e][j] = in ? add : 0.0f;
        l[j] += l2;
        s[j] = step_apply<MASK>(c[e][j], s[j], g[e][j]);
      }
      if (MASK) cuts |= start[e] && e < live;
    }
    load(in_, next);
    float cx[kV], sx[kV], cw[kV];            // of the stretches in front of the lane's, of the wave
#pragma unroll
    for (int j = 0; j < kV; ++j) {
      float P = step_decay<MASK>(hw_exp2(l[j]), cuts);
      join_up<MASK>(at.sub, P, s[j], cx[j], sx[j]);
      const float lw = wave_log(stretch_log<MASK>(l[j], cuts));
      cw[j] = rec_decay_of<MASK>(lw);
      if constexpr (SUM) chunk_log[j].add(lw);
    }
    if (at.sub == 0) {
      put_lds(&tc[buf][at.wv][li], cw);
      put_lds(&ts[buf][at.wv][li], s);
    }
    __syncthreads();
    if constexpr (Z && !SUM) z.fresh();
    float h[kV] = {};
#pragma unroll 2
    for (int w = 0; w < kWaves; ++w) {
      const Floats cv = get_lds(&tc[buf][w][li]);
      const Floats sv = get_lds(&ts[buf][w][li]);
#pragma unroll
      for (int j = 0; j < kV; ++j) {
        if constexpr (!SUM) h[j] = w == at.wv ? H[j].value() : h[j];
        H[j].apply<MASK>(cv.v[j], sv.v[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < kV; ++j) H[j].settle();
    if constexpr (!SUM) {
      const int tw = tb + at.wv * kWaveSteps;          // the wave's first step
      if (p.states && at.sub == 0 && tw < masks.steps && tw % SS_REC_CHUNK == 0) {
        const int64_t n_states = (L + SS_REC_CHUNK - 1) / SS_REC_CHUNK;
        store_f32(p.states + (at.b * n_states + (t0 + tw) / SS_REC_CHUNK) * D + at.c, at.n, h);
      }
#pragma unroll
      for (int j = 0; j < kV; ++j) h[j] = step_apply<MASK>(cx[j], h[j], sx[j]);
      float out[kS][kV];
#pragma unroll
      for (int e = 0; e < kS; ++e) {
        float zv[kV];
        if constexpr (Z) unpack(z.q[e], zv);
#pragma unroll
        for (int j = 0; j < kV; ++j) {
          h[j] = step_apply<MASK>(c[e][j], h[j], g[e][j]);
          out[e][j] = Z ? h[j] * silu(zv[j]) : h[j];
          if (MASK) out[e][j] = e < live ? out[e][j] : 0.0f;
        }
      }
      load_z(in_, next);
#pragma unroll
      for (int e = 0; e < kS; ++e) put<Out>(py, e, now, at.n, out[e]);
      py.move(kBlock);
    }
  };
  for (int tb = 0; tb < masks.steps; tb += 2 * kBlock) {
    run(even, tb, 0);
    run(odd, tb + kBlock, 1);
  }
  float end[kV], log_decay[kV];
#pragma unroll
  for (int j = 0; j < kV; ++j) end[j] = H[j].base;
  if constexpr (SUM) sum_logs<kWaves>(at, tc[0], chunk_log, log_decay);
  if (at.wv == 0 && at.sub == 0) {
    if constexpr (SUM) {
      if (p.h0 && at.chunk == 0) {
        float first[kV];
        load_f32(p.h0 + int64_t(at.b) * D + at.c, at.n, first);
        store_f32(p.first + int64_t(at.b) * D + at.c, at.n, first);
      }
      store_f32(p.clog + crow, at.n, log_decay);
      store_f32(p.cend + crow, at.n, end);
    } else if (p.h_last && at.chunk == p.s.nchunks - 1) {
      store_f32(p.h_last + int64_t(at.b) * D + at.c, at.n, end);
    }
  }
#endif
}

struct StepParams {
  float* h;
  const void *x, *r, *i, *z;
  int64_t ldx, ldr, ldi, ldz, B;
  const float* lam;
  void* y;
  int32_t D, quads, out_bf16;
  float decay;
};
// One token: V channels per thread, four where all rows' quads are aligned.  A launch bounds
// it: 8 x 2560 bf16 takes 3.1 us.
template <typename T, int V, bool Z>
__global__ __launch_bounds__(64) void rec_step_kernel(StepParams p) {
  const int64_t id = int64_t(blockIdx.x) * 64 + threadIdx.x;
  const int64_t b = id / p.quads;
  if (b >= p.B) return;
  const int32_t c = int32_t(id - b * p.quads) * V;
  float x[V], r[V], i[V], z[V], lam[V], h[V], out[V];
  auto get = [&](const void* src, int64_t ld, float (&v)[V]) {
    const T* q = static_cast<const T*>(src) + b * ld + c;
    if constexpr (V == 4) {
      const float4 f = unpack4(load_raw4(q));
      v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
    } else {
      v[0] = to_f32(*q);
    }
  };
  get(p.x, p.ldx, x);
  get(p.r, p.ldr, r);
  get(p.i, p.ldi, i);
  if constexpr (Z) get(p.z, p.ldz, z);
#pragma unroll
  for (int j = 0; j < V; ++j) {
    lam[j] = p.lam[c + j];
    h[j] = p.h[b * p.D + c + j];
  }
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const Decay d = rec_decay(rec_rate(p.decay, lam[j]) * sigmoid(r[j]));
    // a near 1 enters as a - 1: a long loop of steps does not add up a's rounding
    const float g = d.beta * sigmoid(i[j]) * x[j];
    const float near = h[j] + __builtin_fmaf(d.E, h[j], g), far = __builtin_fmaf(d.a, h[j], g);
    h[j] = d.E > -0.25f ? near : far;
    out[j] = Z ? h[j] * silu(z[j]) : h[j];
    p.h[b * p.D + c + j] = h[j];
  }
#pragma unroll
  for (int j = 0; j < V; ++j) {
    if (p.out_bf16) store_out<uint16_t>(static_cast<uint16_t*>(p.y) + b * p.D + c + j, out[j]);
    else store_out<float>(static_cast<float*>(p.y) + b * p.D + c + j, out[j]);
  }
}

}  // namespace

// Time is cut only where the channels leave the GPU empty: below 256 workgroups in one
// pass, into enough chunks for about 1024, of whole pairs of the pass's blocks.  Sequences
// of up to 4 forward blocks stay whole: the pass over their inputs costs a launch more (1 x
// 512 x 768 forward 14.5 us, 18.6 in two chunks; 1 x 2048 x 2560 35 in four chunks, 28 in
// eight).
RecPlan plan_rec(const ss_rec_desc_t& d, int op) {
  RecPlan pl;
  const int64_t groups = d.batch * ((d.dim + kRecChans - 1) / kRecChans);
  const int64_t blocks = (d.seqlen + kBlock - 1) / kBlock;
  int64_t per = blocks;
  if (groups < 256 && blocks > 4) {
    const int64_t want = (1024 + groups - 1) / groups, least = op == SS_REC_FWD ? 2 : 1;
    per = (blocks + want - 1) / want / least * least;
    if (per < least) per = least;
  }
  pl.chunk = per * kBlock;
  pl.nchunks = (d.seqlen + pl.chunk - 1) / pl.chunk;
  const size_t rows = size_t(d.batch) * size_t(pl.nchunks) * size_t(d.dim) * 4;
  const size_t sz = (rows + kAlign - 1) / kAlign * kAlign;
  if (pl.nchunks > 1) {
    pl.off_log = pl.bytes;
    pl.off_carry = pl.bytes + sz;
    pl.bytes += 2 * sz;
    if (op == SS_REC_FWD) {
      pl.off_first = pl.bytes;
      pl.bytes += (size_t(d.batch) * size_t(d.dim) * 4 + kAlign - 1) / kAlign * kAlign;
    }
  }
  if (op == SS_REC_BWD) {
    pl.off_part = pl.bytes;
    pl.bytes += sz;
  }
  return pl;
}

int launch_rec_fwd(const ss_rec_desc_t& d, const RecPlan& pl, const void* x, const void* r,
                   const void* i, const float* lam, const void* z, const float* h0,
                   const uint8_t* starts, const int32_t* lengths, void* y, float* h_last,
                   float* states, char* ws, void* stream) {
  const FwdParams p{rec_shape(d, pl), x, r, i, z, stride_of(d.x_stride, d.dim),
                    stride_of(d.r_stride, d.dim), stride_of(d.i_stride, d.dim),
                    stride_of(d.z_stride, d.dim), lam, h0, starts, lengths, y, h_last, states,
                    reinterpret_cast<float*>(ws + pl.off_log),
                    reinterpret_cast<float*>(ws + pl.off_carry),
                    reinterpret_cast<float*>(ws + pl.off_first)};
  FwdParams out = p;
  if (h0 && pl.nchunks > 1) out.h0 = p.first;
  const bool any = d.dim % kV != 0 || odd_rows(x, p.ldx, d.in_dtype) ||
                   odd_rows(r, p.ldr, d.in_dtype) || odd_rows(i, p.ldi, d.in_dtype) ||
                   odd_rows(z, p.ldz, d.in_dtype);
  hipStream_t st = static_cast<hipStream_t>(stream);
  const unsigned blocks = unsigned(d.batch * p.s.groups * pl.nchunks);
  rec_by_flags(z != nullptr, starts || lengths, any, [&](auto zc, auto mc, auto ac) {
    constexpr bool Z = decltype(zc)::value, M = decltype(mc)::value, A = decltype(ac)::value;
    auto run = [&](auto type) {
      using T = decltype(type);
      if (pl.nchunks > 1)
        rec_fwd_kernel<T, float, false, M, A, true><<<blocks, kWaves * 64, 0, st>>>(p);
      if (d.out_dtype == SS_BF16)
        rec_fwd_kernel<T, uint16_t, Z, M, A, false><<<blocks, kWaves * 64, 0, st>>>(out);
      else
        rec_fwd_kernel<T, float, Z, M, A, false><<<blocks, kWaves * 64, 0, st>>>(out);
    };
    if (d.in_dtype == SS_BF16) run(uint16_t{});
    else run(float{});
  });
  return int(hipGetLastError());
}

int launch_rec_step(const ss_rec_desc_t& d, float* h, const void* x, const void* r, const void* i,
                    const float* lam, const void* z, void* y, void* stream) {
  StepParams p{h, x, r, i, z, stride_of(d.x_stride, d.dim), stride_of(d.r_stride, d.dim),
               stride_of(d.i_stride, d.dim), stride_of(d.z_stride, d.dim), d.batch, lam, y,
               int32_t(d.dim), 0, d.out_dtype == SS_BF16, d.decay};
  auto whole = [&](const void* q, int64_t ld) {
    return !q || (ld % 4 == 0 && reinterpret_cast<uintptr_t>(q) % 16 == 0);
  };
  const bool four = d.dim % 4 == 0 && whole(x, p.ldx) && whole(r, p.ldr) && whole(i, p.ldi) &&
                    whole(z, p.ldz);
  p.quads = int32_t(four ? d.dim / 4 : d.dim);
  const unsigned blocks = unsigned((d.batch * p.quads + 63) / 64);
  hipStream_t st = static_cast<hipStream_t>(stream);
  auto run = [&](auto type) {
    using T = decltype(type);
    if (four && z) rec_step_kernel<T, 4, true><<<blocks, 64, 0, st>>>(p);
    else if (four) rec_step_kernel<T, 4, false><<<blocks, 64, 0, st>>>(p);
    else if (z) rec_step_kernel<T, 1, true><<<blocks, 64, 0, st>>>(p);
    else rec_step_kernel<T, 1, false><<<blocks, 64, 0, st>>>(p);
  };
  if (d.in_dtype == SS_BF16) run(uint16_t{});
  else run(float{});
  return int(hipGetLastError());
}

}  // namespace ss
