// Backward of the gated linear recurrence for gfx950.  Layout and chunks are the
// forward's (ss_rec.hpp, ss_rec.hip); time runs backward.
//
// The adjoint that leaves a step, w_t = a_t (v_t + w_(t+1)), is a recurrence of the same
// decays in reverse, and the states are recomputed from the kept one in front of each
// SS_REC_CHUNK steps.  So a stretch is summed up by one decay, an end state and a
// leaving adjoint; both walks are joined by one barrier per block, then every lane runs
// its steps forward (states) and backward (adjoints, gradients) from true values.
//
// Measured (bf16): 8 x 2048 x 2560 with a gate 245 us, 3.1 TB/s; the vector ALU is busy 57% of
// it (114 operations an element), and what else holds is the forward's.
#include "ss_rec.hpp"

namespace ss {
namespace {

constexpr int kS = 4;                       // steps of a lane's stretch
constexpr int kWaveSteps = kSubs * kS;
constexpr int kWaves = 4;
constexpr int kBlock = kWaves * kWaveSteps;
[[maybe_unused]] constexpr int kRun = 16;                  // blocks of a run of dlam's sums
// waves between two kept states
[[maybe_unused]] constexpr int kPerState = SS_REC_CHUNK / kWaveSteps;
static_assert(SS_REC_CHUNK % kWaveSteps == 0 && kBlock % SS_REC_CHUNK == 0,
              "states are kept at a wave's first step");

struct BwdParams {
  RecShape s;
  const void *x, *r, *i, *z, *dy;
  int64_t ldx, ldr, ldi, ldz;
  const float* lam;
  const uint8_t* starts;
  const int32_t* lengths;
  const float *states, *dh_last;
  void *dx, *dr, *di, *dz;
  float* dh0;
  float *clog, *cadj;        // (B, nchunks, D) chunks' log decays and the adjoints that leave them
  float* part;               // (B * nchunks, D) sums of dlam
};

// Two waves to a SIMD: at three the registers do not suffice (bf16 8 x 2048 x 2560 with a gate
// 290 us, 237 so, 245 now; 8 waves of 2 steps 252, 8 of 4 259).
// SUM: only the chunks' carries (decay, and the adjoint that leaves with none
// entering).
template <typename T, typename Dy, bool Z, bool MASK, bool ANY, bool SUM>
__global__ __launch_bounds__(kWaves * 64, 2)
void rec_bwd_kernel(BwdParams p) {
#if defined(__HIP_DEVICE_COMPILE__)
  __shared__ float tc[2][kWaves][kRecChans], ts[2][kWaves][kRecChans], tq[2][kWaves][kRecChans];
  const Place at(p.s, !SUM && p.s.nchunks > 1);
  const int32_t D = p.s.D;
  const int64_t L = p.s.L, row0 = int64_t(at.b) * L;
  const int64_t t0 = at.chunk * p.s.chunk;
  Masks masks;
  masks.init<MASK>(p.starts, p.lengths, at.b, L, t0, p.s.chunk);
  const int64_t crow = int64_t(at.b * p.s.nchunks + at.chunk) * D + at.c;
  const int64_t n_states = (L + SS_REC_CHUNK - 1) / SS_REC_CHUNK;
  float k[kV], entering[kV] = {};
  float run[kV] = {}, sum[kV] = {};     // of dlam: of kRun blocks, of the chunk
  load_f32(p.lam + at.c, at.n, k);
#pragma unroll
  for (int j = 0; j < kV; ++j) k[j] = rec_rate(p.s.decay, k[j]);
  if (!SUM && p.dh_last) load_f32(p.dh_last + int64_t(at.b) * D + at.c, at.n, entering);
  Carry W[kV];
#pragma unroll
  for (int j = 0; j < kV; ++j) W[j] = Carry{entering[j], 0.0f};
  [[maybe_unused]] LogSum chunk_log[kV];
  const int off = at.wv * kWaveSteps + at.sub * kS;      // of the lane's stretch in a block
  const int li = at.lane % kRecLanes * kV;
  int tb = (masks.steps - 1) / kBlock * kBlock;          // the block's first step

  Stream<ANY> px, pr, pi, pz, pd, ox, or_, oi, oz;
  pr.init(p.r, p.ldr, sizeof(T), p.s, row0 + t0 + tb, off, at);
  pd.init(p.dy, D, sizeof(Dy), p.s, row0 + t0 + tb, off, at);
  if constexpr (Z) pz.init(p.z, p.ldz, sizeof(T), p.s, row0 + t0 + tb, off, at);
  if constexpr (!SUM) {
    px.init(p.x, p.ldx, sizeof(T), p.s, row0 + t0 + tb, off, at);
    pi.init(p.i, p.ldi, sizeof(T), p.s, row0 + t0 + tb, off, at);
    ox.init(p.dx, D, sizeof(T), p.s, row0 + t0 + tb, off, at);
    or_.init(p.dr, D, sizeof(T), p.s, row0 + t0 + tb, off, at);
    oi.init(p.di, D, sizeof(T), p.s, row0 + t0 + tb, off, at);
    if constexpr (Z) oz.init(p.dz, D, sizeof(T), p.s, row0 + t0 + tb, off, at);
  }
  // the kept state in front of the wave's steps (its stretch of SS_REC_CHUNK)
  auto state = [&](int tb, float (&st)[kV]) {
    int64_t ks = (t0 + tb + at.wv * kWaveSteps) / SS_REC_CHUNK;
    ks = ks < n_states ? ks : n_states - 1;
    load_f32(p.states + (at.b * n_states + ks) * D + at.c, at.n, st);
  };
  // two blocks in turn: each one's rows are loaded as soon as those before are used up
  struct Block {
    Rows<T, kS, ANY> x, r, i, z;
    Rows<Dy, kS, ANY> dy;
    float st[kV];
  } even, odd;
  auto load_gates = [&](Block& b, int valid) {
    b.r.load(pr, valid);
    pr.move(-kBlock);
    if constexpr (!SUM) {
      b.i.load(pi, valid);
      pi.move(-kBlock);
    }
    __builtin_amdgcn_sched_barrier(0);       // loads stay in the order of their use
  };
  auto load_rest = [&](Block& b, int tb, int valid) {
    b.dy.load(pd, valid);
    pd.move(-kBlock);
    if constexpr (Z) {
      b.z.load(pz, valid);
      pz.move(-kBlock);
    }
    if constexpr (!SUM) {
      b.x.load(px, valid);
      px.move(-kBlock);
      state(tb < 0 ? 0 : tb, b.st);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  // steps of the lane's stretch in front of `end`, of the block from step tb on (a block in
  // front of the chunk's first step is empty)
  auto steps = [&](int end, int tb) { return tb < 0 ? 0 : end - tb - off; };
  load_gates(even, steps(masks.len, tb));
  load_rest(even, tb, steps(masks.len, tb));
  load_gates(odd, steps(masks.len, tb - kBlock));
  load_rest(odd, tb - kBlock, steps(masks.len, tb - kBlock));
  if (!SUM && at.chunk < p.s.nchunks - 1) {       // from the last chunk on
    const int64_t last = (int64_t(at.b + 1) * p.s.nchunks - 1) * D + at.c;
    fold_chunks<MASK, kWaves>(p.clog + last, p.cadj + last, -int64_t(D),
                              p.s.nchunks - 1 - at.chunk, at, tc[1], tq[1], W);
  }
  int turn = 0;
  auto work = [&](Block& in_, int tb, int buf) {
    const int now = steps(masks.steps, tb), live = steps(masks.len, tb);
    const int next = steps(masks.len, tb - 2 * kBlock);
    auto& x = in_.x;
    auto& r = in_.r;
    auto& i = in_.i;
    auto& z = in_.z;
    auto& dy = in_.dy;
    auto& st = in_.st;
    bool start[kS] = {};
    if constexpr (MASK) masks.marks(tb + off, start);
    float c[kS][kV], sr[kS][kV], si[kS][kV], beta[kS][kV], v[kS][kV];
    float l[kV] = {}, s[kV] = {}, q[kV] = {};
    bool cuts = false;
#pragma unroll
    for (int e = 0; e < kS; ++e) {
      __builtin_amdgcn_sched_barrier(0);
      float xv[kV], rv[kV], iv[kV], zv[kV], dv[kV];
      unpack(r.q[e], rv);
      unpack(dy.q[e], dv);
      if constexpr (Z) unpack(z.q[e], zv);
      if constexpr (!SUM) {
        unpack(x.q[e], xv);
        unpack(i.q[e], iv);
      }
      const bool in = e < live, cut = MASK && start[e] && in;
      if (MASK) cuts |= cut;
#pragma unroll
      for (int j = 0; j < kV; ++j) {
        sr[e][j] = sigmoid(rv[j]);
        float l2 = k[j] * sr[e][j];
        l2 = in ? l2 : 0.0f;
        const Decay f = rec_decay(l2);
        c[e][j] = step_decay<MASK>(f.a, cut);
        const float d = Z ? dv[j] * silu(zv[j]) : dv[j];
        v[e][j] = in ? d : 0.0f;
        l[j] += l2;
        if constexpr (!SUM) {
          beta[e][j] = f.beta;
          si[e][j] = sigmoid(iv[j]);
          const float add = f.beta * si[e][j] * xv[j];
          s[j] = step_apply<MASK>(c[e][j], s[j], in ? add : 0.0f);
        }
      }
    }
    load_gates(in_, next);
#pragma unroll
    for (int e = kS - 1; e >= 0; --e)
#pragma unroll
      for (int j = 0; j < kV; ++j) q[j] = step_apply<MASK>(c[e][j], v[e][j] + q[j], 0.0f);
    // of the stretches in front of the lane's, behind it, of the wave
    float cx[kV], sx[kV], cy[kV], qy[kV], cw[kV];
#pragma unroll
    for (int j = 0; j < kV; ++j) {
      float P = step_decay<MASK>(hw_exp2(l[j]), cuts);
      join_both<MASK, !SUM>(at.sub, P, s[j], q[j], cx[j], sx[j], cy[j], qy[j]);
      const float lw = wave_log(stretch_log<MASK>(l[j], cuts));
      cw[j] = rec_decay_of<MASK>(lw);
      if constexpr (SUM) chunk_log[j].add(lw);
    }
    if (at.sub == 0) {
      put_lds(&tc[buf][at.wv][li], cw);
      put_lds(&tq[buf][at.wv][li], q);
      if constexpr (!SUM)
        put_lds(&ts[buf][at.wv][li], s);
    }
    __syncthreads();
    if constexpr (!SUM) {
      x.fresh();
      dy.fresh();
      if constexpr (Z) z.fresh();
    }
    float w[kV] = {}, h[kV];
#pragma unroll
    for (int j = 0; j < kV; ++j) h[j] = st[j];
#pragma unroll 2
    for (int o = kWaves - 1; o >= 0; --o) {
      const Floats cv = get_lds(&tc[buf][o][li]);
      const Floats qv = get_lds(&tq[buf][o][li]);
#pragma unroll
      for (int j = 0; j < kV; ++j) {
        if constexpr (!SUM) w[j] = o == at.wv ? W[j].value() : w[j];
        W[j].apply<MASK>(cv.v[j], qv.v[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < kV; ++j) W[j].settle();
    if constexpr (!SUM) {
      // the waves between the kept state and this one
      for (int o = at.wv / kPerState * kPerState; o < at.wv; ++o) {
        const Floats cv = get_lds(&tc[buf][o][li]);
        const Floats sv = get_lds(&ts[buf][o][li]);
#pragma unroll
        for (int j = 0; j < kV; ++j) h[j] = rec_apply<MASK>(cv.v[j], h[j], sv.v[j]);
      }
      float hs[kS + 1][kV];       // the state in front of each step, behind the last
#pragma unroll
      for (int j = 0; j < kV; ++j) {
        hs[0][j] = step_apply<MASK>(cx[j], h[j], sx[j]);
        w[j] = step_apply<MASK>(cy[j], w[j], qy[j]);
      }
#pragma unroll
      for (int e = 0; e < kS; ++e) {
        float xv[kV];
        unpack(x.q[e], xv);
#pragma unroll
        for (int j = 0; j < kV; ++j) {
          const float add = beta[e][j] * si[e][j] * xv[j];
          hs[e + 1][j] = step_apply<MASK>(c[e][j], hs[e][j], e < live ? add : 0.0f);
        }
      }
#pragma unroll
      for (int e = kS - 1; e >= 0; --e) {
        __builtin_amdgcn_sched_barrier(0);
        float xv[kV], zv[kV], dv[kV], gx[kV], gr[kV], gi[kV], gz[kV];
        unpack(x.q[e], xv);
        if constexpr (Z) {
          unpack(z.q[e], zv);
          unpack(dy.q[e], dv);
        }
        const bool in = e < live;
#pragma unroll
        for (int j = 0; j < kV; ++j) {
          const float u = v[e][j] + w[j], bt = beta[e][j], l2 = k[j] * sr[e][j], la = l2 * kLn2;
          w[j] = step_apply<MASK>(c[e][j], u, 0.0f);
          // log a / sqrt(1 - a^2): 0 where log a underflows to 0
          const float ratio = la * hw_rcp(bt), lb = bt > 0.0f ? ratio : 0.0f;
          const float ah = step_apply<MASK>(c[e][j], hs[e][j], 0.0f) * la;
          // a^2 with its relative accuracy, which 1 - (1 - a^2) loses where a is small (a = e^-16:
          // dr 1.4e-5 off); a start's own a is not in c
          const float aa = MASK && c[e][j] == 0.0f ? hw_exp2(2.0f * l2) : c[e][j] * c[e][j];
          const float dl = u * (ah - aa * lb * (si[e][j] * xv[j]));
          const float vx = u * bt * si[e][j], vi = vx * xv[j] * (1.0f - si[e][j]);
          const float vr = dl * (1.0f - sr[e][j]);         // dl: of log a, times log a
          gx[j] = in ? vx : 0.0f;
          gi[j] = in ? vi : 0.0f;
          gr[j] = in ? vr : 0.0f;
          run[j] += in ? dl : 0.0f;
          if constexpr (Z) {
            const float sz = sigmoid(zv[j]);
            const float vz = dv[j] * hs[e + 1][j] * sz * __builtin_fmaf(zv[j], 1.0f - sz, 1.0f);
            gz[j] = in ? vz : 0.0f;
          }
        }
        put<T>(ox, e, now, at.n, gx);
        put<T>(or_, e, now, at.n, gr);
        put<T>(oi, e, now, at.n, gi);
        if constexpr (Z) put<T>(oz, e, now, at.n, gz);
      }
      ox.move(-kBlock);
      or_.move(-kBlock);
      oi.move(-kBlock);
      if constexpr (Z) oz.move(-kBlock);
      if (++turn == kRun || tb <= 0) {
        turn = 0;
#pragma unroll
        for (int j = 0; j < kV; ++j) {
          sum[j] += run[j];
          run[j] = 0.0f;
        }
      }
    }
    load_rest(in_, tb - 2 * kBlock, next);
  };
  for (; tb >= 0; tb -= 2 * kBlock) {
    work(even, tb, 0);
    work(odd, tb - kBlock, 1);
  }
  float leaving[kV];
#pragma unroll
  for (int j = 0; j < kV; ++j) leaving[j] = W[j].base;
  if constexpr (SUM) {
    float log_decay[kV];
    sum_logs<kWaves>(at, tc[0], chunk_log, log_decay);
    if (at.wv == 0 && at.sub == 0) {
      store_f32(p.clog + crow, at.n, log_decay);
      store_f32(p.cadj + crow, at.n, leaving);
    }
  } else {
    // dlam: the workgroup's stretches, in order
    __syncthreads();
    float* const box = &tc[0][0][0];
#pragma unroll
    for (int pass = 0; pass < kSubs; ++pass) {
      if (at.sub == pass) {
#pragma unroll
        for (int j = 0; j < kV; ++j) {
          float* d = box + at.wv * kRecChans + li + j;
          *d = pass > 0 ? *d + sum[j] : sum[j];
        }
      }
      __syncthreads();
    }
    if (at.wv == 0 && at.sub == 0) {
      // d log a / d lam = log a sigmoid(lam) / softplus(lam); the ratio is 1 far below 0
      float tot[kV], lam[kV];
      load_f32(p.lam + at.c, at.n, lam);
#pragma unroll
      for (int j = 0; j < kV; ++j) {
        tot[j] = 0.0f;
#pragma unroll
        for (int o = 0; o < kWaves; ++o) tot[j] += box[o * kRecChans + li + j];
        const float sp = softplus_log2(lam[j] * kLog2e) * kLn2, ratio = sigmoid(lam[j]) / sp;
        tot[j] *= sp > 0.0f ? ratio : 1.0f;
      }
      store_f32(p.part + crow, at.n, tot);
      if (p.dh0 && at.chunk == 0) store_f32(p.dh0 + int64_t(at.b) * D + at.c, at.n, leaving);
    }
  }
#endif
}

}  // namespace

int launch_rec_bwd(const ss_rec_desc_t& d, const RecPlan& pl, const void* x, const void* r,
                   const void* i, const float* lam, const void* z, const uint8_t* starts,
                   const int32_t* lengths, const float* states, const void* dy,
                   const float* dh_last, void* dx, void* dr, void* di, void* dz, float* dlam,
                   float* dh0, char* ws, void* stream) {
  const BwdParams p{rec_shape(d, pl), x, r, i, z, dy, stride_of(d.x_stride, d.dim),
                    stride_of(d.r_stride, d.dim), stride_of(d.i_stride, d.dim),
                    stride_of(d.z_stride, d.dim), lam, starts, lengths, states, dh_last, dx, dr,
                    di, dz, dh0, reinterpret_cast<float*>(ws + pl.off_log),
                    reinterpret_cast<float*>(ws + pl.off_carry),
                    reinterpret_cast<float*>(ws + pl.off_part)};
  const bool any = d.dim % kV != 0 || odd_rows(x, p.ldx, d.in_dtype) ||
                   odd_rows(r, p.ldr, d.in_dtype) || odd_rows(i, p.ldi, d.in_dtype) ||
                   odd_rows(z, p.ldz, d.in_dtype);
  hipStream_t st = static_cast<hipStream_t>(stream);
  const unsigned blocks = unsigned(d.batch * p.s.groups * pl.nchunks);
  const bool xb = d.in_dtype == SS_BF16, yb = d.out_dtype == SS_BF16;
  rec_by_flags(z != nullptr, starts || lengths, any, [&](auto zc, auto mc, auto ac) {
    constexpr bool Z = decltype(zc)::value, M = decltype(mc)::value, A = decltype(ac)::value;
    auto run = [&](auto type, auto dtype) {
      using T = decltype(type);
      using Dy = decltype(dtype);
      if (pl.nchunks > 1)
        rec_bwd_kernel<T, Dy, Z, M, A, true><<<blocks, kWaves * 64, 0, st>>>(p);
      rec_bwd_kernel<T, Dy, Z, M, A, false><<<blocks, kWaves * 64, 0, st>>>(p);
    };
    if (xb && yb) run(uint16_t{}, uint16_t{});
    else if (xb) run(uint16_t{}, float{});
    else if (yb) run(float{}, uint16_t{});
    else run(float{}, float{});
  });
  launch_column_sums(p.part, dlam, nullptr, nullptr, d.batch * pl.nchunks, int32_t(d.dim), stream);
  return int(hipGetLastError());
}

}  // namespace ss
