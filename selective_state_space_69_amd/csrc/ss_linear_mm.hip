// The linear projections' products for gfx950, on the matrix cores: 256 x 256
// output tiles for large bf16 problems, 128 x 128 for the rest, 64 x 64 for fp32.
//
// 256 x 256.  A workgroup is 8 waves, one workgroup to a CU; a wave owns 128 (s) x 64
// (r) of the tile as 8 x 4 accumulators of v_mfma_f32_16x16x32_bf16 (128 registers).
// A stage is 64 of the contraction: R 256 x 64 and S 256 x 64 bf16, copied from
// global memory straight into LDS (16 bytes per lane), two stages deep.
//
// Schedule.  The waves of a SIMD form two groups that run half a turn apart: while
// one group multiplies, the other reads its next fragments from LDS and issues
// copies, and a barrier swaps the roles.  A stage takes four turns of a read half
// and a multiply half (4 S by 4 R fragments, 16 MFMAs):
//     turn 0: S rows lo, t 0..31     turn 1: S lo, t 32..63
//     turn 2: S rows hi, t 0..31     turn 3: S hi, t 32..63
// R fragments of both t halves stay in registers from turns 0 and 1 on, so R and
// S lo of a buffer are free after turn 1 and are refilled (stage k + 2) in turns 2
// and 3; S hi (stage k + 1) is refilled in turns 0 and 1.  Every copy thus has a
// whole stage of time to land, and a wave waits for the copies of the next two
// turns with the 8 younger ones still in flight.  Stages past the end are issued as
// well, out of the buffer's range (no memory is read), so that the counts hold to
// the last stage.  (Copies issued in the multiply halves instead cost 4%.)
//
// LDS layouts, permuted at the copy's source addresses (its destination is linear)
// so that fragment reads touch all banks evenly (no conflicts by the counters):
//   t contiguous:   128-byte rows of t, 16-byte unit c of row i at c ^ (i & 7);
//                   a fragment is one 16-byte read per lane;
//   t strided:      rows of t hold the operand's 256 (R) or 128 (S half) columns,
//                   32-byte unit u of row t at u ^ f(t), f = t & 3 | (t & 8) / 2;
//                   a fragment is two transposing 8-byte reads per lane
//                   (ds_read_b64_tr_b16: 16 lanes read 4 rows of 16 and each
//                   receives one column).
// SUM2 (backward products, R not exact in bf16): R's values are sums of two bf16, hi =
// bf16(v) and lo = bf16(v - hi), a unit of 8 neighbours' hi followed by the unit of
// their lo.  A stage then holds 32 of the contraction: positions 16 j .. + 7 are hi and
// 16 j + 8 .. + 15 lo of the values 8 j .. + 7, and S's rows of these come twice.  The
// sums are those of R with 16 bits at twice the MFMAs; only the copies' source
// addresses differ.
//
// The transposing reads are written in assembly, with their wait in the same
// block: before the builtin the compiler waits for every copy in flight.
//
// Measured, 16384 rows: 2560 -> 10240 forward 651 us (1320 TFLOP/s; the matrix cores
// are busy 65% of the cycles, at the 1.9 GHz that power allows), dx and dw of 5120
// -> 2560 in fp32 714 us together (1200; 360 and 369 us each alone, dw's 200 tiles on
// 256 CUs).
#include "ss_linear_mm.hpp"

namespace ss {

namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void* lds_ptr;

constexpr int kTile = 256;
template <bool SUM2> constexpr int kStep = SUM2 ? 32 : 64;     // t per stage
constexpr int kThreads = 512;
constexpr unsigned kCUs = 256;
// dx's tiles beside dw's: the workgroups below `behind` take `few` of them each
struct Behind { int32_t behind, few; };
constexpr int kOffR = 0, kOffLo = 65536, kOffHi = 98304, kOffEpi = 131072;
constexpr int kLds = 163840;

#if defined(__HIP_DEVICE_COMPILE__)

template <int N>
__device__ __forceinline__ void wait_copies() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
// End of a turn: this wave's LDS reads have landed, then the barrier.  Nothing
// moves across it.
__device__ __forceinline__ void turn_end() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

__device__ __forceinline__ bf16x8 join8(s16x4 x, s16x4 y) {
  struct P { s16x4 x, y; };
  return __builtin_bit_cast(bf16x8, P{x, y});
}
// Four transposed fragments at LDS addresses a[0..3] (+ OFF; the second half of
// t, four rows on, at + HALF), and their wait.
template <int OFF, int HALF>
__device__ __forceinline__ void read_tr4(const uint32_t (&a)[4], bf16x8 (&f)[4]) {
  s16x4 x0, x1, x2, x3, y0, y1, y2, y3;
  asm volatile(
      "ds_read_b64_tr_b16 %0, %8 offset:%12\n"
      "ds_read_b64_tr_b16 %1, %8 offset:%13\n"
      "ds_read_b64_tr_b16 %2, %9 offset:%12\n"
      "ds_read_b64_tr_b16 %3, %9 offset:%13\n"
      "ds_read_b64_tr_b16 %4, %10 offset:%12\n"
      "ds_read_b64_tr_b16 %5, %10 offset:%13\n"
      "ds_read_b64_tr_b16 %6, %11 offset:%12\n"
      "ds_read_b64_tr_b16 %7, %11 offset:%13\n"
      "s_waitcnt lgkmcnt(0)"
      : "=&v"(x0), "=&v"(y0), "=&v"(x1), "=&v"(y1), "=&v"(x2), "=&v"(y2), "=&v"(x3), "=&v"(y3)
      : "v"(a[0]), "v"(a[1]), "v"(a[2]), "v"(a[3]), "n"(OFF), "n"(OFF + HALF)
      : "memory");
  f[0] = join8(x0, y0);
  f[1] = join8(x1, y1);
  f[2] = join8(x2, y2);
  f[3] = join8(x3, y3);
}
// The same for two sets of four.
template <int OFFA, int HALFA, int OFFB, int HALFB>
__device__ __forceinline__ void read_tr8(const uint32_t (&a)[4], bf16x8 (&fa)[4],
                                         const uint32_t (&b)[4], bf16x8 (&fb)[4]) {
  s16x4 x0, x1, x2, x3, y0, y1, y2, y3, u0, u1, u2, u3, v0, v1, v2, v3;
  asm volatile(
      "ds_read_b64_tr_b16 %0, %16 offset:%24\n"
      "ds_read_b64_tr_b16 %1, %16 offset:%25\n"
      "ds_read_b64_tr_b16 %2, %17 offset:%24\n"
      "ds_read_b64_tr_b16 %3, %17 offset:%25\n"
      "ds_read_b64_tr_b16 %4, %18 offset:%24\n"
      "ds_read_b64_tr_b16 %5, %18 offset:%25\n"
      "ds_read_b64_tr_b16 %6, %19 offset:%24\n"
      "ds_read_b64_tr_b16 %7, %19 offset:%25\n"
      "ds_read_b64_tr_b16 %8, %20 offset:%26\n"
      "ds_read_b64_tr_b16 %9, %20 offset:%27\n"
      "ds_read_b64_tr_b16 %10, %21 offset:%26\n"
      "ds_read_b64_tr_b16 %11, %21 offset:%27\n"
      "ds_read_b64_tr_b16 %12, %22 offset:%26\n"
      "ds_read_b64_tr_b16 %13, %22 offset:%27\n"
      "ds_read_b64_tr_b16 %14, %23 offset:%26\n"
      "ds_read_b64_tr_b16 %15, %23 offset:%27\n"
      "s_waitcnt lgkmcnt(0)"
      : "=&v"(x0), "=&v"(y0), "=&v"(x1), "=&v"(y1), "=&v"(x2), "=&v"(y2), "=&v"(x3), "=&v"(y3),
        "=&v"(u0), "=&v"(v0), "=&v"(u1), "=&v"(v1), "=&v"(u2), "=&v"(v2), "=&v"(u3), "=&v"(v3)
      : "v"(a[0]), "v"(a[1]), "v"(a[2]), "v"(a[3]), "v"(b[0]), "v"(b[1]), "v"(b[2]), "v"(b[3]),
        "n"(OFFA), "n"(OFFA + HALFA), "n"(OFFB), "n"(OFFB + HALFB)
      : "memory");
  fa[0] = join8(x0, y0);
  fa[1] = join8(x1, y1);
  fa[2] = join8(x2, y2);
  fa[3] = join8(x3, y3);
  fb[0] = join8(u0, v0);
  fb[1] = join8(u1, v1);
  fb[2] = join8(u2, v2);
  fb[3] = join8(u3, v3);
}

// Byte offsets of one wave-wide copy instruction (pieces (j waves + wave) 64 + lane of
// the stage, BYTES each: 16-byte units, or their elements) from the tile's origin;
// kOutOfRange outside the operand.  TC: rows of t (128 bytes).  W: columns of the
// stage; HALF: they are columns 0..63 and 128..191 of the tile (an S half).  tpos: the
// piece's first t.  SUM: kPlain, or which operand of sums of two bf16 it is.
enum { kPlain, kSums, kFactors };
template <typename T, bool TC, int W, bool HALF, int SUM, int BYTES = 16>
__device__ __forceinline__ uint32_t copy_offset(int piece, int64_t ld, int64_t i0, int64_t n,
                                                int* tpos) {
  constexpr int E = 16 / int(sizeof(T));
  const int id = piece / (16 / BYTES), e = piece % (16 / BYTES);
  if constexpr (TC) {
    const int q = id / 8, c = (id & 7) ^ (q & 7);
    const int row = HALF ? (q & 63) + (q >> 6) * 128 : q;
    *tpos = (SUM == kPlain ? c : c >> 1) * E + e;
    return i0 + row < n ? uint32_t((row * ld + c * E + e) * int(sizeof(T))) : kOutOfRange;
  } else {
    constexpr int per = W / E;
    const int t = id / per, c1 = id % per;
    int c;
    if constexpr (sizeof(T) == 2) {
      const int f = (t & 3) | (((t >> 3) & 1) << 2);
      c = (((c1 >> 1) ^ f) << 1) | (c1 & 1);
    } else {
      c = c1 ^ (((t >> 2) & 3) << 2);
    }
    const int col = HALF ? (c * E & 63) + (c * E >> 6) * 128 : c * E + e;
    const int at = SUM == kPlain ? t : ((t >> 4) << 3) | (t & 7);
    const int place = SUM == kSums ? 2 * col + (t & 8) : col;
    *tpos = at;
    return i0 + col < n ? uint32_t((at * ld + place) * int(sizeof(T))) : kOutOfRange;
  }
}

// The epilogue of a wave's 16 F-column pieces.  The accumulators (lane: row lane &
// 15, four neighbours of each 16-column piece) are turned through 4 KB of LDS into
// whole rows, 8 columns per lane, 2 F lanes to a row.  Bias is fetched once per
// column, a piece's residual before the stores of the piece in front of it: a wave's
// loads wait for its older stores.  The loop over rows is rolled: unrolled, the
// epilogue outgrew the instruction cache and cost 20 us a tile.
template <int F>
struct Piece {
  static constexpr int kPer = 2 * F;                // lanes of a row
  static constexpr int kRows = 64 / kPer;           // rows of one pass
  static constexpr int kPasses = 16 / kRows;
  int64_t r;      // this lane's row in the first pass
  int32_t s;      // its first column
  int64_t o;      // their element of the output
  Res8 res[kPasses];
  __device__ __forceinline__ void place(const MmParams& p, int64_t r0, int32_t s0) {
    const int lane = threadIdx.x & 63;
    r = r0 + lane / kPer;
    s = s0 + (lane % kPer) * 8;
    o = r * p.nS + s;
  }
  __device__ __forceinline__ void fetch(const MmParams& p, int64_t r0, int32_t s0) {
    place(p, r0, s0);
    if (!p.res) return;
#pragma unroll
    for (int h = 0; h < kPasses; ++h)
      res[h] = fetch_res8(p, o + h * kRows * int64_t(p.nS), r + h * kRows < p.nR && s + 8 <= p.nS);
  }
};
__device__ __forceinline__ void fetch_bias(const MmParams& p, int32_t s, float (&bias)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) bias[j] = 0.0f;
  if (p.bias && s + 8 <= p.nS) load8(p.bias + s, bias);
}

// One piece of 16 rows x 16 F columns.  SPLIT: to a split's partial sums instead;
// STREAM: past the caches; RES: with a residual perhaps.
template <int ACT, bool SPLIT, bool STREAM, bool RES, int F>
__device__ __forceinline__ void piece_out(const MmParams& p, char* sl, const f32x4 (&q)[F],
                                          const Piece<F>& at, const float (&bias)[8], int split) {
  const int lane = threadIdx.x & 63, m = lane & 15, g = lane >> 4;
#pragma unroll
  for (int i = 0; i < F; ++i)
    *reinterpret_cast<f32x4*>(sl + m * 256 + (((4 * i + g) ^ m) << 4)) = q[i];
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  const int u = (lane % Piece<F>::kPer) * 2;
  Res8 res;
  if constexpr (RES) res = at.res[0];
#pragma nounroll
  for (int h = 0; h < Piece<F>::kPasses; ++h) {
    const int row = h * Piece<F>::kRows + lane / Piece<F>::kPer;
    const int64_t r = at.r + h * Piece<F>::kRows, o = at.o + h * Piece<F>::kRows * int64_t(p.nS);
    const int32_t s = at.s;
    if (r < p.nR && s < p.nS) {
      if (s + 8 <= p.nS) {
        const f32x4 x = *reinterpret_cast<const f32x4*>(sl + row * 256 + ((u ^ row) << 4));
        const f32x4 y = *reinterpret_cast<const f32x4*>(sl + row * 256 + (((u + 1) ^ row) << 4));
        float v[8] = {x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
        if constexpr (SPLIT) store8(p.part, split * p.nR * p.nS + o, 0, v);
        else epilogue8<ACT, STREAM, RES>(p, o, v, bias, res);
      } else {
#pragma nounroll
        for (int j = 0; s + j < p.nS; ++j) {
          const float v = *reinterpret_cast<const float*>(
              sl + row * 256 + (((u + j / 4) ^ row) << 4) + (j & 3) * 4);
          if constexpr (SPLIT) store1(p.part, split * p.nR * p.nS + o + j, 0, v);
          else epilogue1(p, ACT, r, s + j, v);
        }
      }
    }
    if constexpr (RES && Piece<F>::kPasses > 1) res = at.res[Piece<F>::kPasses - 1];
  }
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
}

// Which tile of a product a workgroup takes in its round'th turn (false: none is
// left).  A turn's takers are `takers` workgroups, this one the i-th; their tiles
// start at `first` and lie together on an XCD.
__device__ __forceinline__ bool turn_tile(const MmParams& p, int64_t first, int64_t takers,
                                          int64_t i, int64_t* tr, int* ts) {
  const int64_t left = int64_t(p.tiles_r) * p.tiles_s - first;
  const int64_t n = left < takers ? left : takers;
  if (i >= n) return false;
  tile_of(p, uint32_t(first + xcd_contiguous(i, n)), tr, ts);
  return true;
}
// every workgroup takes a tile of every round
struct EveryRound {
  __device__ __forceinline__ bool operator()(const MmParams& p, int64_t round, int64_t* tr,
                                             int* ts) const {
    return turn_tile(p, round * gridDim.x, gridDim.x, blockIdx.x, tr, ts);
  }
};
// the workgroups below `behind` come late and take only `few` tiles each
struct BehindOthers {
  Behind b;
  __device__ __forceinline__ bool operator()(const MmParams& p, int64_t round, int64_t* tr,
                                             int* ts) const {
    const int64_t all = gridDim.x, rest = all - b.behind;
    if (round < b.few) return turn_tile(p, round * all, all, blockIdx.x, tr, ts);
    if (int(blockIdx.x) < b.behind) return false;
    return turn_tile(p, b.few * all + (round - b.few) * rest, rest,
                     blockIdx.x - b.behind, tr, ts);
  }
};

// Kernel parameters, read again where they are used from here on: held in scalar
// registers through the main loop they would crowd it.  AT: where a T is among them.
template <typename T, int AT>
__device__ __forceinline__ T reread_params() {
  constexpr int kWords = int(sizeof(T) / 8);
  static_assert(sizeof(T) % 8 == 0 && AT % 8 == 0, "read in 8-byte words");
  uint64_t a = uint64_t(__builtin_amdgcn_kernarg_segment_ptr()) + AT;
  asm volatile("" : "+s"(a));
  struct Words { uint64_t w[kWords]; } v;
#pragma unroll
  for (int i = 0; i < kWords; ++i)
    v.w[i] = ((const __attribute__((address_space(4))) uint64_t*)a)[i];
  return __builtin_bit_cast(T, v);
}

// AT: where p0 is among the kernel's parameters
template <bool RT, bool ST, int ACT, bool SUM2, int AT, typename Turns>
__device__ __forceinline__ void mm256_body(const MmParams& p0, const Turns& turn, char* lds) {
  const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int m = lane & 15, g = lane >> 4;
  int64_t r0, s0;
  uint32_t vr[4], vlo[2], vhi[2];
  int tpr[4], tps[2];
  const char *pr, *ps, *psh;
  constexpr int kR = SUM2 ? kSums : kPlain, kS = SUM2 ? kFactors : kPlain;
  constexpr int kT = kStep<SUM2>;
  auto place = [&](const MmParams& p, int64_t tr, int ts) {
    r0 = tr * kTile;
    s0 = int64_t(ts) * kTile;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      vr[j] = copy_offset<uint16_t, RT, 256, false, kR>((j * 8 + wv) * 64 + lane, p.ldr, r0, p.nR,
                                                        &tpr[j]);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int id = (j * 8 + wv) * 64 + lane;
      vlo[j] = copy_offset<uint16_t, ST, 128, true, kS>(id, p.lds, s0, p.nS, &tps[j]);
      vhi[j] = copy_offset<uint16_t, ST, 128, true, kS>(id, p.lds, s0 + 64, p.nS, &tps[j]);
    }
    pr = static_cast<const char*>(p.R) + (RT ? r0 * p.ldr : SUM2 ? 2 * r0 : r0) * 2;
    ps = static_cast<const char*>(p.S) + (ST ? s0 * p.lds : s0) * 2;
    psh = ps + (ST ? 64 * p.lds : 64) * 2;
  };
  const int64_t dr = RT ? 128 : p0.ldr * kT * 2;
  const int64_t ds = ST ? 128 : p0.lds * kT * 2;
  const int nk = int((p0.nT + kT - 1) / kT);
  const int rem = int(p0.nT - int64_t(nk - 1) * kT);         // t of the last stage, 1..kT

  // resource of a stage k that starts at base; past the last one no byte is in range
  auto rsrc = [&](const char* base, int k) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(base), short(0),
                                             k < nk ? 0x7fffffff : 0, 0x00020000);
  };
  auto copy = [&](Rsrc src, int dst, uint32_t off) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(src, (lds_ptr)(lds + dst), 16, off, 0, 0, 0);
  };
  // a partial last stage: units past the contraction's end read as zero (the empty
  // asm keeps this a branch, taken once: as selects it cost each stage 12 of them)
  const bool partial = rem < kT;
  auto mask_all = [&](int k) {
    if (partial && k == nk - 1) {
      asm volatile("");
#pragma unroll
      for (int j = 0; j < 4; ++j) vr[j] = tpr[j] < rem ? vr[j] : kOutOfRange;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        vlo[j] = tps[j] < rem ? vlo[j] : kOutOfRange;
        vhi[j] = tps[j] < rem ? vhi[j] : kOutOfRange;
      }
    }
  };
  // pr, ps, psh: where the next stage to copy of R, S lo, S hi starts
  auto copy_r = [&](int k, int j) {
    copy(rsrc(pr, k), kOffR + (k & 1) * 32768 + (j * 8 + wv) * 1024, vr[j]);
  };
  auto copy_lo = [&](int k, int j) {
    copy(rsrc(ps, k), kOffLo + (k & 1) * 16384 + (j * 8 + wv) * 1024, vlo[j]);
  };
  auto copy_hi = [&](int k, int j) {
    copy(rsrc(psh, k), kOffHi + (k & 1) * 16384 + (j * 8 + wv) * 1024, vhi[j]);
  };

  const int wr = (wv >> 1) * 64, wsn = (wv & 1) * 128;      // the wave's corner
  // fragment addresses in buffer 0; the other buffer is a constant away
  uint32_t ar[4], as[4];
  const uint32_t l0 = uint32_t(reinterpret_cast<uintptr_t>((lds_ptr)lds));   // 0: the only array
  const int f = (m >> 2) | ((g & 1) << 2);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // t contiguous: unit g of row (h 4 + g ^ lane & 7), h by XOR of 64 bytes
    ar[i] = l0 + kOffR +
            (RT ? uint32_t((wr + i * 16 + m) * 128 + ((g ^ (lane & 7)) << 4))
                : uint32_t((g * 8 + (m >> 2)) * 512 + (((wr / 16 + i) ^ f) << 5) + (m & 3) * 8));
    as[i] = l0 + kOffLo +
            (ST ? uint32_t((wsn / 2 + i * 16 + m) * 128 + ((g ^ (lane & 7)) << 4))
                : uint32_t((g * 8 + (m >> 2)) * 256 + (((wsn / 32 + i) ^ f) << 5) + (m & 3) * 8));
  }
  auto at = [&](uint32_t a) {
    return *(const __attribute__((address_space(3))) bf16x8*)(uintptr_t(a));
  };

  // the first copies of a tile: stage 0, and R and S lo of stage 1
  auto begin = [&]() {
    mask_all(0);
#pragma unroll
    for (int j = 0; j < 4; ++j) copy_r(0, j);
#pragma unroll
    for (int j = 0; j < 2; ++j) copy_lo(0, j);
#pragma unroll
    for (int j = 0; j < 2; ++j) copy_hi(0, j);
    pr += dr;
    ps += ds;
    psh += ds;
    mask_all(1);
#pragma unroll
    for (int j = 0; j < 4; ++j) copy_r(1, j);
#pragma unroll
    for (int j = 0; j < 2; ++j) copy_lo(1, j);
    pr += dr;
    ps += ds;
  };
  f32x4 acc[8][4];
  bf16x8 b[2][4], a[4];
  auto mma = [&](int i0, int h) {
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        acc[i0 + i][j] =
            __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[i], b[h][j], acc[i0 + i][j], 0, 0, 0);
    __builtin_amdgcn_s_setprio(0);
  };
  // fragments of turn (half of S, t half): the S part, and R's with S lo
  auto read = [&](auto hi_c, auto h_c) {
    constexpr int hi = decltype(hi_c)::value, h = decltype(h_c)::value;
    constexpr int so = hi * (kOffHi - kOffLo) + (ST ? 0 : h * 32 * 256);
    constexpr int ro = RT ? 0 : h * 32 * 512;
    if constexpr (hi == 0 && RT) {
#pragma unroll
      for (int j = 0; j < 4; ++j) b[h][j] = at(ar[j] ^ (h * 64));
    }
    if constexpr (ST) {
#pragma unroll
      for (int i = 0; i < 4; ++i) a[i] = at((as[i] ^ (h * 64)) + so);
    }
    if constexpr (hi == 0 && !RT && !ST) read_tr8<ro, 2048, so, 1024>(ar, b[h], as, a);
    else if constexpr (!ST) read_tr4<so, 1024>(as, a);
    else if constexpr (hi == 0 && !RT) read_tr4<ro, 2048>(ar, b[h]);
  };
  // plain reads are waited for at the end of the half-turn, so copies go after them;
  // the transposing ones wait by themselves
  constexpr bool kReadFirst = ST;
  using I0 = std::integral_constant<int, 0>;
  using I1 = std::integral_constant<int, 1>;

  int64_t tr;
  int ts;
  if (!turn(p0, 0, &tr, &ts)) return;
  place(p0, tr, ts);
  begin();
  for (int64_t round = 0;; ++round) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
    // the tile's first copies, and the last tile's stores
    wait_copies<0>();
    turn_end();
    if (wv >= 4) turn_end();            // the second group runs one turn behind
    for (int k = 0; k < nk; ++k) {
      if (!kReadFirst) copy_hi(k + 1, 0);
      read(I0{}, I0{});
      if (kReadFirst) copy_hi(k + 1, 0);
      turn_end();
      mma(0, 0);
      turn_end();
      if (!kReadFirst) copy_hi(k + 1, 1);
      read(I0{}, I1{});
      if (kReadFirst) copy_hi(k + 1, 1);
      wait_copies<8>();
      turn_end();
      psh += ds;
      mask_all(k + 2);
      mma(0, 1);
      turn_end();
      auto half = [&](int j) {
        copy_r(k + 2, 2 * j);
        copy_r(k + 2, 2 * j + 1);
        copy_lo(k + 2, j);
      };
      if (!kReadFirst) half(0);
      read(I1{}, I0{});
      if (kReadFirst) half(0);
      turn_end();
      mma(4, 0);
      turn_end();
      if (!kReadFirst) half(1);
      read(I1{}, I1{});
      if (kReadFirst) half(1);
      wait_copies<8>();
      turn_end();
      pr += dr;
      ps += ds;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        ar[i] ^= 32768;
        as[i] ^= 16384;
      }
      mma(4, 1);
      turn_end();
    }
    if (wv < 4) turn_end();
    wait_copies<0>();
    if (nk & 1) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {     // back to buffer 0
        ar[i] ^= 32768;
        as[i] ^= 16384;
      }
    }
    // the next tile's first copies run under this one's epilogue
    const MmParams p = reread_params<MmParams, AT>();
    const int64_t r = r0 + wr;
    const int32_t c0 = int32_t(s0) + wsn;
    const bool more = turn(p, round + 1, &tr, &ts);
    if (more) {
      place(p, tr, ts);
      begin();
    }
    Piece<4> now, next;
    float bias[2][8];
    fetch_bias(p, c0 + (lane & 7) * 8, bias[0]);
    fetch_bias(p, c0 + 64 + (lane & 7) * 8, bias[1]);
    now.fetch(p, r, c0);
#pragma unroll
    for (int i = 0; i < 8; ++i) {       // rows 16 (i / 2), columns 64 (i & 1)
      const int j = i / 2, c = i & 1;
      if (i < 7) next.fetch(p, r + 16 * ((i + 1) / 2), c0 + 64 * ((i + 1) & 1));
      const f32x4 q[4] = {acc[4 * c][j], acc[4 * c + 1][j], acc[4 * c + 2][j], acc[4 * c + 3][j]};
      piece_out<ACT, false, true, true>(p, lds + kOffEpi + wv * 4096, q, now, bias[c], 0);
      now = next;
    }
    if (!more) return;
  }
}
#endif

template <bool RT, bool ST, int ACT, bool SUM2>
__global__ __launch_bounds__(kThreads, 2) void mm256_kernel(MmParams p) {
#if defined(__HIP_DEVICE_COMPILE__)
  __shared__ __attribute__((aligned(1024))) char lds[kLds];
  mm256_body<RT, ST, ACT, SUM2, 0>(p, EveryRound{}, lds);
#endif
}

// Both products of a backward pass: dw's tiles, of which the last round does not
// reach every workgroup, then dx's (16384 rows, 5120 -> 2560: 750 us one after the
// other, where dw's 200 tiles leave 56 CUs idle, 708 together; 2560 -> 5120 from a
// checkpoint 757 and 686).
template <bool SUM2>
__global__ __launch_bounds__(kThreads, 2) void mm256_both_kernel(MmParams dw, MmParams, Behind) {
#if defined(__HIP_DEVICE_COMPILE__)
  __shared__ __attribute__((aligned(1024))) char lds[kLds];
  constexpr int kDx = int(sizeof(MmParams)), kTurns = 2 * kDx;
  mm256_body<false, false, SS_ACT_NONE, SUM2, 0>(dw, EveryRound{}, lds);
  const MmParams dx = reread_params<MmParams, kDx>();
  mm256_body<true, false, SS_ACT_NONE, SUM2, kDx>(
      dx, BehindOthers{reread_params<Behind, kTurns>()}, lds);
#endif
}

// Square tiles of 128 (bf16 problems too small to fill the GPU with 256 x 256 ones)
// or 64 (fp32): 4 waves of a quarter tile each, stages of 128 bytes of t (64 bf16,
// 32 fp32) in the same layouts, two buffers, so that two (bf16) or five (fp32)
// workgroups share a CU and hide each other's barriers; the contraction may be
// split.  A lane supplies 16 bytes of t at a time to the MFMAs of either type; the
// four fp32 products (v_mfma_f32_16x16x4_f32) of those number t as 4 g + i on both
// sides.  A t-strided fp32 stage has rows of 64 columns, 64-byte blocks u of row t
// at u ^ (t / 4 & 3), read one element at a time.
constexpr int kSmallThreads = 256;
template <typename T> constexpr int kSmallTile = sizeof(T) == 2 ? 128 : 64;

#if defined(__HIP_DEVICE_COMPILE__)
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
#endif

// G = 2 (bf16): two such groups of 4 waves in a workgroup, each with its own buffers
// and half of the stages, for problems with at most one tile per CU; their sums meet
// in LDS and each group stores half of the tile.
// NB = 1 (bf16): one buffer, so that four workgroups share a CU: while one waits for
// its copies or runs its epilogue the others multiply, which pays where a tile has few
// stages (16384 x 160 x 5120 with softplus: 82 us on 256 x 256 tiles, 64 on these, 85
// with two buffers and two to a CU; 4096 rows: 33, 20 and 25).  Its outputs are streamed
// (4096 rows: 21 -> 20 us).
// RES: with a residual perhaps; without, its registers leave room for a fourth
// workgroup on a CU (the same with softplus 72 us with three and 64 with four, without
// an activation 57 and 51).  All of these are times of a call among 150 in a row, the
// kinds in turn.
// BYTES: of a lane's copy, 16, or 4 for fp32 operands that 16-byte units cannot read
// (odd sizes, odd offsets): four times the instructions, beside fp32 MFMAs that leave
// time for them, but no aligned copy first (3001 x 770 x 1537: 84 us with the copy, 78
// so; 700 x 2561 x 513 34 and 28, its backward 55 and 45).
// lds: kSmallLds<T, NB> bytes per group; block: the work item, a tile of a split.
template <typename T, int NB> constexpr int kSmallLds = 2 * NB * kSmallTile<T> * 128;
#if defined(__HIP_DEVICE_COMPILE__)
template <typename T, bool RT, bool ST, int ACT, int G, int NB, int BYTES, bool RES, bool SUM2>
__device__ __forceinline__ void mm_small_body(const MmParams& p, uint32_t block, char* lds) {
  constexpr int kSz = int(sizeof(T)), kT = 128 / kSz / (SUM2 ? 2 : 1);
  constexpr int kR = SUM2 ? kSums : kPlain, kS = SUM2 ? kFactors : kPlain;
  constexpr int kWide = SUM2 ? 2 : 1;                       // elements per value of R
  constexpr int kTileS = kSmallTile<T>, kF = kTileS / 32;   // fragments of a wave per side
  constexpr int kOp = kTileS * 128;                         // bytes of an operand's stage
  constexpr int kCols = kTileS * kSz;                       // bytes of a t-strided row
  const int tid = threadIdx.x, lane = tid & 63;
  const int wv8 = __builtin_amdgcn_readfirstlane(tid >> 6), wv = wv8 & 3, grp = wv8 >> 2;
  const int m = lane & 15, g = lane >> 4;
  const uint32_t tiles = uint32_t(p.tiles_r) * uint32_t(p.tiles_s);
  const int split = int(block / tiles);
  int64_t tr;
  int ts;
  tile_of(p, uint32_t(xcd_contiguous(block - uint32_t(split) * tiles, tiles)), &tr, &ts);
  const int64_t r0 = tr * kTileS, s0 = int64_t(ts) * kTileS;
  const int64_t t0 = split * p.t_split;
  const int64_t t1 = t0 + p.t_split < p.nT ? t0 + p.t_split : p.nT;
  constexpr int kCopies = kOp / (256 * BYTES);              // of a wave, per operand
  uint32_t vr[kCopies], vs[kCopies];
  int tpr[kCopies], tps[kCopies];
#pragma unroll
  for (int j = 0; j < kCopies; ++j) {
    const int id = (j * 4 + wv) * 64 + lane;
    vr[j] = copy_offset<T, RT, kTileS, false, kR, BYTES>(id, p.ldr, r0, p.nR, &tpr[j]);
    vs[j] = copy_offset<T, ST, kTileS, false, kS, BYTES>(id, p.lds, s0, p.nS, &tps[j]);
  }
  const int64_t dr = RT ? 128 : p.ldr * kT * kSz, ds = ST ? 128 : p.lds * kT * kSz;
  const int stages = int((t1 - t0 + kT - 1) / kT);
  const int rem = int(t1 - t0 - int64_t(stages - 1) * kT);
  // the group's stages: nk of them (the walk's length, for both groups) from k0 on
  const int nk = G == 1 ? stages : (stages + 1) / 2, k0 = grp * nk;
  const char* pr = static_cast<const char*>(p.R) +
                   (RT ? r0 * p.ldr + t0 * kWide : t0 * p.ldr + r0 * kWide) * kSz + k0 * dr;
  const char* ps = static_cast<const char*>(p.S) +
                   (ST ? s0 * p.lds + t0 : t0 * p.lds + s0) * kSz + k0 * ds;
  char* const mine = lds + grp * 4 * kOp;
  auto copy = [&](int k) {
    if (k0 + k == stages - 1 && rem < kT) {
#pragma unroll
      for (int j = 0; j < kCopies; ++j) {
        vr[j] = tpr[j] < rem ? vr[j] : kOutOfRange;
        vs[j] = tps[j] < rem ? vs[j] : kOutOfRange;
      }
    }
    // past the last stage nothing is in range, and the buffer is cleared
    const int range = k0 + k < stages ? 0x7fffffff : 0;
    const Rsrc a = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(range ? pr + k * dr : pr),
                                                     short(0), range, 0x00020000);
    const Rsrc b = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(range ? ps + k * ds : ps),
                                                     short(0), range, 0x00020000);
    char* d = mine + (NB == 2 ? (k & 1) * 2 * kOp : 0) + wv * 64 * BYTES;
#pragma unroll
    for (int j = 0; j < kCopies; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(a, (lds_ptr)(d + j * 256 * BYTES), BYTES, vr[j], 0,
                                               0, 0);
#pragma unroll
    for (int j = 0; j < kCopies; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(b, (lds_ptr)(d + kOp + j * 256 * BYTES), BYTES,
                                               vs[j], 0, 0, 0);
  };
  const int wr = (wv >> 1) * (kTileS / 2), wsn = (wv & 1) * (kTileS / 2);
  // fragment addresses in buffer 0
  uint32_t ar[kF], as[kF];
  const uint32_t l0 = uint32_t(reinterpret_cast<uintptr_t>((lds_ptr)mine));
  const int f = (m >> 2) | ((g & 1) << 2);
  auto address = [&](bool tc, int c0) -> uint32_t {      // c0: first row or column
    if (tc) return uint32_t((c0 + m) * 128 + ((g ^ (lane & 7)) << 4));
    if (kSz == 2) return uint32_t((g * 8 + (m >> 2)) * kCols + (((c0 / 16) ^ f) << 5) + (m & 3) * 8);
    return uint32_t(4 * g * kCols + (((c0 / 16) ^ g) << 6) + m * 4);
  };
#pragma unroll
  for (int i = 0; i < kF; ++i) {
    ar[i] = l0 + address(RT, wr + i * 16);
    as[i] = l0 + kOp + address(ST, wsn + i * 16);
  }
  f32x4 acc[kF][kF];
#pragma unroll
  for (int i = 0; i < kF; ++i)
#pragma unroll
    for (int j = 0; j < kF; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
  // four fragments of half h of the stage's t
  auto read = [&](auto tc_c, auto h_c, const uint32_t (&a)[kF], u32x4 (&d)[kF]) {
    constexpr bool tc = decltype(tc_c)::value;
    constexpr int h = decltype(h_c)::value;
    if constexpr (tc) {
#pragma unroll
      for (int i = 0; i < kF; ++i)
        d[i] = *(const __attribute__((address_space(3))) u32x4*)(uintptr_t(a[i] ^ (h * 64)));
    } else if constexpr (kSz == 2) {
      bf16x8 t[4];
      read_tr4<h * 8192, 1024>(a, t);
#pragma unroll
      for (int i = 0; i < 4; ++i) d[i] = __builtin_bit_cast(u32x4, t[i]);
    } else {
#pragma unroll
      for (int i = 0; i < kF; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          d[i][e] = *(const __attribute__((address_space(3))) uint32_t*)(uintptr_t(
              a[i] + h * 16 * kCols + e * kCols));
    }
  };
  auto part = [&](auto h_c) {
    u32x4 a[kF], b[kF];
    if constexpr (kSz == 2 && !RT && !ST) {
      constexpr int h = decltype(h_c)::value;
      bf16x8 ta[4], tb[4];
      read_tr8<h * 8192, 1024, h * 8192, 1024>(ar, tb, as, ta);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[i] = __builtin_bit_cast(u32x4, ta[i]);
        b[i] = __builtin_bit_cast(u32x4, tb[i]);
      }
    } else {
      read(std::integral_constant<bool, RT>{}, h_c, ar, b);
      read(std::integral_constant<bool, ST>{}, h_c, as, a);
    }
#pragma unroll
    for (int i = 0; i < kF; ++i)
#pragma unroll
      for (int j = 0; j < kF; ++j) acc[i][j] = mma<T>(a[i], b[j], acc[i][j]);
  };
  copy(0);
  for (int k = 0; k < nk; ++k) {
    wait_copies<0>();
    turn_end();       // stage k is whole, and stage k - 1 has been read by every wave
    if (NB == 2 && k + 1 < nk) copy(k + 1);
    part(std::integral_constant<int, 0>{});
    // the second half of the last stage may lie past the contraction's end (fp32 takes
    // it all the same: the branch between its halves costs 89 -> 96 us)
    if (kSz == 4 || k0 + k < stages - 1 || rem > kT / 2) part(std::integral_constant<int, 1>{});
    if constexpr (NB == 2) {
#pragma unroll
      for (int i = 0; i < kF; ++i) {
        ar[i] ^= 2 * kOp;
        as[i] ^= 2 * kOp;
      }
    } else {
      turn_end();
      if (k + 1 < nk) copy(k + 1);
    }
  }
  if (NB == 2) turn_end();
  constexpr int kOut = kF / G;          // rows of pieces this group stores
  f32x4 sum[kF][kOut];
  if constexpr (G == 1) {
#pragma unroll
    for (int i = 0; i < kF; ++i)
#pragma unroll
      for (int j = 0; j < kOut; ++j) sum[i][j] = acc[i][j];
  } else {
    // each group hands the other its half: 256 threads x 16 bytes per accumulator
    f32x4* box = reinterpret_cast<f32x4*>(lds) + (tid & 255);
#pragma unroll
    for (int i = 0; i < kF; ++i)
#pragma unroll
      for (int j = 0; j < kOut; ++j) {
        sum[i][j] = grp == 0 ? acc[i][j] : acc[i][kOut + j];
        box[((grp * kF + i) * kOut + j) * 256] = grp == 0 ? acc[i][kOut + j] : acc[i][j];
      }
    turn_end();
#pragma unroll
    for (int i = 0; i < kF; ++i)
#pragma unroll
      for (int j = 0; j < kOut; ++j) sum[i][j] += box[(((grp ^ 1) * kF + i) * kOut + j) * 256];
  }
  char* const sl = lds + (G == 1 ? 0 : 4 * kOp) + wv8 * 4096;
  const int64_t r = r0 + wr + 16 * kOut * grp;
  const int32_t c = int32_t(s0) + wsn;
  Piece<kF> now, next;
  float bias[8];
  fetch_bias(p, c + (lane % Piece<kF>::kPer) * 8, bias);
  if (RES && p.splits == 1) now.fetch(p, r, c);
  else now.place(p, r, c);
#pragma unroll
  for (int j = 0; j < kOut; ++j) {
    f32x4 q[kF];
#pragma unroll
    for (int i = 0; i < kF; ++i) q[i] = sum[i][j];
    if (p.splits > 1) {
      now.place(p, r + 16 * j, c);
      piece_out<ACT, true, false, true>(p, sl, q, now, bias, split);
    } else {
      if constexpr (RES) {
        if (j + 1 < kOut) next.fetch(p, r + 16 * (j + 1), c);
      } else {
        next.place(p, r + 16 * (j + 1), c);
      }
      piece_out<ACT, false, NB == 1, RES>(p, sl, q, now, bias, 0);
      now = next;
    }
  }
}
#endif

template <typename T, bool RT, bool ST, int ACT, int G, int NB, int BYTES = 16, bool RES = true,
          bool SUM2 = false>
__global__ __launch_bounds__(kSmallThreads * G, NB == 1 ? (RES ? 3 : 4) : 2)
void mm_small_kernel(MmParams p) {
#if defined(__HIP_DEVICE_COMPILE__)
  __shared__ __attribute__((aligned(1024))) char lds[kSmallLds<T, NB> * G];
  mm_small_body<T, RT, ST, ACT, G, NB, BYTES, RES, SUM2>(p, blockIdx.x, lds);
#endif
}

// Both products of a backward pass, dx (R t contiguous) and dw (t strided), side by
// side: each alone would leave half of the CUs' slots empty.
template <typename T, int G, int BYTES = 16, bool SUM2 = false>
__global__ __launch_bounds__(kSmallThreads * G, 2) void mm_both_kernel(MmParams dx, MmParams dw) {
#if defined(__HIP_DEVICE_COMPILE__)
  __shared__ __attribute__((aligned(1024))) char lds[kSmallLds<T, 2> * G];
  const uint32_t items = uint32_t(dw.tiles_r) * uint32_t(dw.tiles_s) * uint32_t(dw.splits);
  if (blockIdx.x < items)
    mm_small_body<T, false, false, SS_ACT_NONE, G, 2, BYTES, false, SUM2>(dw, blockIdx.x, lds);
  else
    mm_small_body<T, true, false, SS_ACT_NONE, G, 2, BYTES, false, SUM2>(dx, blockIdx.x - items,
                                                                         lds);
#endif
}

template <bool RT, bool ST, int ACT, bool SUM2 = false>
void run(const MmParams& p, MmTile tile, hipStream_t stream) {
  const unsigned blocks = unsigned(p.tiles_r) * unsigned(p.tiles_s) * unsigned(p.splits);
  switch (tile) {
    case MmTile::kBig:
      mm256_kernel<RT, ST, ACT, SUM2>
          <<<blocks < kCUs ? blocks : kCUs, kThreads, 0, stream>>>(p);
      break;
    case MmTile::kSmall:
      mm_small_kernel<uint16_t, RT, ST, ACT, 1, 2, 16, true, SUM2>
          <<<blocks, kSmallThreads, 0, stream>>>(p);
      break;
    case MmTile::kSmallSingle:
      if (!p.res)
        mm_small_kernel<uint16_t, RT, ST, ACT, 1, 1, 16, false, SUM2>
            <<<blocks, kSmallThreads, 0, stream>>>(p);
      else if constexpr (RT && ST)
        mm_small_kernel<uint16_t, RT, ST, ACT, 1, 1><<<blocks, kSmallThreads, 0, stream>>>(p);
      break;
    case MmTile::kSmallPair:
      mm_small_kernel<uint16_t, RT, ST, ACT, 2, 2, 16, true, SUM2>
          <<<blocks, 2 * kSmallThreads, 0, stream>>>(p);
      break;
    case MmTile::kSmallF32:
      if constexpr (!SUM2)
        mm_small_kernel<float, RT, ST, ACT, 1, 2><<<blocks, kSmallThreads, 0, stream>>>(p);
      break;
    case MmTile::kSmallF32Any:
      if constexpr (!SUM2)
        mm_small_kernel<float, RT, ST, ACT, 1, 2, 4><<<blocks, kSmallThreads, 0, stream>>>(p);
      break;
  }
}

}  // namespace

void launch_mm_both(const MmParams& dx, const MmParams& dw, MmTile tile, int behind, int few,
                    bool sum2, hipStream_t stream) {
  if (tile == MmTile::kBig) {
    if (sum2) mm256_both_kernel<true><<<kCUs, kThreads, 0, stream>>>(dw, dx, Behind{behind, few});
    else mm256_both_kernel<false><<<kCUs, kThreads, 0, stream>>>(dw, dx, Behind{behind, few});
    return;
  }
  const unsigned blocks = unsigned(dx.tiles_r) * unsigned(dx.tiles_s) * unsigned(dx.splits) +
                          unsigned(dw.tiles_r) * unsigned(dw.tiles_s) * unsigned(dw.splits);
  if (tile == MmTile::kSmallPair && sum2)
    mm_both_kernel<uint16_t, 2, 16, true><<<blocks, 2 * kSmallThreads, 0, stream>>>(dx, dw);
  else if (tile == MmTile::kSmall && sum2)
    mm_both_kernel<uint16_t, 1, 16, true><<<blocks, kSmallThreads, 0, stream>>>(dx, dw);
  else if (tile == MmTile::kSmallPair)
    mm_both_kernel<uint16_t, 2><<<blocks, 2 * kSmallThreads, 0, stream>>>(dx, dw);
  else if (tile == MmTile::kSmall)
    mm_both_kernel<uint16_t, 1><<<blocks, kSmallThreads, 0, stream>>>(dx, dw);
  else if (tile == MmTile::kSmallF32)
    mm_both_kernel<float, 1><<<blocks, kSmallThreads, 0, stream>>>(dx, dw);
  else
    mm_both_kernel<float, 1, 4><<<blocks, kSmallThreads, 0, stream>>>(dx, dw);
}

void launch_mm(const MmParams& p, MmTile tile, bool rt, bool st, bool sum2, hipStream_t stream) {
  if (rt && st) {
    // splits leave the activation to the join
    switch (p.splits > 1 ? int(SS_ACT_NONE) : p.act) {
      case SS_ACT_SILU: return run<true, true, SS_ACT_SILU>(p, tile, stream);
      case SS_ACT_GELU: return run<true, true, SS_ACT_GELU>(p, tile, stream);
      case SS_ACT_SOFTPLUS: return run<true, true, SS_ACT_SOFTPLUS>(p, tile, stream);
      default: return run<true, true, SS_ACT_NONE>(p, tile, stream);
    }
  }
  if (rt && sum2) run<true, false, SS_ACT_NONE, true>(p, tile, stream);
  else if (sum2) run<false, false, SS_ACT_NONE, true>(p, tile, stream);
  else if (rt) run<true, false, SS_ACT_NONE>(p, tile, stream);
  else run<false, false, SS_ACT_NONE>(p, tile, stream);
}

}  // namespace ss
