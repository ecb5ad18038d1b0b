// The linear projections' products for gfx950, on the matrix cores: 256 x 256
// output tiles for large bf16 problems, 128 x 128 for the rest, 64 x 64 for fp32.
// Kernel templates, instantiated by ss_linear_mm.hip (plain products), ss_glu_mm.hip
// (two products gated by each other) and ss_q8_mm.hip (8-bit integers).
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
// Two gated products (GLU): O = act(R S^T) (R S'^T), S' the rows nS and on of S's
// storage.  A tile's S columns are half of S and half of S', so that a wave has both
// factors of its outputs in its own accumulators: 256 x 256 tiles take S' as the hi
// halves, the small ones every other quarter.
//
// 8-bit integers: v_mfma_i32_16x16x64_i8 reads 16 bytes of t per lane as the bf16 one
// does, so layouts and schedule are the same at twice the contraction per stage.  Sums
// are exact; the epilogue multiplies them by the row's and the column's scale.
//
// The transposing reads are written in assembly, with their wait in the same
// block: before the builtin the compiler waits for every copy in flight.
//
// Measured, 16384 rows: 2560 -> 10240 forward 651 us (1320 TFLOP/s; the matrix cores
// are busy 65% of the cycles, at the 1.9 GHz that power allows), dx and dw of 5120
// -> 2560 in fp32 714 us together (1200; 360 and 369 us each alone, dw's 200 tiles on
// 256 CUs).  Gated, 2560 -> 2 x 6912 with SiLU: 930 us (1250 TFLOP/s; the matrix cores busy
// 60%); 8-bit integers, 2560 -> 10240: 385 to 405 us (2.2 POP/s, 50%).
#pragma once

#include "ss_linear_mm.hpp"

namespace ss {

namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void* lds_ptr;

template <int KIND> struct KindOf { using Elem = uint16_t; using Acc = f32x4; };
template <> struct KindOf<kInt8> { using Elem = uint8_t; using Acc = i32x4; };

constexpr int kTile = 256;
template <bool SUM2, int KIND> constexpr int kStep = SUM2 ? 32 : KIND == kInt8 ? 128 : 64;   // t per stage
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
// stage; HALF: they are columns 0..63 and 128..191 of the tile (an S half); Q: columns
// of two operands in turn, Q of each.  tpos: the
// piece's first t.  SUM: kPlain, or which operand of sums of two bf16 it is.
enum { kPlain, kSums, kFactors };
template <typename T, bool TC, int W, bool HALF, int SUM, int BYTES = 16, int Q = 0>
__device__ __forceinline__ uint32_t copy_offset(int piece, int64_t ld, int64_t i0, int64_t n,
                                                int* tpos) {
  constexpr int E = 16 / int(sizeof(T));
  const int id = piece / (16 / BYTES), e = piece % (16 / BYTES);
  if constexpr (TC) {
    const int q = id / 8, c = (id & 7) ^ (q & 7);
    constexpr int kQ = Q ? Q : W;
    const int row = HALF ? (q & 63) + (q >> 6) * 128 : q / (2 * kQ) * kQ + q % kQ;
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
// epilogue outgrew the instruction cache and cost 20 us a tile.  kInt8 also fetches the
// rows' scales and the elements of a row's end ahead (3001 x 256 -> 773: 14.2 -> 9.5 us,
// with a residual 20.2 -> 15.6; 16384 x 2560 -> 10240 with one 488 -> 467).
// the columns in front of n of the eight from s on
__device__ __forceinline__ void load_to(const float* base, int32_t s, int32_t n, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (s + j < n) v[j] = load1(base, s + j, 0);
}
template <int F, int KIND = kMm>
struct Piece {
  static constexpr int kPer = 2 * F;                // lanes of a row
  static constexpr int kRows = 64 / kPer;           // rows of one pass
  static constexpr int kPasses = 16 / kRows;
  int64_t r;      // this lane's row in the first pass
  int32_t s;      // its first column
  int64_t o;      // their element of the output
  Res8 res[kPasses];
  float scale[kPasses];      // kInt8: the rows'
  __device__ __forceinline__ void place(const MmParams& p, int64_t r0, int32_t s0) {
    const int lane = threadIdx.x & 63;
    r = r0 + lane / kPer;
    s = s0 + (lane % kPer) * 8;
    o = r * p.nS + s;
    if constexpr (KIND == kInt8) {
#pragma unroll
      for (int h = 0; h < kPasses; ++h)
        if (r + h * kRows < p.nR) scale[h] = load1(p.row_scale, r + h * kRows, 0);
    }
  }
  __device__ __forceinline__ void fetch(const MmParams& p, int64_t r0, int32_t s0) {
    place(p, r0, s0);
    if (!p.res) return;
#pragma unroll
    for (int h = 0; h < kPasses; ++h) {
      res[h] = fetch_res8(p, o + h * kRows * int64_t(p.nS), r + h * kRows < p.nR && s + 8 <= p.nS);
      if (KIND == kInt8 && r + h * kRows < p.nR && s + 8 > p.nS) {      // a row's end: as fp32
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (s + j < p.nS)
            res[h].w[j] =
                __float_as_uint(load1(p.res, o + h * kRows * int64_t(p.nS) + j, p.res_bf16));
      }
    }
  }
};
template <int KIND>
__device__ __forceinline__ void fetch_bias(const MmParams& p, int32_t s, float (&bias)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) bias[j] = 0.0f;
  if (p.bias && s + 8 <= p.nS) load8(p.bias + s, bias);
  else if (KIND == kInt8 && p.bias) load_to(p.bias, s, p.nS, bias);
}

// One piece of 16 rows x 16 F columns.  SPLIT: to a split's partial sums instead;
// STREAM: past the caches; RES: with a residual perhaps.  kInt8: the sums are whole
// numbers, scale those of this lane's columns.
template <int ACT, bool SPLIT, bool STREAM, bool RES, int KIND, int F, typename Acc>
__device__ __forceinline__ void piece_out(const MmParams& p, char* sl, const Acc (&q)[F],
                                          const Piece<F, KIND>& at, const float (&bias)[8],
                                          const float (&scale)[8], int split) {
  const int lane = threadIdx.x & 63, m = lane & 15, g = lane >> 4;
#pragma unroll
  for (int i = 0; i < F; ++i)
    *reinterpret_cast<Acc*>(sl + m * 256 + (((4 * i + g) ^ m) << 4)) = q[i];
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  const int u = (lane % Piece<F>::kPer) * 2;
  Res8 res;
  if constexpr (RES) res = at.res[0];
  float rs = 1.0f;
  if constexpr (KIND == kInt8) rs = at.scale[0];
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
        if constexpr (SPLIT) {
          store8(p.part, split * p.nR * p.nS + o, 0, v);
        } else {
          if constexpr (KIND == kInt8) {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = scaled(__float_as_int(v[j]), RowScale(rs), scale[j]);
          }
          epilogue8<ACT, STREAM, RES>(p, o, v, bias, res);
        }
      } else if constexpr (KIND == kInt8 && !SPLIT) {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          v[j] = *reinterpret_cast<const float*>(sl + row * 256 + (((u + j / 4) ^ row) << 4) +
                                                 (j & 3) * 4);
          v[j] = apply_act(ACT, scaled(__float_as_int(v[j]), RowScale(rs), scale[j]) + bias[j]);
          if (RES && p.res) v[j] += __uint_as_float(res.w[j]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (s + j < p.nS) store1(p.out, o + j, p.out_bf16, v[j]);
      } else {
#pragma nounroll
        for (int j = 0; s + j < p.nS; ++j) {
          float v = *reinterpret_cast<const float*>(
              sl + row * 256 + (((u + j / 4) ^ row) << 4) + (j & 3) * 4);
          if constexpr (SPLIT) store1(p.part, split * p.nR * p.nS + o + j, 0, v);
          else epilogue1(p, ACT, r, s + j, v);
        }
      }
    }
    if constexpr (RES && Piece<F>::kPasses > 1) res = at.res[Piece<F>::kPasses - 1];
    if constexpr (KIND == kInt8 && Piece<F>::kPasses > 1) rs = at.scale[Piece<F>::kPasses - 1];
  }
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
}
// the scales of this lane's eight columns
template <int KIND>
__device__ __forceinline__ void fetch_scale(const MmParams& p, int32_t s, float (&scale)[8]) {
  if constexpr (KIND == kInt8) {
#pragma unroll
    for (int j = 0; j < 8; ++j) scale[j] = 0.0f;
    if (s + 8 <= p.nS) load8(p.col_scale + s, scale);
    else load_to(p.col_scale, s, p.nS, scale);
  }
}

// A piece of 16 rows x 16 F columns at (r0, s0) of an (nR, nS) array with rows of ld
// elements, as it is: turned through LDS into whole rows; one fragment's four neighbours
// per lane are stored from where they are.
template <int F, bool STREAM>
__device__ __forceinline__ void turn_store(void* base, int64_t ld, int bf16, char* sl,
                                           const f32x4 (&q)[F], int64_t r0, int32_t s0, int64_t nR,
                                           int32_t nS) {
  const int lane = threadIdx.x & 63, m = lane & 15, g = lane >> 4;
  if constexpr (F == 1) {
    const int64_t r = r0 + m;
    const int32_t s = s0 + 4 * g;
    if (r < nR) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (s + j < nS) store1(base, r * ld + s + j, bf16, q[0][j]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < F; ++i)
      *reinterpret_cast<f32x4*>(sl + m * 256 + (((4 * i + g) ^ m) << 4)) = q[i];
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    constexpr int kPer = 2 * F, kRows = 64 / kPer;
    const int u = (lane % kPer) * 2;
    const int32_t s = s0 + (lane % kPer) * 8;
#pragma nounroll
    for (int h = 0; h < 16 / kRows; ++h) {
      const int row = h * kRows + lane / kPer;
      const int64_t r = r0 + row, o = r * ld + s;
      if (r < nR && s < nS) {
        if (s + 8 <= nS) {
          const f32x4 x = *reinterpret_cast<const f32x4*>(sl + row * 256 + ((u ^ row) << 4));
          const f32x4 y = *reinterpret_cast<const f32x4*>(sl + row * 256 + (((u + 1) ^ row) << 4));
          const float v[8] = {x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
          store8<STREAM>(base, o, bf16, v);
        } else {
#pragma nounroll
          for (int j = 0; s + j < nS; ++j)
            store1(base, o + j, bf16, *reinterpret_cast<const float*>(
                sl + row * 256 + (((u + j / 4) ^ row) << 4) + (j & 3) * 4));
        }
      }
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  }
}
// The gated epilogue of such a piece: both factors (gate, up), their sums kept where
// asked for, their product.  SPLIT: both to a split's partial sums, (nR, 2 nS).
template <int ACT, bool SPLIT, bool STREAM, int F>
__device__ __forceinline__ void glu_out(const MmParams& p, char* sl, f32x4 (&gate)[F],
                                        f32x4 (&up)[F], int64_t r, int32_t s, int split) {
  const int64_t ld = 2 * int64_t(p.nS);
  if constexpr (SPLIT) {
    float* part = p.part + split * p.nR * ld;
    turn_store<F, false>(part, ld, 0, sl, gate, r, s, p.nR, p.nS);
    turn_store<F, false>(part + p.nS, ld, 0, sl, up, r, s, p.nR, p.nS);
  } else {
    if (p.bias) {
      const int32_t c0 = s + 4 * ((threadIdx.x & 63) >> 4);
#pragma unroll
      for (int i = 0; i < F; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int32_t c = c0 + 16 * i + j < p.nS ? c0 + 16 * i + j : p.nS - 1;
          gate[i][j] += load1(p.bias, c, 0);
          up[i][j] += load1(p.bias, p.nS + c, 0);
        }
    }
    if (p.pre) {
      turn_store<F, STREAM>(p.pre, ld, p.pre_bf16, sl, gate, r, s, p.nR, p.nS);
      char* second = static_cast<char*>(p.pre) + int64_t(p.nS) * (p.pre_bf16 ? 2 : 4);
      turn_store<F, STREAM>(second, ld, p.pre_bf16, sl, up, r, s, p.nR, p.nS);
    }
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) up[i][j] *= apply_act(ACT, gate[i][j]);
    turn_store<F, STREAM>(p.out, p.nS, p.out_bf16, sl, up, r, s, p.nR, p.nS);
  }
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
template <bool RT, bool ST, int ACT, bool SUM2, int AT, int KIND, typename Turns>
__device__ __forceinline__ void mm256_body(const MmParams& p0, const Turns& turn, char* lds) {
  using Elem = typename KindOf<KIND>::Elem;
  using Acc = typename KindOf<KIND>::Acc;
  constexpr int kSz = int(sizeof(Elem));
  const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int m = lane & 15, g = lane >> 4;
  int64_t r0, s0;
  uint32_t vr[4], vlo[2], vhi[2];
  int tpr[4], tps[2];
  const char *pr, *ps, *psh;
  constexpr int kR = SUM2 ? kSums : kPlain, kS = SUM2 ? kFactors : kPlain;
  constexpr int kT = kStep<SUM2, KIND>;
  auto place = [&](const MmParams& p, int64_t tr, int ts) {
    r0 = tr * kTile;
    s0 = int64_t(ts) * (KIND == kGlu ? kTile / 2 : kTile);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      vr[j] = copy_offset<Elem, RT, 256, false, kR>((j * 8 + wv) * 64 + lane, p.ldr, r0, p.nR,
                                                        &tpr[j]);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int id = (j * 8 + wv) * 64 + lane;
      vlo[j] = copy_offset<Elem, ST, 128, KIND != kGlu, kS>(id, p.lds, s0, p.nS, &tps[j]);
      vhi[j] = KIND == kGlu
                   ? vlo[j]
                   : copy_offset<Elem, ST, 128, true, kS>(id, p.lds, s0 + 64, p.nS, &tps[j]);
    }
    pr = static_cast<const char*>(p.R) + (RT ? r0 * p.ldr : SUM2 ? 2 * r0 : r0) * kSz;
    ps = static_cast<const char*>(p.S) + (ST ? s0 * p.lds : s0) * kSz;
    psh = ps + (KIND == kGlu ? p.nS * p.lds : ST ? 64 * p.lds : 64) * kSz;
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
  Acc acc[8][4];
  bf16x8 b[2][4], a[4];
  auto mma = [&](int i0, int h) {
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        acc[i0 + i][j] = mfma<Elem>(a[i], b[h][j], acc[i0 + i][j]);
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
      for (int j = 0; j < 4; ++j) acc[i][j] = Acc{0, 0, 0, 0};
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
    const int32_t c0 = int32_t(s0) + (KIND == kGlu ? wsn / 2 : wsn);
    const bool more = turn(p, round + 1, &tr, &ts);
    if (more) {
      place(p, tr, ts);
      begin();
    }
    if constexpr (KIND == kGlu) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f32x4 gate[4], up[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          gate[i] = acc[i][j];
          up[i] = acc[4 + i][j];
        }
        glu_out<ACT, false, true>(p, lds + kOffEpi + wv * 4096, gate, up, r + 16 * j, c0, 0);
      }
    } else {
      Piece<4, KIND> now, next;
      float bias[2][8], scale[2][8];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        fetch_bias<KIND>(p, c0 + 64 * c + (lane & 7) * 8, bias[c]);
        fetch_scale<KIND>(p, c0 + 64 * c + (lane & 7) * 8, scale[c]);
      }
      now.fetch(p, r, c0);
#pragma unroll
      for (int i = 0; i < 8; ++i) {       // rows 16 (i / 2), columns 64 (i & 1)
        const int j = i / 2, c = i & 1;
        if (i < 7) next.fetch(p, r + 16 * ((i + 1) / 2), c0 + 64 * ((i + 1) & 1));
        const Acc q[4] = {acc[4 * c][j], acc[4 * c + 1][j], acc[4 * c + 2][j], acc[4 * c + 3][j]};
        piece_out<ACT, false, true, true, KIND>(p, lds + kOffEpi + wv * 4096, q, now, bias[c],
                                                scale[c], 0);
        now = next;
      }
    }
    if (!more) return;
  }
}
#endif

template <bool RT, bool ST, int ACT, bool SUM2, int KIND = kMm>
__global__ __launch_bounds__(kThreads, 2) void mm256_kernel(MmParams p) {
#if defined(__HIP_DEVICE_COMPILE__)
  __shared__ __attribute__((aligned(1024))) char lds[kLds];
  mm256_body<RT, ST, ACT, SUM2, 0, KIND>(p, EveryRound{}, lds);
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
template <typename T> constexpr int kSmallTile = sizeof(T) <= 2 ? 128 : 64;


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
template <typename T, bool RT, bool ST, int ACT, int G, int NB, int BYTES, bool RES, bool SUM2,
          int KIND = kMm>
__device__ __forceinline__ void mm_small_body(const MmParams& p, uint32_t block, char* lds) {
  using Acc = typename KindOf<KIND>::Acc;
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
  const int64_t r0 = tr * kTileS, s0 = int64_t(ts) * (KIND == kGlu ? kTileS / 2 : kTileS);
  const int64_t t0 = split * p.t_split;
  const int64_t t1 = t0 + p.t_split < p.nT ? t0 + p.t_split : p.nT;
  constexpr int kCopies = kOp / (256 * BYTES);              // of a wave, per operand
  uint32_t vr[kCopies], vs[kCopies];
  int tpr[kCopies], tps[kCopies];
#pragma unroll
  for (int j = 0; j < kCopies; ++j) {
    const int id = (j * 4 + wv) * 64 + lane;
    vr[j] = copy_offset<T, RT, kTileS, false, kR, BYTES>(id, p.ldr, r0, p.nR, &tpr[j]);
    if constexpr (KIND == kGlu)
      vs[j] = copy_offset<T, ST, kTileS, false, kS, BYTES, kTileS / 4>(id, p.lds, s0, p.nS, &tps[j]);
    else
      vs[j] = copy_offset<T, ST, kTileS, false, kS, BYTES>(id, p.lds, s0, p.nS, &tps[j]);
  }
  // whether a copy's rows are of S' (the same for all of its lanes)
  auto second = [&](int j) {
    return KIND == kGlu && (((j * 4 + wv) * 64 / (16 / BYTES) / 8 / (kTileS / 4)) & 1);
  };
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
    Rsrc b2 = b;
    if constexpr (KIND == kGlu) {
      const char* up = ps + p.nS * p.lds * kSz;
      b2 = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(range ? up + k * ds : up), short(0),
                                             range, 0x00020000);
    }
    char* d = mine + (NB == 2 ? (k & 1) * 2 * kOp : 0) + wv * 64 * BYTES;
#pragma unroll
    for (int j = 0; j < kCopies; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(a, (lds_ptr)(d + j * 256 * BYTES), BYTES, vr[j], 0,
                                               0, 0);
#pragma unroll
    for (int j = 0; j < kCopies; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(second(j) ? b2 : b,
                                               (lds_ptr)(d + kOp + j * 256 * BYTES), BYTES, vs[j],
                                               0, 0, 0);
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
  Acc acc[kF][kF];
#pragma unroll
  for (int i = 0; i < kF; ++i)
#pragma unroll
    for (int j = 0; j < kF; ++j) acc[i][j] = Acc{0, 0, 0, 0};
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
  // an odd contraction of bytes: what lies behind its end in S's last unit is cleared
  const bool odd = KIND == kInt8 && t1 == p.nT && (rem & 15);
  auto part = [&](auto h_c, bool last) {
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
    if (KIND == kInt8 && odd && last) {
      const int left = rem - (decltype(h_c)::value * 64 + g * 16);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int n = left - 4 * e;
        const uint32_t keep = n >= 4 ? ~0u : n > 0 ? (1u << (8 * n)) - 1 : 0u;
#pragma unroll
        for (int i = 0; i < kF; ++i) a[i][e] &= keep;
      }
    }
#pragma unroll
    for (int i = 0; i < kF; ++i)
#pragma unroll
      for (int j = 0; j < kF; ++j) acc[i][j] = mfma<T>(a[i], b[j], acc[i][j]);
  };
  copy(0);
  for (int k = 0; k < nk; ++k) {
    wait_copies<0>();
    turn_end();       // stage k is whole, and stage k - 1 has been read by every wave
    if (NB == 2 && k + 1 < nk) copy(k + 1);
    const bool last = k0 + k == stages - 1;
    part(std::integral_constant<int, 0>{}, last);
    // the second half of the last stage may lie past the contraction's end (fp32 takes
    // it all the same: the branch between its halves costs 89 -> 96 us)
    if (kSz == 4 || k0 + k < stages - 1 || rem > kT / 2)
      part(std::integral_constant<int, 1>{}, last);
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
  Acc sum[kF][kOut];
  if constexpr (G == 1) {
#pragma unroll
    for (int i = 0; i < kF; ++i)
#pragma unroll
      for (int j = 0; j < kOut; ++j) sum[i][j] = acc[i][j];
  } else {
    // each group hands the other its half: 256 threads x 16 bytes per accumulator
    Acc* box = reinterpret_cast<Acc*>(lds) + (tid & 255);
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
  if constexpr (KIND == kGlu) {
    constexpr int kH = kF / 2;
    const int32_t c = int32_t(s0) + wsn / 2;
#pragma unroll
    for (int j = 0; j < kOut; ++j) {
      f32x4 gate[kH], up[kH];
#pragma unroll
      for (int i = 0; i < kH; ++i) {
        gate[i] = sum[i][j];
        up[i] = sum[kH + i][j];
      }
      if (p.splits > 1) glu_out<ACT, true, false>(p, sl, gate, up, r + 16 * j, c, split);
      else glu_out<ACT, false, NB == 1>(p, sl, gate, up, r + 16 * j, c, 0);
    }
    return;
  }
  const int32_t c = int32_t(s0) + wsn;
  Piece<kF, KIND> now, next;
  float bias[8];
  fetch_bias<KIND>(p, c + (lane % Piece<kF>::kPer) * 8, bias);
  float scale[8];
  fetch_scale<KIND>(p, c + (lane % Piece<kF>::kPer) * 8, scale);
  if (RES && p.splits == 1) now.fetch(p, r, c);
  else now.place(p, r, c);
#pragma unroll
  for (int j = 0; j < kOut; ++j) {
    Acc q[kF];
#pragma unroll
    for (int i = 0; i < kF; ++i) q[i] = sum[i][j];
    if (p.splits > 1) {
      now.place(p, r + 16 * j, c);
      piece_out<ACT, true, false, true, KIND>(p, sl, q, now, bias, scale, split);
    } else {
      if constexpr (RES) {
        if (j + 1 < kOut) next.fetch(p, r + 16 * (j + 1), c);
      } else {
        next.place(p, r + 16 * (j + 1), c);
      }
      piece_out<ACT, false, NB == 1, RES, KIND>(p, sl, q, now, bias, scale, 0);
      now = next;
    }
  }
}
#endif

template <typename T, bool RT, bool ST, int ACT, int G, int NB, int BYTES = 16, bool RES = true,
          bool SUM2 = false, int KIND = kMm>
__global__ __launch_bounds__(kSmallThreads * G, NB == 1 ? (RES ? 3 : 4) : 2)
void mm_small_kernel(MmParams p) {
#if defined(__HIP_DEVICE_COMPILE__)
  __shared__ __attribute__((aligned(1024))) char lds[kSmallLds<T, NB> * G];
  mm_small_body<T, RT, ST, ACT, G, NB, BYTES, RES, SUM2, KIND>(p, blockIdx.x, lds);
#endif
}

}  // namespace
}  // namespace ss
