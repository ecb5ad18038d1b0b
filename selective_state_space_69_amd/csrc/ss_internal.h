// Internal interface between the C-ABI layer (ss_api.cpp: validation and
// planning, pure host logic) and the HIP launchers (ss_fwd.hip, ss_bwd.hip,
// ss_step.hip).  Not installed; the public contract is include/ss_scan.h.
#pragma once

#include <cstddef>
#include <cstdint>
#include <initializer_list>

#include "ss_ckpt.h"
#include "ss_conv.h"
#include "ss_glu.h"
#include "ss_linear.h"
#include "ss_norm.h"
#include "ss_q8.h"
#include "ss_rec.h"
#include "ss_ssd.h"
#include "ss_scan.h"

namespace ss {

constexpr int kWave = 64;      // lanes per wavefront on CDNA
constexpr int kMaxState = 16;  // states held per lane
constexpr int kHalfWaveSplit = 8;
constexpr int kOneStateSplit = 16;

// Argument checks shared by the entry points.
constexpr size_t kAlign = 256;     // workspace alignment
constexpr size_t kPtrAlign = 16;   // every tensor pointer (rows are read with 16-byte loads)
inline bool valid_dtype(int32_t t) { return t == SS_F32 || t == SS_BF16; }
inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline bool all_aligned(std::initializer_list<const void*> ptrs) {      // NULL is
  for (const void* p : ptrs)
    if (p && !aligned(p, kPtrAlign)) return false;
  return true;
}
// Rows read or written with a stride need their element alignment only.
inline size_t row_align(int64_t stride, int32_t dtype) {
  return stride == 0 ? kPtrAlign : dtype == SS_BF16 ? 2 : 4;
}
inline bool bad_stride(int64_t stride, int64_t dim, int64_t most) {
  return stride != 0 && (stride < dim || stride > most);
}

// How a forward (or the forward recompute inside the backward) is split.
// nsplit : waves per (b, 64-channel block), each holding 16 / nsplit states;
//          kHalfWaveSplit selects the 32-channel kernel (4 waves per
//          (b, 32-channel block), two states per lane), kOneStateSplit the
//          16-channel kernel (4 waves per (b, 16-channel block), one state per
//          lane).
// nchunks == 1: one sequential pass over time per workgroup.
// nchunks  > 1: (1) chunk summaries, (2) carry scan over chunks, (3) output pass.
struct TimePlan {
  int64_t chunk_len = 0;
  int64_t nchunks = 1;
  int nsplit = 1;
};

// Workspace layout of the forward: fp32 arrays, each 256-byte aligned.
//   brow, crow : (B, L, 16)    B and C rows padded with zeros to 16 states, in
//                              the input type (only when N < 16; else the inputs are read)
//   hend : (B, nchunks, N, D)  chunk-local end state, then (after the carry scan)
//                              the start state of the chunk
//   dsum : (B, nchunks, D)     sum over the chunk of the step, in log2 units
struct FwdPlan {
  TimePlan tp;
  bool packed_rows = false;
  size_t off_brow = 0, off_crow = 0, off_hend = 0, off_dsum = 0, bytes = 0;
};

// Backward workspace (fp32 arrays, 256-byte aligned):
//   brow, crow : (B, L, 16)   B and C rows padded to 16 states (only when N < 16)
//   hend, dsum : (B, nchunks, N, D), (B, nchunks, D)  forward chunk carries
//   lam        : (B, nchunks, N, D)  adjoint carry entering each chunk from its end
//   pB, pC     : (B, L, nblk, N)     dB, dC summed over one 64-channel block
//   pA         : (B, nchunks, N, D)  dA summed over one chunk
//   pD, pbias  : (B, nchunks, D)     dD_skip, ddelta_bias summed over one chunk
// The partial sums are added in a fixed order by reduction kernels, so the
// backward is deterministic.
struct BwdPlan {
  TimePlan tp;
  int64_t nblk = 0;
  bool packed_rows = false;
  size_t off_brow = 0, off_crow = 0, off_hend = 0, off_dsum = 0, off_lam = 0, off_pB = 0,
         off_pC = 0, off_pA = 0, off_pD = 0, off_pbias = 0, bytes = 0;
};

// SS_OK when the current device is a gfx950, SS_ERR_UNSUPPORTED for another
// architecture, SS_ERR_HIP when no device can be queried (ss_runtime.hip; the
// answer is cached per device).
int check_device();

// Size of the static scratch array of ss_scan_fwd_noalloc (ss_runtime.hip).
constexpr size_t kStaticScratchBytes = size_t(SS_SCAN_STATIC_SCRATCH_BYTES);
// This GPU's copy of that array (its device address, looked up once per
// device with the device current): SS_OK, SS_ERR_HIP or SS_ERR_UNSUPPORTED.
int static_scratch(void** out);

TimePlan plan_time(const ss_desc_t& d);
FwdPlan plan_fwd(const ss_desc_t& d);
BwdPlan plan_bwd(const ss_desc_t& d);

struct FwdArgs {
  const void* u;
  const void* delta;
  const float* A;
  const void* Bm;
  const void* Cm;
  const float* Dskip;
  const float* bias;
  const void* z;
  const float* h0;
  void* y;
  float* h_last;
  void* Brow;    // B, C rows padded to 16 per (b, t), input type
  void* Crow;
  float* hend;
  float* dsum;
  int rev = 0;   // reverse time: h_t from h_{t+1}, t = L-1 .. 0
  int acc = 0;   // add the result to y instead of overwriting it
};

struct BwdArgs {
  const void* u;
  const void* delta;
  const float* A;
  const void* Bm;
  const void* Cm;
  const float* Dskip;
  const float* bias;
  const void* z;
  const float* h0;
  const void* dy;
  float* du;
  float* ddelta;
  float* dA;
  float* dB;
  float* dC;
  float* dDskip;
  float* dbias;
  float* dz;
  float* dh0;
  char* ws;
};

struct StepArgs {
  float* h;
  const void* u;
  const void* delta;
  const float* A;
  const void* Bm;
  const void* Cm;
  const float* Dskip;
  const float* bias;
  const void* z;
  void* y;
};

// Launchers: return 0 or a HIP error code (converted to SS_ERR_HIP by the caller).
int launch_fwd(const ss_desc_t& d, const FwdPlan& p, const FwdArgs& a, void* stream);
// B and C rows as (B, L, 16) in the input type, zero past N.
int launch_pack_rows(const ss_desc_t& d, const void* Bm, const void* Cm, void* Brow, void* Crow,
                     void* stream);
// Chunk start states of a chunked forward (summary pass + carry scan) into
// a.hend / a.dsum; a.Brow / a.Crow must hold the 16-wide rows.
int launch_fwd_carries(const ss_desc_t& d, const TimePlan& tp, const FwdArgs& a, void* stream);
int launch_bwd(const ss_desc_t& d, const BwdPlan& p, const BwdArgs& a, void* stream);
// Conv1d + SiLU (ss_conv.hip).  Time runs in independent segments of
// kConvSeg steps; vec = 4 channels per thread when D % 4 == 0, else 1.
// Backward workspace: per-segment partials of dw (B * nseg, D, K) and dbias
// (B * nseg, D), fp32, 256-byte aligned.
constexpr int kConvSeg = 64;
struct ConvPlan {
  int64_t nseg = 1;
  int vec = 1;
  size_t off_dw = 0, off_db = 0, bytes = 0;
};
ConvPlan plan_conv(const ss_conv_desc_t& d);
int launch_conv_fwd(const ss_conv_desc_t& d, const ConvPlan& plan, const void* x, const float* w,
                    const float* bias, void* u, void* stream);
int launch_conv_bwd(const ss_conv_desc_t& d, const ConvPlan& plan, const void* x, const float* w,
                    const float* bias, const float* du, float* dx, float* dw, float* dbias,
                    char* ws, void* stream);
int launch_conv_step(const ss_conv_desc_t& d, float* state, const void* x, const float* w,
                     const float* bias, void* u, void* stream);

// Chunk carries (ss_carry.hip), in place on states (B, nc, N, D): forward turns
// chunk summaries into chunk start states (h0 may be null), reverse turns local
// adjoints into the adjoints entering each chunk from its end.
int launch_chunk_carry(float* states, const float* dsum, const float* A, const float* h0,
                       int64_t batch, int64_t D, int N, int nc, bool reverse, void* stream);
// Both carries of the backward (forward on hstates, reverse on lstates), in
// one launch when the chunks are walked in order.
int launch_chunk_carry_pair(float* hstates, float* lstates, const float* dsum, const float* A,
                            const float* h0, int64_t batch, int64_t D, int N, int nc,
                            void* stream);
int launch_step(const ss_desc_t& d, const StepArgs& a, void* stream);
// Complex-A forward plan: 32 channels per workgroup, time cut into nchunks
// chunks of chunk_len steps (one when nchunks == 1).  Workspace (256-byte
// aligned): hend (B, nchunks, N, D) complex fp32 pairs (chunk summaries, then
// chunk start states) and dsum (B, nchunks, D) fp64 (sums of dt log2 e).
struct CplxPlan {
  int64_t chunk_len = 0;
  int64_t nchunks = 1;
  size_t off_hend = 0, off_dsum = 0, bytes = 0;
};
// allow_chunks = false: the one-pass plan (no workspace)
CplxPlan plan_fwd_complex(const ss_desc_t& d, bool allow_chunks);
// Complex-A forward (ss_complex.hip): A (D,N,2), B, C (B,L,N,2), h0 / h_last (B,D,N,2).
int launch_fwd_complex(const ss_desc_t& d, const CplxPlan& plan, const void* u, const void* delta,
                       const float* A, const void* Bm, const void* Cm, const float* Dskip,
                       const float* bias, const void* z, const float* h0, void* y, float* h_last,
                       char* ws, void* stream);
// Complex-A decode step (ss_complex.hip): h (B,D,N,2) in place, A (D,N,2), B, C (B,N,2).
int launch_step_complex(const ss_desc_t& d, const StepArgs& a, void* stream);
// SSD (Mamba-2) forward (ss_ssd.hip): one workgroup per (batch row, head);
// h0 / h_last (B, H, N, P) may be null and may be the same buffer.
int launch_ssd_fwd(const ss_ssd_desc_t& d, const void* x, const void* dt, const float* A,
                   const void* Bm, const void* Cm, const float* D, const float* dt_bias,
                   const float* h0, void* y, float* h_last, void* stream);
// SSD single step on the state h (B, H, N, P), in place (ss_ssd.hip).
int launch_ssd_step(const ss_ssd_desc_t& d, float* h, const void* x, const void* dt,
                    const float* A, const void* Bm, const void* Cm, const float* D,
                    const float* dt_bias, void* y, void* stream);


// Layer norm (ss_norm.hip): nwaves waves per row with vpt vectors of 8 channels
// per thread, groups rows side by side in a block.  Backward workspace: nparts partial rows (D) of dweight and of
// dbias, fp32, 256-byte aligned.
struct NormPlan {
  int nwaves = 1, vpt = 1, groups = 1;
  int64_t blocks = 1;
  int nparts = 1;
  size_t off_w = 0, off_b = 0, bytes = 0;
};
NormPlan plan_norm(const ss_norm_desc_t& d);
int launch_norm_fwd(const ss_norm_desc_t& d, const void* x, const void* residual,
                    const float* weight, const float* bias, void* y, void* sum, float* mean,
                    float* rstd, void* stream);
int launch_norm_bwd(const ss_norm_desc_t& d, const NormPlan& pl, const void* s,
                    const float* weight, const float* mean, const float* rstd, const void* dy,
                    const void* dsum, void* dx, float* dweight, float* dbias, char* ws,
                    void* stream);
// Column sums of nparts rows of N floats, in a fixed order, of one array or two
// (src1, dst1 null: one); a null dst is skipped (ss_norm.hip).
void launch_column_sums(const float* src0, float* dst0, const float* src1, float* dst1,
                        int64_t nparts, int32_t N, void* stream);

// 8-bit checkpoints (ss_ckpt.hip).
int launch_ckpt_pack(const ss_ckpt_desc_t& d, const void* x, int8_t* q, uint8_t* e, void* stream);
int launch_ckpt_unpack(const ss_ckpt_desc_t& d, const int8_t* q, const uint8_t* e, void* x,
                       void* stream);

// Linear projections (ss_linear.hip).  Workspace, 256-byte aligned arrays:
//   dpre : (M, N) in_dtype, dy act'(pre) (only with an activation, a dy of another
//          type than the operands, or bf16 rows of dy that 16-byte loads cannot read);
//          sum2: as the sum of two bf16, 2 elements per value, where one cannot hold it
//   x, w : (M, K), (N, K) bf16, rows copied to a 16-byte aligned stride where they
//          cannot be read in place (fp32 always is); x: also the checkpoint's values
//   sums : (chunks, N) fp32, dbias sums of chunk_rows rows
//   part : fp32 partial products of split contractions (dx's and dw's in one place,
//          or dw's off_part_dw bytes behind dx's where one launch computes both)
struct LinearPlan {
  bool need_dpre = false, sum2 = false;
  int64_t ld_dpre = 0;                 // elements from one row of dpre to the next
  int64_t chunk_rows = 1, chunks = 1;
  size_t off_dpre = 0, off_x = 0, off_w = 0, off_sums = 0, off_part = 0,
         off_part_dw = 0, bytes = 0;
};
LinearPlan plan_linear(const ss_linear_desc_t& d, int op);
int launch_linear_fwd(const ss_linear_desc_t& d, const void* x, const void* w, const float* bias,
                      const void* residual, void* y, void* pre, char* ws, void* stream);
// x or its checkpoint (q, e)
int launch_linear_bwd(const ss_linear_desc_t& d, const LinearPlan& pl, const void* x,
                      const int8_t* q, const uint8_t* e, const void* w, const void* pre,
                      const void* dy, void* dx, void* dw, float* dbias, char* ws, void* stream);

// Gated linear recurrence (ss_rec.hip): time in nchunks chunks of `chunk` steps, one
// workgroup each per group of channels.  Workspace, fp32 (B, nchunks, D) arrays, 256-byte
// aligned: chunks' log2 decays (off_log) and their end states or leaving adjoints (off_carry)
// where nchunks > 1, and then, forward, a (B, D) copy of h0 (off_first); backward partial sums
// of dlam (off_part).
struct RecPlan {
  int64_t chunk = 0, nchunks = 1;
  size_t off_log = 0, off_carry = 0, off_first = 0, off_part = 0, bytes = 0;
};
RecPlan plan_rec(const ss_rec_desc_t& d, int op);
int launch_rec_fwd(const ss_rec_desc_t& d, const RecPlan& pl, const void* x, const void* r,
                   const void* i, const float* lam, const void* z, const float* h0,
                   const uint8_t* starts, const int32_t* lengths, void* y, float* h_last,
                   float* states, char* ws, void* stream);
int launch_rec_bwd(const ss_rec_desc_t& d, const RecPlan& pl, const void* x, const void* r,
                   const void* i, const float* lam, const void* z, const uint8_t* starts,
                   const int32_t* lengths, const float* states, const void* dy,
                   const float* dh_last, void* dx, void* dr, void* di, void* dz, float* dlam,
                   float* dh0, char* ws, void* stream);
int launch_rec_step(const ss_rec_desc_t& d, float* h, const void* x, const void* r, const void* i,
                    const float* lam, const void* z, void* y, void* stream);

// Gated half of a feed-forward block (ss_linear.hip): the projection's plan for both
// halves' columns.
LinearPlan plan_glu(const ss_glu_desc_t& d, int op);
int launch_glu_fwd(const ss_glu_desc_t& d, const LinearPlan& pl, const void* x, const void* w,
                   const float* bias, void* y, void* pre, char* ws, void* stream);
int launch_glu_bwd(const ss_glu_desc_t& d, const LinearPlan& pl, const void* x, const void* w,
                   const void* pre, const void* dy, void* dx, void* dw, float* dbias, char* ws,
                   void* stream);

// Projection in 8-bit integers (ss_linear.hip, ss_q8.hip).  Workspace: rows of xq and wq at
// a 16-byte aligned stride where they cannot be read in place, int32 partial sums.
struct Q8Plan {
  size_t off_x = 0, off_w = 0, off_part = 0, bytes = 0;
};
Q8Plan plan_q8(const ss_q8_desc_t& d);
int launch_q8_pack(const ss_q8_pack_desc_t& d, const void* x, int8_t* q, float* s, void* stream);
int launch_q8_linear(const ss_q8_desc_t& d, const Q8Plan& pl, const int8_t* xq, const float* xs,
                     const int8_t* wq, const float* wsc, const float* bias, const void* residual,
                     void* y, char* ws, void* stream);

}  // namespace ss
