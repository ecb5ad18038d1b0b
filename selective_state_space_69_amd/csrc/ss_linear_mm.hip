// Plain products of the linear projections (templates and their measurements in
// ss_mm_kernels.hpp): forward, and both products of a backward pass.
#include "ss_mm_kernels.hpp"

namespace ss {

namespace {

// Both products of a backward pass: dw's tiles, of which the last round does not
// reach every workgroup, then dx's (16384 rows, 5120 -> 2560: 750 us one after the
// other, where dw's 200 tiles leave 56 CUs idle, 708 together; 2560 -> 5120 from a
// checkpoint 757 and 686).
template <bool SUM2>
__global__ __launch_bounds__(kThreads, 2) void mm256_both_kernel(MmParams dw, MmParams, Behind) {
#if defined(__HIP_DEVICE_COMPILE__)
  __shared__ __attribute__((aligned(1024))) char lds[kLds];
  constexpr int kDx = int(sizeof(MmParams)), kTurns = 2 * kDx;
  mm256_body<false, false, SS_ACT_NONE, SUM2, 0, kMm>(dw, EveryRound{}, lds);
  const MmParams dx = reread_params<MmParams, kDx>();
  mm256_body<true, false, SS_ACT_NONE, SUM2, kDx, kMm>(
      dx, BehindOthers{reread_params<Behind, kTurns>()}, lds);
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
