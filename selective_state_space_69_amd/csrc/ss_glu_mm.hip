// The gated half of a feed-forward block: instantiations of the product kernels whose
// tiles hold both factors of their outputs (ss_mm_kernels.hpp).
#include "ss_mm_kernels.hpp"

namespace ss {
namespace {

template <int ACT>
void run(const MmParams& p, MmTile tile, hipStream_t stream) {
  const unsigned blocks = unsigned(p.tiles_r) * unsigned(p.tiles_s) * unsigned(p.splits);
  switch (tile) {
    case MmTile::kBig:
      mm256_kernel<true, true, ACT, false, kGlu>
          <<<blocks < kCUs ? blocks : kCUs, kThreads, 0, stream>>>(p);
      break;
    case MmTile::kSmall:
      mm_small_kernel<uint16_t, true, true, ACT, 1, 2, 16, false, false, kGlu>
          <<<blocks, kSmallThreads, 0, stream>>>(p);
      break;
    case MmTile::kSmallSingle:
      mm_small_kernel<uint16_t, true, true, ACT, 1, 1, 16, false, false, kGlu>
          <<<blocks, kSmallThreads, 0, stream>>>(p);
      break;
    case MmTile::kSmallPair:
      mm_small_kernel<uint16_t, true, true, ACT, 2, 2, 16, false, false, kGlu>
          <<<blocks, 2 * kSmallThreads, 0, stream>>>(p);
      break;
    case MmTile::kSmallF32:
      mm_small_kernel<float, true, true, ACT, 1, 2, 16, false, false, kGlu>
          <<<blocks, kSmallThreads, 0, stream>>>(p);
      break;
    case MmTile::kSmallF32Any:
      mm_small_kernel<float, true, true, ACT, 1, 2, 4, false, false, kGlu>
          <<<blocks, kSmallThreads, 0, stream>>>(p);
      break;
  }
}

}  // namespace

void launch_mm_glu(const MmParams& p, MmTile tile, hipStream_t stream) {
  // splits leave the activation to the join
  switch (p.splits > 1 ? int(SS_ACT_NONE) : p.act) {
    case SS_ACT_SILU: return run<SS_ACT_SILU>(p, tile, stream);
    case SS_ACT_GELU: return run<SS_ACT_GELU>(p, tile, stream);
    default: return run<SS_ACT_NONE>(p, tile, stream);
  }
}

}  // namespace ss
