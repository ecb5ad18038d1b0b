// The projection in 8-bit integers: instantiations of the product kernels on
// v_mfma_i32_16x16x64_i8 (ss_mm_kernels.hpp).
#include "ss_mm_kernels.hpp"

namespace ss {
namespace {

template <int ACT>
void run(const MmParams& p, MmTile tile, hipStream_t stream) {
  const unsigned blocks = unsigned(p.tiles_r) * unsigned(p.tiles_s) * unsigned(p.splits);
  switch (tile) {
    case MmTile::kBig:
      mm256_kernel<true, true, ACT, false, kInt8>
          <<<blocks < kCUs ? blocks : kCUs, kThreads, 0, stream>>>(p);
      break;
    case MmTile::kSmall:
      mm_small_kernel<uint8_t, true, true, ACT, 1, 2, 16, true, false, kInt8>
          <<<blocks, kSmallThreads, 0, stream>>>(p);
      break;
    case MmTile::kSmallSingle:
      if (p.res)
        mm_small_kernel<uint8_t, true, true, ACT, 1, 1, 16, true, false, kInt8>
            <<<blocks, kSmallThreads, 0, stream>>>(p);
      else
        mm_small_kernel<uint8_t, true, true, ACT, 1, 1, 16, false, false, kInt8>
            <<<blocks, kSmallThreads, 0, stream>>>(p);
      break;
    case MmTile::kSmallPair:
      mm_small_kernel<uint8_t, true, true, ACT, 2, 2, 16, true, false, kInt8>
          <<<blocks, 2 * kSmallThreads, 0, stream>>>(p);
      break;
    default: break;     // fp32 tiles are never planned for it
  }
}

}  // namespace

void launch_mm_q8(const MmParams& p, MmTile tile, hipStream_t stream) {
  // splits leave the epilogue to the join
  switch (p.splits > 1 ? int(SS_ACT_NONE) : p.act) {
    case SS_ACT_SILU: return run<SS_ACT_SILU>(p, tile, stream);
    case SS_ACT_GELU: return run<SS_ACT_GELU>(p, tile, stream);
    case SS_ACT_SOFTPLUS: return run<SS_ACT_SOFTPLUS>(p, tile, stream);
    default: return run<SS_ACT_NONE>(p, tile, stream);
  }
}

}  // namespace ss
