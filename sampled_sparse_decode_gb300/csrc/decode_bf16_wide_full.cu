// decode_bf16_wide_full.cu — instantiations of the attend-only decode kernel with full weights for
// bf16 K/V, wide variant (decode_kernel.cuh, template flag FULL).
#include "decode_kernel.cuh"

namespace santa {

cudaError_t decode_launch_bf16_wide_full(const DecodeParams& p, int head_dim, int group, dim3 grid,
                                   int cluster, cudaStream_t stream) {
  if (head_dim == 128) {
    SANTA_DISPATCH_G(
        group, return (decode_launch_t<true, 128, GG, true, 0, true>(p, grid, cluster, stream)))
  }
  SANTA_DISPATCH_G(
      group, return (decode_launch_t<true, 64, GG, true, 0, true>(p, grid, cluster, stream)))
}

}  // namespace santa
