// mod_attn_kernel, decode, D = 64, more than 8 query heads per KV head.
#include "mod_sm103a.cuh"

namespace attn {

cudaError_t launch_mod_split_d64_h0(const ModKernelParams& p, unsigned grid, int dev,
                                 cudaStream_t stream) {
  return launch_variant<64, true, 0>(p, grid, dev, stream);
}

}  // namespace attn
