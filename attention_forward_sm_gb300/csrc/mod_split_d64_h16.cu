// mod_attn_kernel, decode, D = 64, at most 16 query heads per KV head.
#include "mod_sm103a.cuh"

namespace attn {

cudaError_t launch_mod_split_d64_h16(const ModKernelParams& p, unsigned grid, int dev,
                                 cudaStream_t stream) {
  return launch_variant<64, true, 16>(p, grid, dev, stream);
}

}  // namespace attn
