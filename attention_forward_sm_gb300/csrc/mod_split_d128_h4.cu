// mod_attn_kernel, decode, D = 128, at most 4 query heads per KV head.
#include "mod_sm103a.cuh"

namespace attn {

cudaError_t launch_mod_split_d128_h4(const ModKernelParams& p, unsigned grid, int dev,
                                 cudaStream_t stream) {
  return launch_variant<128, true, 4>(p, grid, dev, stream);
}

}  // namespace attn
