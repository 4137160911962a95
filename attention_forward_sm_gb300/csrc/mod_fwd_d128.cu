// mod_attn_kernel, prefill, D = 128 (translation units of their own compile in
// parallel).
#include "mod_sm103a.cuh"

namespace attn {

cudaError_t launch_mod_fwd_d128(const ModKernelParams& p, unsigned grid, int dev,
                                 cudaStream_t stream) {
  return launch_variant<128, false, 0>(p, grid, dev, stream);
}

}  // namespace attn
