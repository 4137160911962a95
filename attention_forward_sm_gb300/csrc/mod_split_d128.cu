// mod_attn_kernel, decode, D = 128 (a translation unit of its own: they compile in parallel).
#include "mod_sm103a.cuh"

namespace attn {

cudaError_t launch_mod_split_d128(const ModKernelParams& p, unsigned grid, cudaStream_t stream) {
  return launch_variant<128, true>(p, grid, stream);
}

}  // namespace attn
