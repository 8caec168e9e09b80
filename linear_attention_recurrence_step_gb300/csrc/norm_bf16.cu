// norm_bf16.cu -- the gated norm on bf16 tensors.
#include "gated_norm.cuh"

namespace gdn {

cudaError_t launch_norm_bf16(const NormArgs &a, int sm_count, cudaStream_t s) { return launch_norm<__nv_bfloat16>(a, sm_count, s); }

}  // namespace gdn
