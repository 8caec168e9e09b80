// norm_f16.cu -- the gated norm on f16 tensors.
#include "gated_norm.cuh"

namespace gdn {

cudaError_t launch_norm_f16(const NormArgs &a, int sm_count, cudaStream_t s) { return launch_norm<__half>(a, sm_count, s); }

}  // namespace gdn
