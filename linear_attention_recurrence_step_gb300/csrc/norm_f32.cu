// norm_f32.cu -- the gated norm on f32 tensors.
#include "gated_norm.cuh"

namespace gdn {

cudaError_t launch_norm_f32(const NormArgs &a, int sm_count, cudaStream_t s) { return launch_norm<float>(a, sm_count, s); }

}  // namespace gdn
