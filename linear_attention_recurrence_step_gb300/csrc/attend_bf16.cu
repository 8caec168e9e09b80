// attend_bf16.cu -- kv_attend.cuh for bf16 queries.
#include "kv_attend.cuh"

namespace gdn {

cudaError_t launch_attend_bf16(const AttendArgs &a, cudaStream_t s) { return launch_attend<__nv_bfloat16>(a, s); }

}  // namespace gdn
