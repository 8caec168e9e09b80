// attend_tc_bf16.cu -- attend_tc.cuh for bf16 queries.
#include "attend_tc.cuh"

namespace gdn {

cudaError_t launch_attend_tc_bf16(const AttendArgs &a, cudaStream_t s) { return launch_attend_tc<__nv_bfloat16>(a, s); }

}  // namespace gdn
