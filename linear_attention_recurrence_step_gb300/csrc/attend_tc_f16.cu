// attend_tc_f16.cu -- attend_tc.cuh for f16 queries.
#include "attend_tc.cuh"

namespace gdn {

cudaError_t launch_attend_tc_f16(const AttendArgs &a, cudaStream_t s) { return launch_attend_tc<__half>(a, s); }

}  // namespace gdn
