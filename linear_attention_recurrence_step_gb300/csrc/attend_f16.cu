// attend_f16.cu -- kv_attend.cuh for f16 queries.
#include "kv_attend.cuh"

namespace gdn {

cudaError_t launch_attend_f16(const AttendArgs &a, cudaStream_t s) { return launch_attend<__half>(a, s); }

}  // namespace gdn
