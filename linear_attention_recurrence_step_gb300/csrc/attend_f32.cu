// attend_f32.cu -- kv_attend.cuh for f32 queries.
#include "kv_attend.cuh"

namespace gdn {

cudaError_t launch_attend_f32(const AttendArgs &a, cudaStream_t s) { return launch_attend<float>(a, s); }

int64_t attend_workspace_bytes(int64_t B, int64_t T, int64_t Hq, int64_t H, int64_t D) {
    int64_t rows, pairs;
    if (H > 65535 || __builtin_mul_overflow(T, Hq / H, &rows) || rows > INT32_MAX - 64) return -1;
    const int NB = eights_of(rows);
    if (__builtin_mul_overflow(B, (rows + 8 * NB - 1) / (8 * NB), &pairs) || pairs > INT32_MAX) return -1;
    // whichever form the call takes
    const int64_t tc = attend_tc_workspace_bytes(B, T, Hq, H, D);
    const int blocks = kSms * resident(NB, (int)D, false);  // (no fewer than for f32)
    if (!cut(pairs, H, blocks)) return tc;
    const int64_t own = ((int64_t)2 * blocks * partial_floats(8 * NB, (int)D) + kBaseFloats) * 4;
    return own > tc ? own : tc;
}

}  // namespace gdn
