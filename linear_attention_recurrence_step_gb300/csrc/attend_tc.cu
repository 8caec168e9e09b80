// attend_tc.cu -- which calls attend_tc.cuh's kernel takes, and its wait-expiry flag.
#include "attend_tc.cuh"

namespace gdn {

__device__ unsigned g_attend_tc_wait_flag;

cudaError_t attend_tc_wait_flag(unsigned **flag) {
    void *p = nullptr;
    const cudaError_t e = cudaGetSymbolAddress(&p, g_attend_tc_wait_flag);
    *flag = static_cast<unsigned *>(p);
    return e;
}

int64_t attend_tc_workspace_bytes(int64_t B, int64_t T, int64_t Hq, int64_t H, int64_t D) {
    const int64_t rows = T * (Hq / H);
    return attend_tc_rows(B * H, rows) ? tc_plan(B, rows, H, D).workspace : 0;
}

// The rows of a (sequence, key head) from which they go here and not to
// kv_attend.cuh's kernel.  16 sequences of 2048 to 8192 tokens, 8 heads of 128: here 79 to
// 82 us with 32 to 128 rows; there 72 (32 rows), 78 (48), 108 (64) and 172 (128) where
// sequences bring half of their rows in the mean, 83, 116, 146 and 242 where they bring
// all.  Heads of 64: here 65, there 52, 74, 91 and 142; of 256: here 152, there 179, 233,
// 291 and 532.  One sequence of 8192, which has to be joined here, heads of 64, 128 and
// 256: here 20, 27 and 43 us with 32 to 128 rows; there 19, 28 and 55 (64 rows), 29, 38 and
// 86 (128).
bool attend_tc_rows(int64_t units, int64_t rows) { return rows > (2 * units >= kTcSms ? 48 : 64); }
bool attend_takes_tc(DType dt, const AttendArgs &a) { return dt != DType::F32 && attend_tc_rows(a.B * a.H, a.T * (a.Hq / a.H)); }

cudaError_t launch_attend_tc(DType dt, const AttendArgs &a, cudaStream_t s) {
    return dt == DType::BF16 ? launch_attend_tc_bf16(a, s) : launch_attend_tc_f16(a, s);
}

cudaError_t attend_tc_take_wait_flag(unsigned *was_set) {
    unsigned v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_attend_tc_wait_flag, sizeof v);
    if (e != cudaSuccess) return e;
    *was_set = v;
    if (v) {
        const unsigned zero = 0;
        e = cudaMemcpyToSymbol(g_attend_tc_wait_flag, &zero, sizeof zero);
    }
    return e;
}

}  // namespace gdn
