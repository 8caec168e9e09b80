// attend.h -- internal interface between attend_abi.cu and the kernels of the
// operators of an attention layer: page slots, rotary positions, the 4-bit
// paged cache and attention over it.  Arguments arrive here already
// validated; strides are in elements.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "launch.h"

namespace gdn {

struct SlotsArgs {
    const int32_t *lengths, *add;       // [B]; add may be null (T)
    const int32_t *held, *ring_state;   // [B], [2]: first free place, free pages
    int32_t *table, *ring;              // [B,width], [pages]
    int32_t *slots, *positions;         // [B,T]
    int32_t *granted, *lengths_out, *held_out, *ring_state_out;
    int64_t B, T;
    int width, pages, page_shift;
};
cudaError_t launch_page_slots(const SlotsArgs &a, cudaStream_t s);

struct RotaryArgs {
    const void *q, *k;                  // k may be null
    const int32_t *positions;           // [B,T]
    const float *inv_freq;              // [R/2]
    void *q_out, *k_out;
    int64_t B, T;
    int Hq, Hk, D, R;
    int64_t q_sb, q_st, k_sb, k_st, qo_sb, qo_st, ko_sb, ko_st;
    float scale;
    bool half, inverse;
    bool vec;                           // every row can be read and written in 16-byte pieces
};
cudaError_t launch_rotary(DType dt, const RotaryArgs &a, int sm_count, cudaStream_t s);

// Bytes of a page of one head: the keys' codes and scales, then the values'.
constexpr int64_t kv_block_bytes(int64_t page, int64_t D) { return page * D * 9 / 8; }

struct KvArgs {
    const void *k_in, *v_in;            // append: [B,T,H,D]
    void *k_out, *v_out;                // read: dense [B*T,H,D]
    const int32_t *slots;               // [B,T]
    const float *k_scale, *v_scale;     // [H] or null (1)
    unsigned char *cache;
    int64_t B, T, pages;
    int H, D, page_shift;
    int64_t k_sb, k_st, v_sb, v_st;     // append
    bool vec;                           // every row can be read (or written) in 16-byte pieces
};
cudaError_t launch_kv_append(DType dt, const KvArgs &a, cudaStream_t s);
cudaError_t launch_kv_read(DType dt, const KvArgs &a, cudaStream_t s);

struct AttendArgs {
    const void *q;                      // [B,T,Hq,D]
    const unsigned char *cache;
    const int32_t *table, *lengths, *fresh;  // [B,width], [B], [B] or null (T)
    const float *k_scale, *v_scale;     // [H] or null (1)
    void *y;                            // [B,T,Hq,D]
    float *lse;                         // [B,T,Hq] or null
    float *workspace;
    int64_t B, T, pages, q_sb, q_st;
    int Hq, H, D, width, page_shift;
    float scale;
    int window;                         // 0: none
    bool vec_q, vec_y;                  // rows of q, y begin on 16 bytes
};
int64_t attend_workspace_bytes(int64_t B, int64_t T, int64_t Hq, int64_t H, int64_t D);
// One translation unit per element type.
cudaError_t launch_attend_f32(const AttendArgs &a, cudaStream_t s);
cudaError_t launch_attend_bf16(const AttendArgs &a, cudaStream_t s);
cudaError_t launch_attend_f16(const AttendArgs &a, cudaStream_t s);
// The tcgen05 form (attend_tc.cuh, a translation unit per type), for f16 and bf16 calls
// of many query rows; its wait-expiry flag.
bool attend_tc_rows(int64_t units, int64_t rows);
bool attend_takes_tc(DType dt, const AttendArgs &a);
int64_t attend_tc_workspace_bytes(int64_t B, int64_t T, int64_t Hq, int64_t H, int64_t D);
cudaError_t launch_attend_tc(DType dt, const AttendArgs &a, cudaStream_t s);
cudaError_t launch_attend_tc_bf16(const AttendArgs &a, cudaStream_t s);
cudaError_t launch_attend_tc_f16(const AttendArgs &a, cudaStream_t s);
cudaError_t attend_tc_wait_flag(unsigned **flag);
cudaError_t attend_tc_take_wait_flag(unsigned *was_set);

}  // namespace gdn
