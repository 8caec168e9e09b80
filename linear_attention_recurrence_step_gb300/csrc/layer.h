// layer.h -- internal interface between layer_abi.cu and the kernels of the
// operators around the recurrence: short causal convolution, selective scan,
// gated norm, sampling.  Arguments arrive here already validated; strides are
// in elements.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "launch.h"

namespace gdn {

struct ConvArgs {
    const void *x, *weight, *bias;      // bias may be null
    const void *state_in;               // [B,W-1,C] or null (zeros)
    const int32_t *lengths;             // [B] or null (T)
    void *y;                            // [B,T,C] or null
    void *state_out;                    // [B,W-1,C] or null
    int64_t B, T, C;
    int64_t x_sb, x_st;
    int W;
    bool silu;
    bool vec;                           // every row can be read in 16-byte pieces
};
cudaError_t launch_causal_conv(DType dt, const ConvArgs &a, int sm_count, cudaStream_t s);

struct ScanArgs {
    const void *x, *dt, *Bm, *Cm;
    const float *A, *D, *dt_bias;       // [H]; D, dt_bias may be null
    const float *state_in;              // [B,H,P,N] or null (zeros)
    const int32_t *lengths;             // [B] or null (T)
    void *y;                            // [B,T,H,P] or null
    float *state_out;                   // [B,H,P,N] or null
    float *workspace;
    int64_t B, T, H, P, G;
    int64_t x_sb, x_st, dt_sb, dt_st, b_sb, b_st, c_sb, c_st;
    int N;
    bool softplus;
    bool vec_bc;                        // B and C rows can be read in 16-byte pieces
    bool vec_x;                         // and x rows
    bool chunked;                       // the tensor-core form (scan_chunk.cu)
    int segments;                       // parts that the steps are split into
    int64_t seg_steps;                  // steps per part (the last may be shorter)
};
struct ScanPlan {
    int segments;
    int64_t seg_steps;
    int64_t bytes;                      // workspace, -1 on overflow
};
ScanPlan scan_plan(int64_t B, int64_t T, int64_t H, int64_t P, int64_t N, bool chunked);
bool scan_supported_n(int64_t N);
// Warps per CTA and CTAs per head of the tensor-core form; whether a call of
// these sizes takes it (its tensors' alignment permitting).
int scan_chunk_warps(int64_t P, int64_t *row_blocks);
bool scan_chunk_sizes(DType dt, int64_t T, int64_t P, int64_t N);
cudaError_t launch_scan_chunk(const ScanArgs &a, cudaStream_t s);
// What a kernel of a call does: all of it; or, of a call in segments, the
// segments' end states (then launch_scan_join), or its output.
enum ScanPhase { kScanWhole = 0, kScanFold = 1, kScanOutput = 2 };
cudaError_t launch_scan_join(const ScanArgs &a, cudaStream_t s);
cudaError_t launch_selective_scan(DType dt, const ScanArgs &a, int sm_count, cudaStream_t s);

struct NormArgs {
    const void *x, *weight, *gate, *residual;  // gate, residual may be null
    void *y, *residual_out;                    // residual_out is null without residual
    int64_t M, K, D;                           // tokens, heads, width of a norm
    int64_t x_st, gate_st;                     // token strides of x and gate
    int64_t weight_rows;                       // 1, or K
    float scale, eps;
    bool gate_first;
    bool vec;                                  // every row is whole 16-byte pieces
    bool shift;                                // dense rows of another width from 16-byte aligned bases
};
// One translation unit per element type.
cudaError_t launch_norm_f32(const NormArgs &a, int sm_count, cudaStream_t s);
cudaError_t launch_norm_bf16(const NormArgs &a, int sm_count, cudaStream_t s);
cudaError_t launch_norm_f16(const NormArgs &a, int sm_count, cudaStream_t s);

struct SampleArgs {
    const void *logits;
    const float *noise;
    const float *temperature, *top_p, *min_p;  // [R] or null (then the value below)
    const int32_t *top_k;
    float temperature_v, top_p_v, min_p_v;
    int32_t top_k_v;
    int32_t *token;
    float *logprob;                            // may be null
    int64_t R, V;
    int64_t logits_st, noise_st;
};
cudaError_t launch_sample(DType dt, const SampleArgs &a, int sm_count, cudaStream_t s);

}  // namespace gdn
