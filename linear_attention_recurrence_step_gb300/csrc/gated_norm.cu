// gated_norm.cu -- root-mean-square norm with the gate and the residual sum
// around it:
//     u = x                      (gate first: u = x * silu(gate))
//     u = residual + scale * u   (with a residual; also written out)
//     y = u * rsqrt(mean(u^2) + eps) * weight      (gate last: * silu(gate))
//
// Bound by memory: x, gate and residual are read once, y and the new residual
// written once, about ten operations per element.  A row stays in registers
// between its sum and its scaling; TPR threads share a row, so that narrow
// rows (a head of 128) fill a warp with several rows and wide ones a block.
// The sum, the mean and the scaled values are f32; y and the residual are
// each rounded once, and the norm takes the unrounded sum.
#include "pieces.cuh"
#include "layer.h"

namespace gdn {

namespace {

// Sum over the TPR threads of a row; every thread of the row gets it.
template <int TPR>
__device__ __forceinline__ float row_sum(float s, float *red) {
#pragma unroll
    for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if constexpr (TPR > 32) {
        const int warp = threadIdx.x / 32;
        if (threadIdx.x % 32 == 0) red[warp] = s;
        __syncthreads();
        s = 0.f;
#pragma unroll
        for (int i = 0; i < TPR / 32; ++i) s += red[i];
    }
    return s;
}

// TPR threads per row, NV pieces of VEC elements per thread.  A block holds
// max(1, 128 / TPR) rows.
template <typename T, int VEC, int TPR, int NV>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR) norm_kernel(const NormArgs a, int64_t rows) {
    constexpr int kRows = TPR < 128 ? 128 / TPR : 1;
    __shared__ float red[32];
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x % TPR;
    const int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / TPR;
    const bool on = row < rows;
    const int64_t m = on ? row / a.K : 0, k = on ? row % a.K : 0;
    const T *x = static_cast<const T *>(a.x) + m * a.x_st + k * a.D;
    const T *gate = a.gate ? static_cast<const T *>(a.gate) + m * a.gate_st + k * a.D : nullptr;
    const int64_t dense = (m * a.K + k) * a.D;
    const T *res = a.residual ? static_cast<const T *>(a.residual) + dense : nullptr;

    float u[NV][VEC], g[NV][VEC], rs[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int64_t d = ((int64_t)i * TPR + lane) * VEC;
#pragma unroll
        for (int e = 0; e < VEC; ++e) u[i][e] = 0.f;
        if (on && d < a.D) {
            load_piece<T, VEC>(u[i], x + d);
            if (gate) load_piece<T, VEC>(g[i], gate + d);
            if (res) load_piece<T, VEC>(rs[i], res + d);
        }
    }
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int64_t d = ((int64_t)i * TPR + lane) * VEC;
        if (on && d < a.D) {
            if (gate) {
#pragma unroll
                for (int e = 0; e < VEC; ++e) g[i][e] = silu(g[i][e]);
                if (a.gate_first)
#pragma unroll
                    for (int e = 0; e < VEC; ++e) u[i][e] *= g[i][e];
            }
            if (res) {
#pragma unroll
                for (int e = 0; e < VEC; ++e) u[i][e] = fmaf(a.scale, u[i][e], rs[i][e]);
                store_piece<T, VEC>(static_cast<T *>(a.residual_out) + dense + d, u[i]);
            }
#pragma unroll
            for (int e = 0; e < VEC; ++e) sum = fmaf(u[i][e], u[i][e], sum);
        }
    }
    sum = row_sum<TPR>(sum, red);
    const float inv = 1.f / sqrtf(sum / (float)a.D + a.eps);
    const T *w = static_cast<const T *>(a.weight) + (a.weight_rows > 1 ? k * a.D : 0);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int64_t d = ((int64_t)i * TPR + lane) * VEC;
        if (on && d < a.D) {
            float wv[VEC];
            load_piece<T, VEC>(wv, w + d);
            const bool last = gate && !a.gate_first;
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float v = u[i][e] * inv * wv[e];
                u[i][e] = last ? v * g[i][e] : v;
            }
            store_piece<T, VEC>(static_cast<T *>(a.y) + dense + d, u[i]);
        }
    }
}

// Rows wider than the registers of a block: two passes over the row, the
// second one from L2.
template <typename T>
__global__ void __launch_bounds__(1024) norm_wide_kernel(const NormArgs a) {
    __shared__ float red[32];
    pdl_trigger();
    pdl_wait();
    const int64_t m = blockIdx.x / a.K, k = blockIdx.x % a.K;
    const T *x = static_cast<const T *>(a.x) + m * a.x_st + k * a.D;
    const T *gate = a.gate ? static_cast<const T *>(a.gate) + m * a.gate_st + k * a.D : nullptr;
    const int64_t dense = (m * a.K + k) * a.D;
    const T *res = a.residual ? static_cast<const T *>(a.residual) + dense : nullptr;
    const T *w = static_cast<const T *>(a.weight) + (a.weight_rows > 1 ? k * a.D : 0);
    auto value = [&](int64_t d) {
        float u = ld_f32(x + d);
        if (gate && a.gate_first) u *= silu(ld_f32(gate + d));
        return res ? fmaf(a.scale, u, ld_f32(res + d)) : u;
    };
    float sum = 0.f;
    for (int64_t d = threadIdx.x; d < a.D; d += 1024) {
        const float u = value(d);
        sum = fmaf(u, u, sum);
    }
    sum = row_sum<1024>(sum, red);
    const float inv = 1.f / sqrtf(sum / (float)a.D + a.eps);
    for (int64_t d = threadIdx.x; d < a.D; d += 1024) {
        const float u = value(d);
        float v = u * inv * ld_f32(w + d);
        if (gate && !a.gate_first) v *= silu(ld_f32(gate + d));
        // residual_out and y may be x's, the residual's or the gate's own
        // buffer: this thread has read every input at d
        if (res) st_from_f32(static_cast<T *>(a.residual_out) + dense + d, u);
        st_from_f32(static_cast<T *>(a.y) + dense + d, v);
    }
}

template <typename T, int VEC, int TPR, int NV>
cudaError_t launch_cfg(const NormArgs &a, cudaStream_t s) {
    constexpr int kRows = TPR < 128 ? 128 / TPR : 1;
    const int64_t rows = a.M * a.K, blocks = (rows + kRows - 1) / kRows;
    if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
    return launch_dependent(norm_kernel<T, VEC, TPR, NV>, (unsigned)blocks, TPR < 128 ? 128 : TPR, 0, s, a, rows);
}

template <typename T, int VEC>
cudaError_t launch_v(const NormArgs &a, cudaStream_t s) {
    const int64_t n = (a.D + VEC - 1) / VEC;  // pieces per row
    if (n <= 16) return launch_cfg<T, VEC, 16, 1>(a, s);
    if (n <= 32) return launch_cfg<T, VEC, 32, 1>(a, s);
    if (n <= 64) return launch_cfg<T, VEC, 32, 2>(a, s);
    if (n <= 128) return launch_cfg<T, VEC, 128, 1>(a, s);
    if (n <= 256) return launch_cfg<T, VEC, 128, 2>(a, s);
    if (n <= 512) return launch_cfg<T, VEC, 256, 2>(a, s);
    if (n <= 1024) return launch_cfg<T, VEC, 512, 2>(a, s);
    if (n <= 2048) return launch_cfg<T, VEC, 512, 4>(a, s);
    if constexpr (VEC == 1) {
        if (n <= 8192) return launch_cfg<T, VEC, 512, 16>(a, s);
    }
    if (a.M * a.K > INT32_MAX) return cudaErrorInvalidConfiguration;
    return launch_dependent(norm_wide_kernel<T>, (unsigned)(a.M * a.K), 1024, 0, s, a);
}

template <typename T>
cudaError_t launch_t(const NormArgs &a, cudaStream_t s) {
    return a.vec ? launch_v<T, 16 / sizeof(T)>(a, s) : launch_v<T, 1>(a, s);
}

}  // namespace

cudaError_t launch_gated_norm(DType dt, const NormArgs &a, int, cudaStream_t s) {
    switch (dt) {
    case DType::F32: return launch_t<float>(a, s);
    case DType::BF16: return launch_t<__nv_bfloat16>(a, s);
    case DType::F16: return launch_t<__half>(a, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace gdn
