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

// TPR threads per row, NV pieces of VEC elements per thread, RPG rows per
// group of threads with their loads in flight together.  A block holds
// max(1, 128 / TPR) groups.  SHIFT: rows start `mis` elements past a 16-byte
// boundary (dense rows of a width that is no whole number of pieces); pieces
// are cut on those boundaries, and those at a row's ends go element by element.
template <typename T, int VEC, int TPR, int NV, int RPG, bool SHIFT>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR) norm_kernel(const NormArgs a, int64_t rows) {
    constexpr int kGroups = TPR < 128 ? 128 / TPR : 1;
    static_assert(RPG == 1 || TPR <= 32, "several rows of a group only within a warp");
    __shared__ float red[32];
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x % TPR;
    const int64_t row0 = ((int64_t)blockIdx.x * kGroups + threadIdx.x / TPR) * RPG;
    const T *const xb = static_cast<const T *>(a.x), *const gb = static_cast<const T *>(a.gate);
    const T *const rb = static_cast<const T *>(a.residual), *const wb = static_cast<const T *>(a.weight);
    T *const yb = static_cast<T *>(a.y), *const ob = static_cast<T *>(a.residual_out);

    RawPiece<T, VEC> xr[RPG][NV], gr[RPG][NV], rr[RPG][NV];
    int64_t dense[RPG], at_x[RPG], at_g[RPG];
    int64_t at_w[RPG];
    int mis[RPG];
    bool on[RPG];
#pragma unroll
    for (int q = 0; q < RPG; ++q) {
        const int64_t row = row0 + q;
        on[q] = row < rows;
        int64_t m = row, k = 0;
        if (a.K > 1) {
            m = row / a.K;
            k = row - m * a.K;
        }
        dense[q] = row * a.D;
        at_x[q] = m * a.x_st + k * a.D;
        at_g[q] = m * a.gate_st + k * a.D;
        at_w[q] = a.weight_rows > 1 ? k * a.D : 0;
        mis[q] = SHIFT ? (int)(dense[q] % VEC) : 0;
    }
    // whether piece i of row q lies inside the row, or across one of its ends
    auto place = [&](int q, int i) { return ((int64_t)i * TPR + lane) * VEC - mis[q]; };
    auto inside = [&](int q, int64_t d) { return on[q] && d >= 0 && d + VEC <= a.D; };
    auto across = [&](int q, int64_t d) { return SHIFT && on[q] && d + VEC > 0 && d < a.D && !(d >= 0 && d + VEC <= a.D); };
#pragma unroll
    for (int q = 0; q < RPG; ++q)
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int64_t d = place(q, i);
            if (inside(q, d)) {
                xr[q][i] = load_raw<T, VEC>(xb + at_x[q] + d);
                if (gb) gr[q][i] = load_raw<T, VEC>(gb + at_g[q] + d);
                if (rb) rr[q][i] = load_raw<T, VEC>(rb + dense[q] + d);
            }
        }
#pragma unroll
    for (int q = 0; q < RPG; ++q) {
        float u[NV][VEC], g[NV][VEC];
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int64_t d = place(q, i);
            const bool in = inside(q, d), end = across(q, d);
#pragma unroll
            for (int e = 0; e < VEC; ++e) u[i][e] = g[i][e] = 0.f;
            if (in || end) {
                float rs[VEC];
                if (in) {
                    widen<T, VEC>(u[i], xr[q][i]);
                    if (gb) widen<T, VEC>(g[i], gr[q][i]);
                    if (rb) widen<T, VEC>(rs, rr[q][i]);
                } else {
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        const bool there = d + e >= 0 && d + e < a.D;
                        u[i][e] = there ? ld_f32(xb + at_x[q] + d + e) : 0.f;
                        g[i][e] = there && gb ? ld_f32(gb + at_g[q] + d + e) : 0.f;
                        rs[e] = there && rb ? ld_f32(rb + dense[q] + d + e) : 0.f;
                    }
                }
                if (gb) {
#pragma unroll
                    for (int e = 0; e < VEC; ++e) g[i][e] = silu(g[i][e]);
                    if (a.gate_first)
#pragma unroll
                        for (int e = 0; e < VEC; ++e) u[i][e] *= g[i][e];
                }
                if (rb) {
#pragma unroll
                    for (int e = 0; e < VEC; ++e) u[i][e] = fmaf(a.scale, u[i][e], rs[e]);
                    if (in) {
                        store_piece<T, VEC>(ob + dense[q] + d, u[i]);
                    } else {
#pragma unroll
                        for (int e = 0; e < VEC; ++e)
                            if (d + e >= 0 && d + e < a.D) st_from_f32(ob + dense[q] + d + e, u[i][e]);
                    }
                }
#pragma unroll
                for (int e = 0; e < VEC; ++e) sum = fmaf(u[i][e], u[i][e], sum);
            }
        }
        sum = row_sum<TPR>(sum, red);
        const float inv = 1.f / sqrtf(sum / (float)a.D + a.eps);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int64_t d = place(q, i);
            const bool in = inside(q, d), end = across(q, d);
            if (in || end) {
                float wv[VEC];
                if (!SHIFT && in) {
                    load_piece<T, VEC>(wv, wb + at_w[q] + d);
                } else {
#pragma unroll
                    for (int e = 0; e < VEC; ++e)
                        wv[e] = d + e >= 0 && d + e < a.D ? ld_f32(wb + at_w[q] + d + e) : 0.f;
                }
                const bool last = gb && !a.gate_first;
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float v = u[i][e] * inv * wv[e];
                    u[i][e] = last ? v * g[i][e] : v;
                }
                if (in) {
                    store_piece<T, VEC>(yb + dense[q] + d, u[i]);
                } else {
#pragma unroll
                    for (int e = 0; e < VEC; ++e)
                        if (d + e >= 0 && d + e < a.D) st_from_f32(yb + dense[q] + d + e, u[i][e]);
                }
            }
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

template <typename T, int VEC, bool SHIFT, int TPR, int NV, int RPG = 1>
cudaError_t launch_cfg(const NormArgs &a, cudaStream_t s) {
    constexpr int kRows = (TPR < 128 ? 128 / TPR : 1) * RPG;
    const int64_t rows = a.M * a.K, blocks = (rows + kRows - 1) / kRows;
    if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
    return launch_dependent(norm_kernel<T, VEC, TPR, NV, RPG, SHIFT>, (unsigned)blocks, TPR < 128 ? 128 : TPR, 0, s, a,
                            rows);
}

template <typename T, int VEC, bool SHIFT>
cudaError_t launch_v(const NormArgs &a, int sm_count, cudaStream_t s) {
    const int64_t n = (a.D + VEC - 1) / VEC + SHIFT;  // pieces per row
    // several rows per thread once there are enough rows to fill the SMs anyway
    const bool many = a.M * a.K >= (int64_t)(sm_count > 0 ? sm_count : 152) * 256;
    if (n <= 16) return many ? launch_cfg<T, VEC, SHIFT, 16, 1, 4>(a, s) : launch_cfg<T, VEC, SHIFT, 16, 1>(a, s);
    if (n <= 32) return many ? launch_cfg<T, VEC, SHIFT, 32, 1, 4>(a, s) : launch_cfg<T, VEC, SHIFT, 32, 1>(a, s);
    if (n <= 64) return many ? launch_cfg<T, VEC, SHIFT, 32, 2, 2>(a, s) : launch_cfg<T, VEC, SHIFT, 32, 2>(a, s);
    if (n <= 128) return launch_cfg<T, VEC, SHIFT, 128, 1>(a, s);
    if (n <= 256) return launch_cfg<T, VEC, SHIFT, 128, 2>(a, s);
    if (n <= 512) return launch_cfg<T, VEC, SHIFT, 256, 2>(a, s);
    if (n <= 1024) return launch_cfg<T, VEC, SHIFT, 512, 2>(a, s);
    if (n <= 2048) return launch_cfg<T, VEC, SHIFT, 512, 4>(a, s);
    if constexpr (VEC == 1) {
        if (n <= 8192) return launch_cfg<T, VEC, SHIFT, 512, 16>(a, s);
    }
    if (a.M * a.K > INT32_MAX) return cudaErrorInvalidConfiguration;
    return launch_dependent(norm_wide_kernel<T>, (unsigned)(a.M * a.K), 1024, 0, s, a);
}

template <typename T>
cudaError_t launch_t(const NormArgs &a, int sm_count, cudaStream_t s) {
    if (a.vec) return launch_v<T, 16 / sizeof(T), false>(a, sm_count, s);
    if (a.shift) return launch_v<T, 16 / sizeof(T), true>(a, sm_count, s);
    return launch_v<T, 1, false>(a, sm_count, s);
}

}  // namespace

cudaError_t launch_gated_norm(DType dt, const NormArgs &a, int sm_count, cudaStream_t s) {
    switch (dt) {
    case DType::F32: return launch_t<float>(a, sm_count, s);
    case DType::BF16: return launch_t<__nv_bfloat16>(a, sm_count, s);
    case DType::F16: return launch_t<__half>(a, sm_count, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace gdn
