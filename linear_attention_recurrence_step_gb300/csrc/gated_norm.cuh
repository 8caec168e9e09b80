// gated_norm.cuh -- root-mean-square norm with the gate and the residual sum
// around it:
//     u = x                      (gate first: u = x * silu(gate))
//     u = residual + scale * u   (with a residual; also written out)
//     y = u * rsqrt(mean(u^2) + eps) * weight      (gate last: * silu(gate))
//
// Bound by memory: x, gate and residual are read once, y and the new residual
// written once.  At ten operations per element the instruction rate is not far
// behind, so what is known at launch (gate, residual, dense rows) is known to
// the compiler, and pairs of elements share packed instructions.
//
// Measured: 4096 x 32 rows of 128 in bf16 with a gate 18.4 us (5.5 TB/s),
// 1000 rows of 5001 in f32 with a residual 16.6 us (4.8 TB/s; rows that
// straddle 16-byte boundaries), 16 x 32 rows 1.7 us.
//
// A row stays in registers between its sum and its scaling.  TPR threads share
// a row: eight of them a head of 128, a block a wide row; each holds NV pieces
// of 16 bytes of each of RPG rows, whose loads are in flight together.  The
// sum, the mean and the scaled values are f32; y and the residual are each
// rounded once, and the norm takes the unrounded sum.
#pragma once

#include "layer.h"
#include "pieces.cuh"

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

// How rows lie: whole 16-byte pieces; dense rows of another width (a row then
// starts `mis` elements past a 16-byte boundary: pieces are cut on those
// boundaries, and those at a row's ends go element by element); anything,
// element by element.
enum NormRows { kRowsWhole = 0, kRowsShifted = 1, kRowsAny = 2 };

template <typename T, int ROWS, int TPR, int NV, int RPG, bool GATE, bool RES>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR) norm_kernel(const NormArgs a, int64_t rows) {
    constexpr int VEC = ROWS == kRowsAny ? 1 : 16 / sizeof(T), NP = kPairs<VEC>;
    constexpr bool SHIFT = ROWS == kRowsShifted;
    constexpr int kGroups = TPR < 128 ? 128 / TPR : 1;
    static_assert(RPG == 1 || TPR <= 32, "several rows of a group only within a warp");
    __shared__ float red[32];
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x % TPR;
    const int64_t row0 = ((int64_t)blockIdx.x * kGroups + threadIdx.x / TPR) * RPG;
    const int D = (int)a.D;

    const T *px[RPG], *pg[RPG], *pw[RPG];
    int64_t dense[RPG];
    int mis[RPG];
#pragma unroll
    for (int q = 0; q < RPG; ++q) {
        const int64_t row = row0 + q;
        dense[q] = row * a.D;
        int64_t ox = dense[q], og = dense[q], ow = 0;
        if (a.K > 1) {  // (one head: the token stride is the row's)
            const int64_t m = row / a.K, k = row - m * a.K;
            ox = m * a.x_st + k * a.D;
            og = m * a.gate_st + k * a.D;
            if (a.weight_rows > 1) ow = k * a.D;
        } else {
            ox = row * a.x_st;
            og = row * a.gate_st;
        }
        px[q] = static_cast<const T *>(a.x) + ox;
        if (GATE) pg[q] = static_cast<const T *>(a.gate) + og;
        pw[q] = static_cast<const T *>(a.weight) + ow;
        mis[q] = SHIFT ? (int)(dense[q] & (VEC - 1)) : 0;
    }
    // first element of piece i of row q; whether the piece is inside the row,
    // or across one of its ends
    auto place = [&](int q, int i) { return (i * TPR + lane) * VEC - mis[q]; };
    auto inside = [&](int q, int d) { return row0 + q < rows && (!SHIFT || d >= 0) && d + VEC <= D; };
    auto across = [&](int q, int d) {
        return SHIFT && row0 + q < rows && d + VEC > 0 && d < D && (d < 0 || d + VEC > D);
    };
    RawPiece<T, VEC> xr[RPG][NV], gr[RPG][NV], rr[RPG][NV];
#pragma unroll
    for (int q = 0; q < RPG; ++q)
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int d = place(q, i);
            if (inside(q, d)) {
                xr[q][i] = load_raw<T, VEC>(px[q] + d);
                if (GATE) gr[q][i] = load_raw<T, VEC>(pg[q] + d);
                if (RES) rr[q][i] = load_raw<T, VEC>(static_cast<const T *>(a.residual) + dense[q] + d);
            } else if (across(q, d)) {
                // gather the elements that are the row's, zeros beside them
                alignas(16) T ex[VEC], eg[VEC], er[VEC];
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const bool there = d + e >= 0 && d + e < D;
                    ex[e] = there ? px[q][d + e] : Elem<T>::from_f32(0.f);
                    if (GATE) eg[e] = there ? pg[q][d + e] : Elem<T>::from_f32(0.f);
                    if (RES)
                        er[e] = there ? static_cast<const T *>(a.residual)[dense[q] + d + e] : Elem<T>::from_f32(0.f);
                }
                xr[q][i] = load_raw<T, VEC>(ex);
                if (GATE) gr[q][i] = load_raw<T, VEC>(eg);
                if (RES) rr[q][i] = load_raw<T, VEC>(er);
            }
        }
    auto put = [&](T *base, int q, int d, bool in, const float2 (&v)[NP]) {
        T *p = base + dense[q] + d;
        if (in) {
            store_piece2<T, VEC>(p, v);
        } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                if (d + e >= 0 && d + e < D) st_from_f32(p + e, e % 2 ? v[e / 2].y : v[e / 2].x);
        }
    };
#pragma unroll
    for (int q = 0; q < RPG; ++q) {
        float2 u[NV][NP], g[NV][NP];
        float2 part = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int d = place(q, i);
            const bool in = inside(q, d);
            if (!in && !across(q, d)) continue;
            widen2<T, VEC>(u[i], xr[q][i]);
            if (GATE) {
                widen2<T, VEC>(g[i], gr[q][i]);
#pragma unroll
                for (int e = 0; e < NP; ++e) g[i][e] = silu2(g[i][e]);
                if (a.gate_first)
#pragma unroll
                    for (int e = 0; e < NP; ++e) u[i][e] = fmul2(u[i][e], g[i][e]);
            }
            if (RES) {
                float2 rs[NP];
                widen2<T, VEC>(rs, rr[q][i]);
#pragma unroll
                for (int e = 0; e < NP; ++e) u[i][e] = ffma2(make_float2(a.scale, a.scale), u[i][e], rs[e]);
                put(static_cast<T *>(a.residual_out), q, d, in, u[i]);
            }
#pragma unroll
            for (int e = 0; e < NP; ++e) part = ffma2(u[i][e], u[i][e], part);
        }
        const float sum = row_sum<TPR>(part.x + part.y, red);
        const float inv = 1.f / sqrtf(sum / (float)D + a.eps);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int d = place(q, i);
            const bool in = inside(q, d);
            if (!in && !across(q, d)) continue;
            float2 w[NP];
            if (SHIFT) {  // the weight does not share the row's shift
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float v = in || (d + e >= 0 && d + e < D) ? ld_f32(pw[q] + d + e) : 0.f;
                    if (e % 2) w[e / 2].y = v;
                    else w[e / 2].x = v;
                }
            } else {
                widen2<T, VEC>(w, load_raw<T, VEC>(pw[q] + d));
            }
#pragma unroll
            for (int e = 0; e < NP; ++e) {
                const float2 v = fmul2(fmul2(u[i][e], make_float2(inv, inv)), w[e]);
                u[i][e] = GATE && !a.gate_first ? fmul2(v, g[i][e]) : v;
            }
            put(static_cast<T *>(a.y), q, d, in, u[i]);
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

template <typename T, int ROWS, bool GATE, bool RES, int TPR, int NV, int RPG = 1>
cudaError_t launch_cfg(const NormArgs &a, cudaStream_t s) {
    constexpr int kRows = (TPR < 128 ? 128 / TPR : 1) * RPG;
    const int64_t rows = a.M * a.K, blocks = (rows + kRows - 1) / kRows;
    if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
    return launch_dependent(norm_kernel<T, ROWS, TPR, NV, RPG, GATE, RES>, (unsigned)blocks, TPR < 128 ? 128 : TPR, 0, s,
                            a, rows);
}

template <typename T, int ROWS, bool GATE, bool RES>
cudaError_t launch_rows(const NormArgs &a, int sm_count, cudaStream_t s) {
    constexpr int VEC = ROWS == kRowsAny ? 1 : 16 / sizeof(T);
    const int64_t n = (a.D + VEC - 1) / VEC + (ROWS == kRowsShifted);  // pieces per row
    if constexpr (ROWS == kRowsWhole) {
        // Fewer threads per row, with more in flight each, once there are enough
        // rows to fill the SMs anyway: rows of 128 in bf16 with a gate take 18.6 us
        // so at 131072 rows (19.4 us with one piece per thread), 2.7 us at 512 rows
        // (1.9 us); 16384 rows of 512 take 11.6 us (10.4 us).
        const bool many = a.M * a.K >= (int64_t)(sm_count > 0 ? sm_count : 152) * 256;
        if (n <= 16)
            return many ? launch_cfg<T, ROWS, GATE, RES, 8, 2, 2>(a, s) : launch_cfg<T, ROWS, GATE, RES, 16, 1>(a, s);
        if (n <= 32)
            return many ? launch_cfg<T, ROWS, GATE, RES, 16, 2, 2>(a, s) : launch_cfg<T, ROWS, GATE, RES, 32, 1>(a, s);
        if (n <= 64)
            return many ? launch_cfg<T, ROWS, GATE, RES, 32, 2, 2>(a, s) : launch_cfg<T, ROWS, GATE, RES, 32, 2>(a, s);
    } else {
        if (n <= 32) return launch_cfg<T, ROWS, GATE, RES, 32, 1>(a, s);
    }
    if (n <= 128) return launch_cfg<T, ROWS, GATE, RES, 128, 1>(a, s);
    if constexpr (ROWS == kRowsWhole) {
        if (n <= 256) return launch_cfg<T, ROWS, GATE, RES, 128, 2>(a, s);
    }
    if (n <= 512) return launch_cfg<T, ROWS, GATE, RES, 256, 2>(a, s);
    if constexpr (ROWS == kRowsAny) {
        if (n <= 2048) return launch_cfg<T, ROWS, GATE, RES, 256, 8>(a, s);
        if (n <= 8192) return launch_cfg<T, ROWS, GATE, RES, 1024, 8>(a, s);
    } else {
        // (up to 1344 pieces by 448 threads: 4096 bf16 rows of 8192 with a gate take
        // 40.2 us so, 62.7 us by 512 threads of four pieces, and 43.0 and 42.2 us with
        // a residual instead; 1000 f32 rows of 5001 16.7 and 16.9 us)
        if (n <= 768) return launch_cfg<T, ROWS, GATE, RES, 256, 3>(a, s);
        if (n <= 1344) return launch_cfg<T, ROWS, GATE, RES, 448, 3>(a, s);
        if (n <= 2048) return launch_cfg<T, ROWS, GATE, RES, 512, 4>(a, s);
    }
    if (a.M * a.K > INT32_MAX) return cudaErrorInvalidConfiguration;
    return launch_dependent(norm_wide_kernel<T>, (unsigned)(a.M * a.K), 1024, 0, s, a);
}

template <typename T, int ROWS>
cudaError_t launch_gate(const NormArgs &a, int sm_count, cudaStream_t s) {
    if (a.gate)
        return a.residual ? launch_rows<T, ROWS, true, true>(a, sm_count, s)
                          : launch_rows<T, ROWS, true, false>(a, sm_count, s);
    return a.residual ? launch_rows<T, ROWS, false, true>(a, sm_count, s)
                      : launch_rows<T, ROWS, false, false>(a, sm_count, s);
}

template <typename T>
cudaError_t launch_norm(const NormArgs &a, int sm_count, cudaStream_t s) {
    if (a.vec) return launch_gate<T, kRowsWhole>(a, sm_count, s);
    if (a.shift) return launch_gate<T, kRowsShifted>(a, sm_count, s);
    return launch_gate<T, kRowsAny>(a, sm_count, s);
}

}  // namespace

}  // namespace gdn
