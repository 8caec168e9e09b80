// selective_scan.cu -- the selective state space scan, one scalar decay per
// head and step:
//     dl    = softplus(dt[b,t,h] + dt_bias[h])      (or dt + dt_bias)
//     s    <- exp(dl * A[h]) * s + (dl * x[b,t,h,p]) * B[b,t,g,:]
//     y     = s . C[b,t,g,:] + D[h] * x[b,t,h,p]
// for every state row s = state[b,h,p,:] (f32, N entries), g = h / (H/G).
//
// Step form (this file): a row's N entries lie in the registers of LR lanes,
// a lane holds VPL of them for each of RPL rows.  One call reads and writes
// the state once; the rows of up to kStage steps wait in shared memory.  A
// call of few steps is bound by the state's bytes: one step of 32 sequences with
// 32 heads of 128 x 128 takes 26.5 us (5.1 TB/s), 8 steps of 16 sequences 19.4 us
// (3.6 TB/s: 8 dependent steps with a sum over lanes each).  A long call with few
// heads is split along the steps: a first kernel folds every segment (the
// first from state_in, the others from zero) into its end state and its total
// decay, a second one joins these into the state after every segment, and a
// third one runs the segments from those.
#include "layer.h"
#include "pieces.cuh"
#include "tile.cuh"

namespace gdn {

namespace {

constexpr int kStage = 16;      // steps staged in shared memory at a time
constexpr int kScanWarps = 4;   // most warps per CTA

// SHORT (2 to 16 steps): half of the rows per lane, for more CTAs per SM while
// a CTA waits for its step's sums (16 sequences of 8 steps, 64 heads of 64 x
// 128: 19.5 us, 23.3 us without); one step alone has no such wait and is
// better off with the larger tile (32 sequences: 25.8 us, 26.5 us).
template <int N, bool SHORT> struct ScanShape {
    static constexpr int LR = N >= 32 ? 8 : 4;        // lanes per row
    static constexpr int VPL = N / LR;                // entries per lane and row
    static constexpr int RPL = (N >= 256 ? 2 : 4) / (SHORT && N >= 128 ? 2 : 1);  // rows per lane
    static constexpr int RW = 32 / LR;                // rows side by side in a warp
    static constexpr int kWarpRows = RW * RPL;
};

// Whether a kernel has room to copy a stage ahead.
__host__ __device__ constexpr bool scan_ahead(int N, bool SHORT) { return !SHORT && N <= 128; }

// workspace: end states [segments][B][H][P][N], then decays [segments][B][H]
template <typename T, int N, int phase, bool SHORT>
__global__ void __launch_bounds__(kScanWarps * 32)
scan_step_kernel(const ScanArgs a, const int64_t row_blocks) {
    using S = ScanShape<N, SHORT>;
    constexpr int LR = S::LR, VPL = S::VPL, RPL = S::RPL, RW = S::RW, WR = S::kWarpRows;
    constexpr int NV4 = VPL / 4;  // float4 groups per lane and row: entries j*4*LR + lane*4
    constexpr bool AHEAD = scan_ahead(N, SHORT);
    extern __shared__ __align__(16) unsigned char smem_raw[];
    const int warps = blockDim.x / 32, rows_cta = warps * WR;
    float *sB = reinterpret_cast<float *>(smem_raw);      // [kStage][N]
    float *sC = sB + kStage * N;                          // [kStage][N]
    float *sx = sC + kStage * N;                          // [kStage][rows_cta]: x
    float *sg = sx + kStage * rows_cta;                   // [kStage] decay
    float *sd = sg + kStage;                              // [kStage] step
    pdl_trigger();
    pdl_wait();

    const int64_t rb = blockIdx.x % row_blocks;
    int64_t rest = blockIdx.x / row_blocks;
    const int64_t h = rest % a.H;
    rest /= a.H;
    const int64_t b = rest % a.B;
    const int64_t seg = rest / a.B;
    const int64_t g = h / (a.H / a.G);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int sub = lane % LR, grp = lane / LR;
    const int64_t p0 = rb * rows_cta + warp * WR + grp;   // row of pass r: p0 + r * RW
    const int64_t tile = (b * a.H + h) * a.P * N;
    const int64_t tiles = a.B * a.H * a.P * N;

    int64_t len = a.T;
    if (a.lengths) {
        const int64_t n = a.lengths[b];
        len = n < 0 ? 0 : (n < a.T ? n : a.T);
    }
    const int64_t t_begin = seg * a.seg_steps;
    int64_t t_end = t_begin + a.seg_steps;
    if (t_end > len) t_end = len;

    // where the segment starts: the call's state, zeros, or the state after the
    // segment before it
    const float *from = seg == 0 ? a.state_in : phase == kScanOutput ? a.workspace + (seg - 1) * tiles : nullptr;
    float4 s[RPL][NV4];
#pragma unroll
    for (int r = 0; r < RPL; ++r) {
        const int64_t p = p0 + r * RW;
#pragma unroll
        for (int j = 0; j < NV4; ++j) {
            s[r][j] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (from && p < a.P)
                s[r][j] = *reinterpret_cast<const float4 *>(from + tile + p * N + j * 4 * LR + sub * 4);
        }
    }
    if (phase == kScanOutput && seg == 0 && a.state_out) {
        // the first segment writes the call's state: it alone reads state_in,
        // which may be the same buffer
        const float *last = a.workspace + (a.segments - 1) * tiles + tile;
#pragma unroll
        for (int r = 0; r < RPL; ++r) {
            const int64_t p = p0 + r * RW;
#pragma unroll
            for (int j = 0; j < NV4; ++j)
                if (p < a.P)
                    *reinterpret_cast<float4 *>(a.state_out + tile + p * N + j * 4 * LR + sub * 4) =
                        *reinterpret_cast<const float4 *>(last + p * N + j * 4 * LR + sub * 4);
        }
    }

    const float Ah = a.A[h], bias = a.dt_bias ? a.dt_bias[h] : 0.f, Dh = a.D ? a.D[h] : 0.f;
    const T *x = static_cast<const T *>(a.x) + b * a.x_sb + h * a.P;
    const T *dtp = static_cast<const T *>(a.dt) + b * a.dt_sb + h;
    const T *Bp = static_cast<const T *>(a.Bm) + b * a.b_sb + g * N;
    const T *Cp = static_cast<const T *>(a.Cm) + b * a.c_sb + g * N;
    const bool out = phase != kScanFold && a.y != nullptr;
    float decay = 1.f;

    // The next stage's rows are copied while this one is worked on, where whole
    // pieces can be (`ahead`); the step sizes go by a register.
    constexpr int VE = 16 / sizeof(T);
    const bool ahead = AHEAD && a.T > kStage && a.vec_bc && a.vec_x;
    T *const rB = reinterpret_cast<T *>(sd + kStage), *const rC = rB + kStage * N, *const rx = rC + kStage * N;
    float next_dt = 0.f;
    auto fetch = [&](int64_t t0) {
        const int n = (int)(t_end - t0 < kStage ? t_end - t0 : kStage);
        constexpr int PR = N / VE;
        for (int i = threadIdx.x; i < n * PR; i += blockDim.x) {
            const int t = i / PR, c = i % PR * VE;
            cp_async16(rB + t * N + c, Bp + (t0 + t) * a.b_st + c);
            if (out) cp_async16(rC + t * N + c, Cp + (t0 + t) * a.c_st + c);
        }
        const int px = rows_cta / VE;
        for (int i = threadIdx.x; i < n * px; i += blockDim.x) {
            const int t = i / px, p = i % px * VE;
            if (rb * rows_cta + p < a.P)
                cp_async16(rx + t * rows_cta + p, x + (t0 + t) * a.x_st + rb * rows_cta + p);
        }
        cp_async_commit();
        if (threadIdx.x < n) next_dt = ld_f32(dtp + (t0 + threadIdx.x) * a.dt_st);
    };
    if (ahead && t_begin < t_end) fetch(t_begin);

    for (int64_t t0 = t_begin; t0 < t_end; t0 += kStage) {
        const int n = (int)(t_end - t0 < kStage ? t_end - t0 : kStage);
        if (ahead) cp_async_wait_all();
        __syncthreads();
        float dt_now = next_dt;
        if (ahead) {
            for (int i = threadIdx.x * VE; i < n * N; i += blockDim.x * VE) {
                float v[VE];
                load_piece<T, VE>(v, rB + i);
#pragma unroll
                for (int e = 0; e < VE; e += 4)
                    *reinterpret_cast<float4 *>(sB + i + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
                if (out) {
                    load_piece<T, VE>(v, rC + i);
#pragma unroll
                    for (int e = 0; e < VE; e += 4)
                        *reinterpret_cast<float4 *>(sC + i + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
                }
            }
            for (int i = threadIdx.x * VE; i < n * rows_cta; i += blockDim.x * VE) {
                float v[VE];
                load_piece<T, VE>(v, rx + i);
                const bool in = rb * rows_cta + i % rows_cta < a.P;
#pragma unroll
                for (int e = 0; e < VE; e += 4)
                    *reinterpret_cast<float4 *>(sx + i + e) =
                        in ? make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
        } else {
            if (a.vec_bc) {
                constexpr int PR = N / VE;  // pieces of a row
                for (int i = threadIdx.x; i < n * PR; i += blockDim.x) {
                    const int t = i / PR, c = i % PR * VE;
                    const RawPiece<T, VE> rB = load_raw<T, VE>(Bp + (t0 + t) * a.b_st + c);
                    float v[VE];
                    if (out) {
                        const RawPiece<T, VE> rC = load_raw<T, VE>(Cp + (t0 + t) * a.c_st + c);
                        widen<T, VE>(v, rC);
#pragma unroll
                        for (int e = 0; e < VE; e += 4)
                            *reinterpret_cast<float4 *>(sC + t * N + c + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
                    }
                    widen<T, VE>(v, rB);
#pragma unroll
                    for (int e = 0; e < VE; e += 4)
                        *reinterpret_cast<float4 *>(sB + t * N + c + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
                }
            } else {
                for (int i = threadIdx.x; i < n * N; i += blockDim.x) {
                    const int t = i / N, c = i % N;
                    sB[i] = ld_f32(Bp + (t0 + t) * a.b_st + c);
                    if (out) sC[i] = ld_f32(Cp + (t0 + t) * a.c_st + c);
                }
            }
            for (int i = threadIdx.x; i < n * rows_cta; i += blockDim.x) {
                const int t = i / rows_cta, p = i % rows_cta;
                sx[i] = rb * rows_cta + p < a.P ? ld_f32(x + (t0 + t) * a.x_st + rb * rows_cta + p) : 0.f;
            }
            if (threadIdx.x < n) dt_now = ld_f32(dtp + (t0 + threadIdx.x) * a.dt_st);
        }
        if (threadIdx.x < n) {
            float d = dt_now + bias;
            if (a.softplus) d = fmaxf(d, 0.f) + log1pf(expf(-fabsf(d)));
            sd[threadIdx.x] = d;
            sg[threadIdx.x] = expf(d * Ah);
        }
        __syncthreads();
        if (ahead && t0 + kStage < t_end) fetch(t0 + kStage);
        for (int t = 0; t < n; ++t) {
            const float gt = sg[t], dl = sd[t];
            decay *= gt;
            float xv[RPL];
            float2 acc2[RPL];
#pragma unroll
            for (int r = 0; r < RPL; ++r) {
                xv[r] = dl * sx[t * rows_cta + warp * WR + grp + r * RW];
                acc2[r] = make_float2(0.f, 0.f);
            }
#pragma unroll
            for (int j = 0; j < NV4; ++j) {
                const float4 Bv = *reinterpret_cast<const float4 *>(sB + t * N + j * 4 * LR + sub * 4);
                float4 Cv = make_float4(0.f, 0.f, 0.f, 0.f);
                if (out) Cv = *reinterpret_cast<const float4 *>(sC + t * N + j * 4 * LR + sub * 4);
#pragma unroll
                for (int r = 0; r < RPL; ++r) {
                    const float2 dx2 = make_float2(xv[r], xv[r]), g2 = make_float2(gt, gt);
                    const float2 lo = ffma2(g2, lo2(s[r][j]), fmul2(dx2, lo2(Bv)));
                    const float2 hi = ffma2(g2, hi2(s[r][j]), fmul2(dx2, hi2(Bv)));
                    s[r][j] = cat4(lo, hi);
                    if (out) acc2[r] = ffma2(hi, hi2(Cv), ffma2(lo, lo2(Cv), acc2[r]));
                }
            }
            if (out) {
                // the lanes of a row share its sum out: half of the rows go to
                // each side until a lane holds one row, then plain exchanges
                float acc[RPL];
#pragma unroll
                for (int r = 0; r < RPL; ++r) acc[r] = acc2[r].x + acc2[r].y;
                int row = 0, left = RPL;
#pragma unroll
                for (int o = LR / 2; o > 0; o >>= 1) {
                    if (left > 1) {
                        const int half = left / 2;
                        const bool up = (sub & o) != 0;
#pragma unroll
                        for (int i = 0; i < RPL / 2; ++i)
                            if (i < half) {
                                const float send = up ? acc[i] : acc[i + half];
                                const float keep = up ? acc[i + half] : acc[i];
                                acc[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
                            }
                        row += up ? half : 0;
                        left = half;
                    } else {
                        acc[0] += __shfl_xor_sync(0xffffffffu, acc[0], o);
                    }
                }
                if constexpr (RPL > LR) static_assert(RPL <= LR, "a lane ends with one row");
                const int64_t p = p0 + row * RW;
                const bool writer = (sub & (LR / RPL - 1)) == 0;
                if (writer && p < a.P) {
                    const float xr = sx[t * rows_cta + warp * WR + grp + row * RW];
                    st_from_f32(static_cast<T *>(a.y) + ((b * a.T + t0 + t) * a.H + h) * a.P + p,
                                fmaf(Dh, xr, acc[0]));
                }
            }
        }
    }

    if (phase == kScanOutput) return;
    float *dst = phase == kScanFold ? a.workspace + seg * tiles : a.state_out;
    if (dst) {
#pragma unroll
        for (int r = 0; r < RPL; ++r) {
            const int64_t p = p0 + r * RW;
            if (p < a.P)
#pragma unroll
                for (int j = 0; j < NV4; ++j)
                    *reinterpret_cast<float4 *>(dst + tile + p * N + j * 4 * LR + sub * 4) = s[r][j];
        }
    }
    if (phase == kScanFold && rb == 0 && threadIdx.x == 0)
        a.workspace[(int64_t)a.segments * tiles + (seg * a.B + b) * a.H + h] = decay;
}

// The segments' end states and decays, joined in place: slot i becomes the
// state after segment i.  The last one goes to `state_out` too when that is
// given (calls without y).
__global__ void __launch_bounds__(256) scan_join_kernel(float *ws, float *state_out, int segments, int64_t tiles,
                                                        int64_t heads, int64_t per_head) {
    pdl_trigger();
    pdl_wait();
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (i >= tiles) return;
    const float *dec = ws + (int64_t)segments * tiles + i / per_head;
    float4 v = *reinterpret_cast<const float4 *>(ws + i);
#pragma unroll 4
    for (int k = 1; k < segments; ++k) {
        const float d = dec[k * heads];
        float4 *slot = reinterpret_cast<float4 *>(ws + k * tiles + i);
        const float4 e = *slot;
        v.x = fmaf(d, v.x, e.x);
        v.y = fmaf(d, v.y, e.y);
        v.z = fmaf(d, v.z, e.z);
        v.w = fmaf(d, v.w, e.w);
        *slot = v;
    }
    if (state_out) *reinterpret_cast<float4 *>(state_out + i) = v;
}

template <int N, bool SHORT> int64_t scan_warps(int64_t P, int64_t *row_blocks) {
    constexpr int WR = ScanShape<N, SHORT>::kWarpRows;
    const int64_t w = (P + WR - 1) / WR;
    *row_blocks = (w + kScanWarps - 1) / kScanWarps;
    return (w + *row_blocks - 1) / *row_blocks;
}

template <typename T, int N, int PHASE, bool SHORT>
cudaError_t launch_phase(const ScanArgs &a, cudaStream_t s) {
    int64_t row_blocks;
    const int warps = (int)scan_warps<N, SHORT>(a.P, &row_blocks);
    const size_t row = 2 * N + warps * ScanShape<N, SHORT>::kWarpRows;  // of B, C and x
    const size_t smem = kStage * ((row + 2) * 4 + (scan_ahead(N, SHORT) ? row * sizeof(T) : 0));
    const int64_t ctas = a.B * a.H * row_blocks * a.segments;
    if (ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
    return launch_dependent(scan_step_kernel<T, N, PHASE, SHORT>, (unsigned)ctas, warps * 32, smem, s, a, row_blocks);
}

template <typename T, int N>
cudaError_t launch_n(const ScanArgs &a, cudaStream_t s) {
    if (a.segments == 1)
        return a.T > 1 && a.T <= kStage ? launch_phase<T, N, kScanWhole, true>(a, s) : launch_phase<T, N, kScanWhole, false>(a, s);
    cudaError_t e = launch_phase<T, N, kScanFold, false>(a, s);
    if (e == cudaSuccess) e = launch_scan_join(a, s);
    if (e != cudaSuccess || !a.y) return e;
    return launch_phase<T, N, kScanOutput, false>(a, s);
}

template <typename T>
cudaError_t launch_t(const ScanArgs &a, cudaStream_t s) {
    switch (a.N) {
    case 16: return launch_n<T, 16>(a, s);
    case 32: return launch_n<T, 32>(a, s);
    case 64: return launch_n<T, 64>(a, s);
    case 128: return launch_n<T, 128>(a, s);
    case 256: return launch_n<T, 256>(a, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_scan_join(const ScanArgs &a, cudaStream_t s) {
    const int64_t per_head = a.P * a.N, tiles = a.B * a.H * per_head, blocks = (tiles + 1023) / 1024;
    if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
    return launch_dependent(scan_join_kernel, (unsigned)blocks, 256, 0, s, a.workspace,
                            a.y ? (float *)nullptr : a.state_out, a.segments, tiles, a.B * a.H, per_head);
}

bool scan_supported_n(int64_t N) { return N == 16 || N == 32 || N == 64 || N == 128 || N == 256; }

// From one whole chunk on: 16 sequences of 32 steps, 32 heads of 128 x 128, take
// 27.0 us in chunks, 48.2 us by steps; one sequence 8.4 and 13.6 us.
bool scan_chunk_sizes(DType dt, int64_t T, int64_t P, int64_t N) {
    return dt == DType::BF16 && (N == 64 || N == 128) && P % 8 == 0 && T >= 32;
}

ScanPlan scan_plan(int64_t B, int64_t T, int64_t H, int64_t P, int64_t N, bool chunked) {
    ScanPlan plan{1, T, 0};
    int64_t row_blocks = 1;
    // CTAs that fill 152 SMs, and the fewest steps of a segment (128 instead of
    // 64 at 512 steps of 32 heads of 128 x 128: 49 us instead of 35 in the chunk
    // form, 161 instead of 93 by steps)
    double target = 608.0;
    const int64_t least = 64;
    int64_t unit = kStage;
    if (chunked) {
        // sixteen warps per SM
        target = 152.0 * (16 / scan_chunk_warps(P, &row_blocks));
        unit = 32;
    } else {
        switch (N) {
        case 16: scan_warps<16, false>(P, &row_blocks); break;
        case 32: scan_warps<32, false>(P, &row_blocks); break;
        case 64: scan_warps<64, false>(P, &row_blocks); break;
        case 128: scan_warps<128, false>(P, &row_blocks); break;
        case 256: scan_warps<256, false>(P, &row_blocks); break;
        }
    }
    const double ctas = (double)B * (double)H * (double)row_blocks;
    int64_t want = ctas >= target ? 1 : (int64_t)(target / ctas);
    if (want > T / least) want = T / least;
    // Three kernels instead of one pay for themselves from 256 steps on in the
    // chunk form (one sequence, 32 heads of 128 x 128: 31.3 us split in four, 31.8 us
    // whole; 26 and 18.4 us at 128 steps, 35 and 59 us at 512).
    if (chunked && T < 256) want = 1;
    if (want > 64) want = 64;
    if (want > 1) {
        const int64_t steps = ((T + want - 1) / want + unit - 1) / unit * unit;
        plan.segments = (int)((T + steps - 1) / steps);
        plan.seg_steps = steps;
    }
    if (plan.segments > 1) {
        int64_t n = 4;
        for (int64_t d : {(int64_t)plan.segments, B, H})
            if (__builtin_mul_overflow(n, d, &n)) return ScanPlan{0, 0, -1};
        const int64_t decays = n;
        for (int64_t d : {P, N})
            if (__builtin_mul_overflow(n, d, &n)) return ScanPlan{0, 0, -1};
        if (__builtin_add_overflow(n, decays, &plan.bytes)) return ScanPlan{0, 0, -1};
    }
    return plan;
}

cudaError_t launch_selective_scan(DType dt, const ScanArgs &a, int, cudaStream_t s) {
    if (a.chunked) return launch_scan_chunk(a, s);
    switch (dt) {
    case DType::F32: return launch_t<float>(a, s);
    case DType::BF16: return launch_t<__nv_bfloat16>(a, s);
    case DType::F16: return launch_t<__half>(a, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace gdn
