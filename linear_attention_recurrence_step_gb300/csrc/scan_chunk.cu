// scan_chunk.cu -- the selective scan over long calls in chunks of L = 32
// steps on the tensor cores (warp-level mma.sync, bf16 operands, f32
// accumulate).  bf16 inputs, f32 state, N = 64 or 128.
//
// Within a chunk, with c_t the sum of the logarithms of the decays up to and
// including step t, and S the state (rows p, columns n) the chunk starts from,
//     y_t = exp(c_t) S C_t + sum_{s<=t} W[t][s] x_s + D x_t,
//           W[t][s] = (C_t . B_s) exp(c_t - c_s) dl_s
//     S  <- exp(c_L) S + sum_s x_s (exp(c_L - c_s) dl_s) B_s^T
// so a chunk is four products: C B^T (L x L x N), S C^T (P x L x N), x^T W^T
// (P x L x L, the half below the diagonal) and x^T B (P x N x L).
//
// A CTA owns up to 128 rows p of one head and walks the chunks of its segment
// in order.  A warp owns 16 rows: their state stays in its registers as the
// f32 accumulator of the last product, and is, in the same registers, the left
// operand of the second, so the state never goes through shared memory.  The
// next chunk's rows of x, B and C arrive by cp.async meanwhile.
//
// Precision: x, B and C enter as they are (bf16).  The weighted x, which goes
// into the state, enters as three bf16 terms (24 significant bits: f32's own),
// and the state is only ever scaled and added to in f32; W enters as three
// terms too.  Two terms are taken where it costs most and only y sees it: the
// state as an operand of y (its third term would cost 12 us of the 134 below),
// and the weighted x in the second pass over a split call (11 us).  Two terms
// are off by 2^-17 of a value at most, so the part of y that comes through the
// state is off by 2^-17 of its terms, 2^-16 in a split call, where rounding y
// to bf16 costs 2^-9.  (W in two terms saved 3 us and moved one y in 1700 to
// its neighbour.)  c_t is summed in f64 and kept as two f32 terms, so that
// exp(c_t - c_s) loses nothing to a chunk's large |c|.
//
// A call with few heads is split along the steps as in selective_scan.cu: a
// first pass forms the segments' end states (the last product alone), and the
// output pass starts every segment from the state after the one before it.
//
// Measured (one sequence of 4096 steps, 32 heads of 128 x 128): 134 us, of
// which the first pass takes 50, the join 9 and the output pass 75; the step
// form takes 614 us on f32 inputs of that size.  Chunks of 64 steps, one CTA
// per SM, took 139 us: more of the products lies above the diagonal and nothing
// else runs while a CTA waits for its W.  What bounds it: the warps' issue of
// about 150 mma.sync (190 in a call that is not split) and their operand loads
// per chunk (tensor pipe 45 % of its cycles, issue slots 44 %), between the
// barriers around W and the decays.
#include "layer.h"
#include "pieces.cuh"
#include "record_mma.cuh"

namespace gdn {

namespace {

constexpr int kL = 32;               // steps of a chunk
constexpr int kWPitch = kL + 8;      // elements between rows of W in shared memory

struct ChunkDecay {
    float2 c[kL];      // c_t in units of log(2), two terms
    float dl[kL];
    float w[kL];       // exp(c_L - c_t) dl_t
    float ec[kL];      // exp(c_t)
    float total;       // exp(c_L)
    float pad[3];
};

__host__ __device__ constexpr int bc_pitch(int N) { return N + 8; }
__host__ __device__ constexpr int x_pitch(int warps) { return warps * 16 + 8; }

// Shared memory (bytes): two stages of x, B, C; W (hi, mid, lo); two decay blocks;
// y tiles, unless they fit over a stage's C
__host__ __device__ constexpr size_t stage_bytes(int N, int warps) {
    return (size_t)kL * (x_pitch(warps) + 2 * bc_pitch(N)) * 2;
}
__host__ __device__ constexpr bool y_over_c(int N, int warps) { return warps * kL * 16 <= kL * bc_pitch(N); }
__host__ __device__ constexpr size_t chunk_smem(int N, int warps) {
    return 2 * stage_bytes(N, warps) + 3 * (size_t)kL * kWPitch * 2 + 2 * sizeof(ChunkDecay) +
           (y_over_c(N, warps) ? 0 : (size_t)warps * kL * 16 * 2);
}

// (Shared memory goes by 32-bit addresses here: a generic pointer per ldmatrix
// costs more instructions than the product it feeds.)
__device__ __forceinline__ void stsm_x4_t(uint32_t a, const uint32_t (&r)[4]) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};\n" ::"r"(a), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3])
                 : "memory");
}
__device__ __forceinline__ void put_pair(uint32_t a, uint32_t v) {
    asm volatile("st.shared.u32 [%0], %1;\n" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ uint4 get_piece(uint32_t a) {
    uint4 w;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];\n"
                 : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                 : "r"(a)
                 : "memory");
    return w;
}
// 16 bytes, or zeros.
__device__ __forceinline__ void cp_async16_or_zero(uint32_t s, const void *gmem, bool on) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(s), "l"(gmem), "r"(on ? 16 : 0) : "memory");
}
// (x0, x1) ~ hi + mid + lo in packed bf16 pairs: all 24 bits of the f32 values.
__device__ __forceinline__ void split3(float x0, float x1, uint32_t &hi, uint32_t &mid, uint32_t &lo) {
    hi = pack2<__nv_bfloat16>(x0, x1);
    const float2 h = unpack2<__nv_bfloat16>(hi);
    split_bf16x2(x0 - h.x, x1 - h.y, mid, lo);
}
// OUT: y is wanted (else only the state: the first pass, and calls without y).
template <int N, bool OUT, int PHASE>
__global__ void __launch_bounds__(256, 2) scan_chunk_kernel(const ScanArgs a, const int64_t row_blocks) {
    constexpr int TERMS = PHASE == kScanOutput ? 2 : 3;
    using T = __nv_bfloat16;
    constexpr int NT = N / 8;              // 8-column tiles of the state
    constexpr int BP = bc_pitch(N);
    extern __shared__ __align__(16) unsigned char smem_raw[];
    const int warps = blockDim.x / 32, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int XP = x_pitch(warps);
    const uint32_t stage = (uint32_t)stage_bytes(N, warps);
    const uint32_t smem = static_cast<uint32_t>(__cvta_generic_to_shared(smem_raw));
    const uint32_t sW = smem + 2 * stage;                               // hi, mid, lo
    constexpr uint32_t kWBytes = kL * kWPitch * 2;
    ChunkDecay *const sdec = reinterpret_cast<ChunkDecay *>(smem_raw + 2 * stage + 3 * kWBytes);
    const uint32_t sYown = sW + 3 * kWBytes + 2 * (uint32_t)sizeof(ChunkDecay);
    auto sx = [&](int b) { return smem + b * stage; };
    auto sB = [&](int b) { return sx(b) + kL * XP * 2; };
    auto sC = [&](int b) { return sB(b) + kL * BP * 2; };
    pdl_trigger();
    pdl_wait();

    const int64_t rb = blockIdx.x % row_blocks;
    int64_t rest = blockIdx.x / row_blocks;
    const int64_t h = rest % a.H;
    rest /= a.H;
    const int64_t b = rest % a.B;
    const int64_t seg = rest / a.B;
    const int64_t g = h / (a.H / a.G);
    const int64_t p_cta = rb * warps * 16;              // first row of the CTA
    const int rows = (int)(a.P - p_cta < warps * 16 ? a.P - p_cta : warps * 16);
    const int64_t tile = (b * a.H + h) * a.P * N, tiles = a.B * a.H * a.P * N;
    const int gr = lane >> 2, tq = lane & 3;            // accumulator row and column pair

    int64_t len = a.T;
    if (a.lengths) {
        const int64_t n = a.lengths[b];
        len = n < 0 ? 0 : (n < a.T ? n : a.T);
    }
    const int64_t t_begin = seg * a.seg_steps;
    const int64_t t_end = t_begin + a.seg_steps < len ? t_begin + a.seg_steps : len;
    const int chunks = t_end > t_begin ? (int)((t_end - t_begin + kL - 1) / kL) : 0;

    const T *const x = static_cast<const T *>(a.x) + b * a.x_sb + h * a.P + p_cta;
    const T *const dtp = static_cast<const T *>(a.dt) + b * a.dt_sb + h;
    const T *const Bp = static_cast<const T *>(a.Bm) + b * a.b_sb + g * N;
    const T *const Cp = static_cast<const T *>(a.Cm) + b * a.c_sb + g * N;
    const float A2 = a.A[h] * 1.44269504088896341f, bias = a.dt_bias ? a.dt_bias[h] : 0.f, Dh = a.D ? a.D[h] : 0.f;

    // rows past the end, and columns past the head, are zeros; an x row has two
    // 16-byte pieces per warp, so the CTA copies 16 rows at a time
    auto fetch = [&](int c) {
        const int64_t t0 = t_begin + (int64_t)c * kL;
        const int buf = c & 1, n = (int)(t_end - t0 < kL ? t_end - t0 : kL);
        {
            const int t = threadIdx.x / (warps * 2), q = threadIdx.x % (warps * 2) * 8;
            const T *src = x + (t0 + t) * a.x_st + q;
#pragma unroll
            for (int i = 0; i < kL / 16; ++i) {
                const bool on = q < rows && t + 16 * i < n;
                cp_async16_or_zero(sx(buf) + ((t + 16 * i) * XP + q) * 2, on ? src + 16 * i * a.x_st : x, on);
            }
        }
        for (int i = threadIdx.x; i < kL * (N / 8); i += blockDim.x) {
            const int t = i / (N / 8), q = i % (N / 8);
            const bool on = t < n;
            cp_async16_or_zero(sB(buf) + (t * BP + q * 8) * 2, on ? Bp + (t0 + t) * a.b_st + q * 8 : Bp, on);
            if (OUT) cp_async16_or_zero(sC(buf) + (t * BP + q * 8) * 2, on ? Cp + (t0 + t) * a.c_st + q * 8 : Cp, on);
        }
        cp_async_commit();
    };
    // the decays of a chunk, by one warp, a step per lane: the last two warps in
    // turn, which have the least to do for W; each has read its next steps'
    // sizes by then
    auto step_size = [&](int c) {
        const int64_t t = t_begin + (int64_t)c * kL + lane;
        return t < t_end ? ld_f32(dtp + t * a.dt_st) : 0.f;
    };
    auto decay_warp = [&](int c) { return warps > 1 ? warps - 1 - (c & 1) : 0; };
    float next_size = 0.f;
    auto decays = [&](int c) {
        const int64_t t = t_begin + (int64_t)c * kL + lane;
        ChunkDecay &d = sdec[c & 1];
        // (steps past the end have no size, and no decay whatever the rate)
        float dl = 0.f, l2 = 0.f;
        const float size = next_size;
        next_size = step_size(c + (warps > 1 ? 2 : 1));
        if (t < t_end) {
            const float v = size + bias;
            dl = a.softplus ? fmaxf(v, 0.f) + log1pf(expf(-fabsf(v))) : v;
            l2 = dl * A2;
        }
        // a decay below 2^-256 is zero in f32
        double ct = l2 < -256.f ? -256.0 : (double)l2;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const double v = __shfl_up_sync(0xffffffffu, ct, o);
            if (lane >= o) ct += v;
        }
        const double last = __shfl_sync(0xffffffffu, ct, 31);
        const float hi = (float)ct;
        d.c[lane] = make_float2(hi, (float)(ct - (double)hi));
        d.dl[lane] = dl;
        d.w[lane] = ex2f((float)(last - ct)) * dl;
        d.ec[lane] = ex2f(hi);
        if (lane == 0) d.total = ex2f((float)last);
    };

    // the state of the warp's rows, accumulator tiles of 16 x 8: the call's
    // state, zeros, or the state after the segment before this one
    float S[NT][4];
    {
        const float *from = seg == 0 ? a.state_in : PHASE == kScanOutput ? a.workspace + (seg - 1) * tiles : nullptr;
        // the first segment writes the call's state: it alone reads state_in,
        // which may be the same buffer
        const bool hand_on = PHASE == kScanOutput && seg == 0 && a.state_out;
        const float *last = a.workspace + (a.segments - 1) * tiles;
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int pr = warp * 16 + gr + 8 * r;
                const int64_t off = tile + (p_cta + pr) * N + j * 8 + tq * 2;
                float2 v = make_float2(0.f, 0.f);
                if (from && pr < rows) v = *reinterpret_cast<const float2 *>(from + off);
                S[j][2 * r] = v.x;
                S[j][2 * r + 1] = v.y;
                if (hand_on && pr < rows)
                    *reinterpret_cast<float2 *>(a.state_out + off) = *reinterpret_cast<const float2 *>(last + off);
            }
    }

    float decay = 1.f;
    const int lr = lane & 7, lm = lane >> 3;            // ldmatrix: row and matrix of this lane's address
    if (chunks > 0) {
        fetch(0);
        if (warp == decay_warp(0)) {
            next_size = step_size(0);
            decays(0);
        } else if (warp == decay_warp(1)) {
            next_size = step_size(1);
        }
    }
    for (int c = 0; c < chunks; ++c) {
        const int buf = c & 1;
        cp_async_wait_all();
        __syncthreads();
        if (c + 1 < chunks) {
            fetch(c + 1);
            if (warp == decay_warp(c + 1)) decays(c + 1);
        }
        const ChunkDecay &d = sdec[buf];
        // where this lane's ldmatrix rows start: plain tiles of B and C (rows
        // across matrices 0-1 or 2-3), and transposed ones of x and B
        const uint32_t Bs = sB(buf), Cs = sC(buf);
        const uint32_t c_rows = Cs + ((lr + 8 * (lm & 1)) * BP + 8 * (lm >> 1)) * 2;   // left operand
        const uint32_t c_cols = Cs + ((lr + 8 * (lm >> 1)) * BP + 8 * (lm & 1)) * 2;   // right operand
        const uint32_t w_cols = sW + ((lr + 8 * (lm >> 1)) * kWPitch + 8 * (lm & 1)) * 2;
        const uint32_t x_t = sx(buf) + ((lr + 8 * (lm >> 1)) * XP + warp * 16 + 8 * (lm & 1)) * 2;
        const uint32_t b_t = Bs + ((lr + 8 * (lm & 1)) * BP + 8 * (lm >> 1)) * 2;
        float Y[kL / 8][4];
        if constexpr (OUT) {
            // W by tiles of 16 rows t and 8 columns s, those below the diagonal
            for (int job = warp; job < 6; job += warps) {
                const int ti = job < 4 ? 1 : 0, sb = job < 4 ? job : job - 4;
                float G[4] = {0.f, 0.f, 0.f, 0.f};
                const uint32_t b_row = Bs + ((sb * 8 + lr) * BP + 8 * lm) * 2, c_row = c_rows + ti * 16 * BP * 2;
#pragma unroll
                for (int kk = 0; kk < N / 16; kk += 2) {
                    uint32_t ca[4], bb[4];
                    ldsm_x4_a(bb, b_row + kk * 32);
                    ldsm_x4_a(ca, c_row + kk * 32);
                    mma_bf16_16816(G, ca, bb[0], bb[1]);
                    ldsm_x4_a(ca, c_row + kk * 32 + 32);
                    mma_bf16_16816(G, ca, bb[2], bb[3]);
                }
                const int t0 = ti * 16 + gr, s0 = sb * 8 + tq * 2;
                const float2 cs0 = d.c[s0], cs1 = d.c[s0 + 1];
                const float dl0 = d.dl[s0], dl1 = d.dl[s0 + 1];
                auto wt = [&](float gv, const float2 &ct, const float2 &cs, float dl, int t, int st) {
                    if (st > t) return 0.f;
                    const float w = gv * ex2f((ct.x - cs.x) + (ct.y - cs.y)) * dl;
                    return st == t ? w + Dh : w;
                };
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int t = t0 + 8 * r;
                    const float2 ct = d.c[t];
                    uint32_t hi, mid, lo;
                    split3(wt(G[2 * r], ct, cs0, dl0, t, s0), wt(G[2 * r + 1], ct, cs1, dl1, t, s0 + 1), hi, mid,
                           lo);
                    put_pair(sW + (t * kWPitch + s0) * 2, hi);
                    put_pair(sW + kWBytes + (t * kWPitch + s0) * 2, mid);
                    put_pair(sW + 2 * kWBytes + (t * kWPitch + s0) * 2, lo);
                }
            }
            // S C^T: the state's accumulators are the left operand
#pragma unroll
            for (int j = 0; j < kL / 8; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) Y[j][e] = 0.f;
#pragma unroll
            for (int kk = 0; kk < N / 16; ++kk) {
                uint32_t hi[4], lo[4];
                split_bf16x2(S[2 * kk][0], S[2 * kk][1], hi[0], lo[0]);
                split_bf16x2(S[2 * kk][2], S[2 * kk][3], hi[1], lo[1]);
                split_bf16x2(S[2 * kk + 1][0], S[2 * kk + 1][1], hi[2], lo[2]);
                split_bf16x2(S[2 * kk + 1][2], S[2 * kk + 1][3], hi[3], lo[3]);
#pragma unroll
                for (int j = 0; j < kL / 8; j += 2) {
                    uint32_t cb[4];
                    ldsm_x4_a(cb, c_cols + (j * 8 * BP + kk * 16) * 2);
                    mma_bf16_16816(Y[j], hi, cb[0], cb[1]);
                    mma_bf16_16816(Y[j + 1], hi, cb[2], cb[3]);
                    mma_bf16_16816(Y[j], lo, cb[0], cb[1]);
                    mma_bf16_16816(Y[j + 1], lo, cb[2], cb[3]);
                }
            }
#pragma unroll
            for (int j = 0; j < kL / 8; ++j) {
                const float2 e = *reinterpret_cast<const float2 *>(&d.ec[j * 8 + tq * 2]);
                Y[j][0] *= e.x;
                Y[j][1] *= e.y;
                Y[j][2] *= e.x;
                Y[j][3] *= e.y;
            }
        }
        {
            const float total = d.total;
            decay *= total;
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) S[j][e] *= total;
        }
        if (OUT) __syncthreads();  // W is whole; no warp reads this stage's C any more
#pragma unroll
        for (int ks = 0; ks < kL / 16; ++ks) {
            // x^T, rows p of this warp, 16 steps
            uint32_t xa[4];
            ldsm_x4_t_a(xa, x_t + ks * 16 * XP * 2);
            if constexpr (OUT) {
#pragma unroll
                for (int j = 2 * ks; j < kL / 8; j += 2) {
                    uint32_t wb[4];
#pragma unroll
                    for (int k = 2; k >= 0; --k) {  // lo first
                        ldsm_x4_a(wb, w_cols + k * kWBytes + (j * 8 * kWPitch + ks * 16) * 2);
                        mma_bf16_16816(Y[j], xa, wb[0], wb[1]);
                        mma_bf16_16816(Y[j + 1], xa, wb[2], wb[3]);
                    }
                }
            }
            // weighted by w_t
            uint32_t hi[4], mid[4], lo[4];
            const float2 w0 = *reinterpret_cast<const float2 *>(&d.w[ks * 16 + tq * 2]);
            const float2 w1 = *reinterpret_cast<const float2 *>(&d.w[ks * 16 + 8 + tq * 2]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 v = unpack2<T>(xa[i]), w = i < 2 ? w0 : w1;
                if (TERMS == 3) split3(v.x * w.x, v.y * w.y, hi[i], mid[i], lo[i]);
                else split_bf16x2(v.x * w.x, v.y * w.y, hi[i], mid[i]);
            }
#pragma unroll
            for (int j = 0; j < NT; j += 2) {
                uint32_t bb[4];
                ldsm_x4_t_a(bb, b_t + (ks * 16 * BP + j * 8) * 2);
                if (TERMS == 3) {
                    mma_bf16_16816(S[j], lo, bb[0], bb[1]);
                    mma_bf16_16816(S[j + 1], lo, bb[2], bb[3]);
                }
                mma_bf16_16816(S[j], mid, bb[0], bb[1]);
                mma_bf16_16816(S[j + 1], mid, bb[2], bb[3]);
                mma_bf16_16816(S[j], hi, bb[0], bb[1]);
                mma_bf16_16816(S[j + 1], hi, bb[2], bb[3]);
            }
        }
        if constexpr (OUT) {
            // y: the warp's 16 rows turned into 32 rows of 16 (32 bytes; the two
            // 16-byte halves swap places every fourth row against bank conflicts)
            const uint32_t ys = (y_over_c(N, warps) ? Cs : sYown) + warp * kL * 32;
#pragma unroll
            for (int j = 0; j < kL / 8; j += 2) {
                uint32_t r[4];
                r[0] = pack2<T>(Y[j][0], Y[j][1]);
                r[1] = pack2<T>(Y[j][2], Y[j][3]);
                r[2] = pack2<T>(Y[j + 1][0], Y[j + 1][1]);
                r[3] = pack2<T>(Y[j + 1][2], Y[j + 1][3]);
                const int t = (j + (lm >> 1)) * 8 + lr;
                stsm_x4_t(ys + t * 32 + ((lm & 1) ^ ((t >> 2) & 1)) * 16, r);
            }
            __syncwarp();
            const int64_t t0 = t_begin + (int64_t)c * kL;
            const int n = (int)(t_end - t0 < kL ? t_end - t0 : kL);
            const int q = lane & 1;
            T *y = static_cast<T *>(a.y) + ((b * a.T + t0) * a.H + h) * a.P + p_cta + warp * 16 + q * 8;
#pragma unroll
            for (int i = 0; i < kL / 16; ++i) {
                const int t = i * 16 + (lane >> 1);
                if (t < n && warp * 16 + q * 8 < rows)
                    *reinterpret_cast<uint4 *>(y + (int64_t)t * a.H * a.P) =
                        get_piece(ys + t * 32 + (q ^ ((t >> 2) & 1)) * 16);
            }
        }
    }

    if (PHASE == kScanOutput) return;
    float *dst = PHASE == kScanFold ? a.workspace + seg * tiles : a.state_out;
    if (dst) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int pr = warp * 16 + gr + 8 * r;
                if (pr < rows)
                    *reinterpret_cast<float2 *>(dst + tile + (p_cta + pr) * N + j * 8 + tq * 2) =
                        make_float2(S[j][2 * r], S[j][2 * r + 1]);
            }
    }
    if (PHASE == kScanFold && rb == 0 && threadIdx.x == 0)
        a.workspace[(int64_t)a.segments * tiles + (seg * a.B + b) * a.H + h] = decay;
}

template <int N, bool OUT, int PHASE>
cudaError_t launch_phase(const ScanArgs &a, int64_t ctas, int warps, int64_t row_blocks, cudaStream_t s) {
    const size_t smem = chunk_smem(N, warps);
    const cudaError_t e = cudaFuncSetAttribute(scan_chunk_kernel<N, OUT, PHASE>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    return launch_dependent(scan_chunk_kernel<N, OUT, PHASE>, (unsigned)ctas, warps * 32, smem, s, a, row_blocks);
}

template <int N> cudaError_t launch_n(const ScanArgs &a, cudaStream_t s) {
    int64_t row_blocks;
    const int warps = scan_chunk_warps(a.P, &row_blocks);
    const int64_t ctas = a.B * a.H * row_blocks;
    if (ctas * a.segments > INT32_MAX) return cudaErrorInvalidConfiguration;
    if (a.segments == 1)
        return a.y ? launch_phase<N, true, kScanWhole>(a, ctas, warps, row_blocks, s)
                   : launch_phase<N, false, kScanWhole>(a, ctas, warps, row_blocks, s);
    cudaError_t e = launch_phase<N, false, kScanFold>(a, ctas * a.segments, warps, row_blocks, s);
    if (e == cudaSuccess) e = launch_scan_join(a, s);
    if (e != cudaSuccess || !a.y) return e;
    return launch_phase<N, true, kScanOutput>(a, ctas * a.segments, warps, row_blocks, s);
}

}  // namespace

int scan_chunk_warps(int64_t P, int64_t *row_blocks) {
    const int64_t w = (P + 15) / 16;
    *row_blocks = (w + 7) / 8;
    return (int)((w + *row_blocks - 1) / *row_blocks);
}

cudaError_t launch_scan_chunk(const ScanArgs &a, cudaStream_t s) {
    switch (a.N) {
    case 64: return launch_n<64>(a, s);
    case 128: return launch_n<128>(a, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace gdn
