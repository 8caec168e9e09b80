// kv_attend.cu -- attention over the 4-bit paged cache.
//
// A unit is up to 16 query rows (draft tokens times query heads of one key
// head) of one sequence and key head.  Each warp takes 16 tokens at a time
// through S = Q K^T, the running maximum and sum of the softmax, and O += P V on
// mma.sync (m16n8k16, f16 operands, f32 sums), and keeps its own maximum, sum
// and O until the end of its part of the unit.
//
// Operands.  Codes times scales are exact in f16 (fp4.cuh).  A query row is
// scaled by a power of two and split into f16 terms: one for f16 and bf16
// inputs (exact to 2^-24 of the row's largest), two for f32 (2^-23 of an
// element).  Probabilities are rounded to one f16 term (2^-12, against 2^-9 of a
// bf16 output and 2^-12 of an f16 one), two for f32.
//
// Layout.  The order of the contracted index is free as long as both operands
// use it: a lane's four elements of a k-step are neighbours in its row of the
// cache, so it reads its row in 16-byte pieces; column c of an n-tile of S is
// token 4 (c % 2) + c / 2 of the eight, and column c of O's n-tile j is channel
// c D/8 + j, so a lane reads a run of D/8 channels of each of its tokens and
// interleaves the codes of two tokens with four logic instructions per 16.
//
// The tokens of all units, in chunks of 64, form one line that is cut in
// equal parts, one per block; the parts of a unit that is cut are joined by a
// second kernel in the order of the line, so results do not change from run
// to run.  With many units (long prompts) a block takes a whole unit.
#include <algorithm>

#include "attend.h"
#include "fp4.cuh"
#include "pieces.cuh"

namespace gdn {

namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kRows = kAttendRows;
constexpr int kTile = 16;                    // tokens of a warp at a time
constexpr int kChunk = kTile * kWarps;       // tokens of a block at a time
constexpr int kGrid = 3 * 152;               // blocks of a call that is cut along its tokens
constexpr int kMaxPairs = 1024;              // (sequence, row block) pairs of such a call
constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.693147180559945309f;
// Probabilities carry a factor 2^boost, so that small ones keep their bits in
// f16 (whose steps end at 2^-24), and the maximum moves once it is 2^slack
// behind; boost + slack stay below f16's 2^16.
template <typename T> constexpr float kBoost = sizeof(T) == 4 ? 14.f : 6.f;
template <typename T> constexpr float kSlack = sizeof(T) == 4 ? 1.f : 8.f;

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;\n" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// What a pair (sequence b, row block rb) sees: tokens [lo, hi), of which every
// row sees [lo_all, hi_all).
struct Span {
    int b, rb, n, len;       // n: the sequence's query tokens
    int rows;                // of this block, 0: nothing to do
    int lo, hi, lo_all, hi_all;
    int chunk0, chunks;
};
__device__ __forceinline__ Span span_of(const AttendArgs &a, int p, int row_blocks) {
    Span s;
    s.b = p / row_blocks;
    s.rb = p - s.b * row_blocks;
    const int G = a.Hq / a.H, T = (int)a.T;
    s.n = a.fresh ? min(max(a.fresh[s.b], 0), T) : T;
    s.len = (int)min((int64_t)max(a.lengths[s.b], 0), (int64_t)a.width << a.page_shift);
    const int r0 = s.rb * kRows;
    s.rows = min(max(s.n * G - r0, 0), kRows);
    s.lo = s.hi = s.lo_all = s.hi_all = s.chunk0 = s.chunks = 0;
    if (s.rows == 0) return s;
    const int pos0 = s.len - s.n + r0 / G, pos1 = s.len - s.n + (r0 + s.rows - 1) / G;
    s.hi = max(pos1 + 1, 0);
    s.hi_all = max(pos0 + 1, 0);
    if (a.window > 0) {
        s.lo = max(pos0 - a.window + 1, 0);
        s.lo_all = max(pos1 - a.window + 1, 0);
    }
    s.chunk0 = s.lo / kChunk;
    s.chunks = max((s.hi + kChunk - 1) / kChunk - s.chunk0, 1);  // (a row that sees nothing is written too)
    return s;
}

template <typename T, int D> struct Smem {
    static constexpr int kTerms = sizeof(T) == 4 ? 2 : 1;
    static constexpr int kQStride = D + 8;                                 // f16 per query row
    static constexpr size_t kQ = (size_t)kTerms * kRows * kQStride * 2;
    // each warp's ring of tiles (K codes, K scales, V codes, V scales of 16
    // tokens), under the warps' O at the end of a unit
    static constexpr int kTileBytes = kTile * D * 9 / 8;
    static constexpr int kStages = D == 64 ? 8 : D == 128 ? 6 : 5;
    static constexpr int kOStride = D + 4;                                 // f32 per row of O
    static constexpr size_t kRing = (size_t)kWarps * kStages * kTileBytes;
    static constexpr size_t kO = (size_t)kWarps * kRows * kOStride * 4;
    static constexpr size_t kBig = kRing > kO ? kRing : kO;
    static constexpr size_t kBytes = kQ + kBig + (size_t)kWarps * kRows * 8 + kRows * 8;
    static_assert(kQ % 16 == 0 && kTileBytes % 16 == 0, "16-byte pieces");
};

__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N> __device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
}

// First index of block c's part of a line of W chunks; the block of index x.
__device__ __forceinline__ int64_t part_begin(int64_t c, int64_t W, int64_t N) { return c * W / N; }
__device__ __forceinline__ int64_t part_of(int64_t x, int64_t W, int64_t N) { return ((x + 1) * N - 1) / W; }

__device__ __forceinline__ int64_t parts_of(int64_t W, int64_t blocks) { return W < blocks ? W : blocks; }

// The workspace: where each pair begins in the line, then two partial results
// per block (O, the maximum and the sum of each row).
constexpr int partial_floats(int D) { return kRows * (D + 2); }
constexpr int kBaseFloats = 2 * (kMaxPairs + 8);
__device__ __forceinline__ float *partial(float *workspace, int D, int i) {
    return workspace + kBaseFloats + (int64_t)i * partial_floats(D);
}

template <typename T>
__device__ __forceinline__ void write_row(const AttendArgs &a, const Span &s, int h, int row, int d0, const float *o,
                                          int n, float inv, float m, float l) {
    const int G = a.Hq / a.H, r = s.rb * kRows + row, t = r / G, hq = h * G + r - t * G;
    const int64_t tok = (int64_t)s.b * a.T + t;
    T *y = static_cast<T *>(a.y) + (tok * a.Hq + hq) * a.D + d0;
    for (int i = 0; i < n; ++i) st_from_f32(y + i, o[i] * inv);
    if (d0 == 0 && a.lse) a.lse[tok * a.Hq + hq] = l == 0.f ? -INFINITY : (m - kBoost<T> + log2f(l)) * kLn2;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, D == 256 ? 2 : 3)
attend_kernel(const AttendArgs a, int pairs, int row_blocks, bool whole) {
    using S = Smem<T, D>;
    constexpr int TERMS = S::kTerms, STEPS = D / 16, NT = D / 8, NS = S::kStages;
    constexpr int KD = D < 128 ? D / 4 : 32, SP = KD / 4;   // a lane's neighbouring channels of K, k-steps that they fill
    constexpr int NP = D / (4 * KD);                        // such pieces per row
    constexpr int VD = D / 8;                               // a lane's channels of V
    constexpr bool kQRegs = TERMS * STEPS * 4 <= 64;        // query fragments stay in registers
    extern __shared__ __align__(16) unsigned char smem[];
    __half *sq = reinterpret_cast<__half *>(smem);
    unsigned char *ring = smem + S::kQ;
    float *so = reinterpret_cast<float *>(smem + S::kQ);
    float *sm = reinterpret_cast<float *>(smem + S::kQ + S::kBig), *sl = sm + kWarps * kRows;
    float2 *sc = reinterpret_cast<float2 *>(sl + kWarps * kRows);
    __shared__ int64_t base[kMaxPairs + 1];
    __shared__ int64_t part[kWarps];
    pdl_trigger();
    pdl_wait();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
    const int page = 1 << a.page_shift, G = a.Hq / a.H;
    const int64_t block_bytes = kv_block_bytes(page, D);
    ring += warp * NS * S::kTileBytes;
    const uint32_t ring_s = static_cast<uint32_t>(__cvta_generic_to_shared(ring));

    int64_t at, end, W = 0;
    if (!whole) {
        int64_t carry = 0;
        for (int p0 = 0; p0 < pairs; p0 += kThreads) {
            const int p = p0 + tid;
            const int64_t mine = p < pairs ? (int64_t)span_of(a, p, row_blocks).chunks * a.H : 0;
            int64_t v = mine;
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
                const int64_t o = __shfl_up_sync(0xffffffffu, v, d);
                if (lane >= d) v += o;
            }
            if (lane == 31) part[warp] = v;
            __syncthreads();
            for (int w = 0; w < kWarps; ++w) {
                if (w < warp) v += part[w];
            }
            if (p < pairs) base[p] = carry + v - mine;
            for (int w = 0; w < kWarps; ++w) carry += part[w];
            __syncthreads();
        }
        if (tid == 0) base[pairs] = carry;
        W = carry;
        const int64_t N = parts_of(W, gridDim.x);
        at = blockIdx.x < N ? part_begin(blockIdx.x, W, N) : W;
        end = blockIdx.x < N ? part_begin(blockIdx.x + 1, W, N) : W;
        __syncthreads();
        // where the pairs begin, for the kernel that joins
        if (blockIdx.x == 0)
            for (int p = tid; p <= pairs; p += kThreads) reinterpret_cast<int64_t *>(a.workspace)[p] = base[p];
    } else {
        at = 0;
        end = 1;
    }

    bool first = true;
    while (at < end) {
        // the unit at `at` and this block's chunks of it
        int p, h, c0, c1;
        Span s;
        if (whole) {
            // later row blocks see more tokens: those first
            const int u = (int)(gridDim.x - 1 - blockIdx.x);
            h = u % a.H;
            const int q = u / a.H, nb = pairs / row_blocks;
            p = (q % nb) * row_blocks + q / nb;
            s = span_of(a, p, row_blocks);
            c0 = 0;
            c1 = s.chunks;
            at = end;
            if (s.rows == 0) return;
        } else {
            int lo = 0, hi = pairs;
            while (hi - lo > 1) {
                const int mid = (lo + hi) / 2;
                if (base[mid] <= at) lo = mid;
                else hi = mid;
            }
            p = lo;
            s = span_of(a, p, row_blocks);
            const int64_t off = at - base[p];
            h = (int)(off / s.chunks);
            c0 = (int)(off - (int64_t)h * s.chunks);
            c1 = (int)min((int64_t)s.chunks, c0 + (end - at));
            at += c1 - c0;
        }

        // ------------------------------------------------ this warp's tiles
        const int n = c1 - c0, first_tok = (s.chunk0 + c0) * kChunk + warp * kTile;
        const int32_t *row_table = a.table + (int64_t)s.b * a.width;
        // the page of tile k + lane, -1: nothing of it is seen
        auto pages_from = [&](int k) {
            const int tok = first_tok + (k + lane) * kChunk;
            int id = -1;
            if (k + lane < n && tok < s.hi && tok + kTile > s.lo) id = row_table[tok >> a.page_shift];
            return id < a.pages ? id : -1;
        };
        int ids = pages_from(0), ids_next = pages_from(32);
        auto fetch = [&](int k, int id) {  // tile k into its slot of the ring
            if (id >= 0) {
                const unsigned char *blk = a.cache + ((int64_t)id * a.H + h) * block_bytes;
                const int row0 = (first_tok + k * kChunk) & (page - 1);
                const unsigned char *kc = blk + row0 * (D / 2), *ks = blk + page * (D / 2) + row0 * (D / 16);
                const int values = page * (D / 2 + D / 16);
                const uint32_t dst = ring_s + (uint32_t)(k % NS) * S::kTileBytes;
                constexpr int CODES = kTile * D / 2, HALF = CODES + kTile * D / 16;
#pragma unroll
                for (int i = 0; i < CODES / 512; ++i) {
                    copy16(dst + 512 * i + 16 * lane, kc + 512 * i + 16 * lane);
                    copy16(dst + HALF + 512 * i + 16 * lane, kc + values + 512 * i + 16 * lane);
                }
                constexpr int SP16 = kTile * D / 16 / 16;  // pieces of scales
                if (lane < 2 * SP16) {
                    const bool v = lane >= SP16;
                    const int o = 16 * (v ? lane - SP16 : lane);
                    copy16(dst + (v ? HALF : 0) + CODES + o, ks + (v ? values : 0) + o);
                }
            }
            copy_commit();
        };
#pragma unroll
        for (int k = 0; k < NS - 1; ++k) fetch(k, __shfl_sync(0xffffffffu, ids, k));

        // ------------------------------------------------ queries to f16 terms
        for (int row = warp; row < kRows; row += kWarps) {
            const int r = s.rb * kRows + row, t = r / G;
            const T *q = static_cast<const T *>(a.q) + s.b * a.q_sb + t * a.q_st + (int64_t)(h * G + r - t * G) * D;
            float v[D / 32], top = 0.f;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                v[i] = row < s.rows ? ld_f32(q + lane + 32 * i) : 0.f;
                top = fmaxf(top, fabsf(v[i]));
            }
#pragma unroll
            for (int d = 16; d; d /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            // the power of two that brings the largest into [2^10, 2^11), with the
            // scale's sign
            const int e = top < INFINITY ? max((int)(__float_as_uint(top) >> 23) - 127, -100) : 10;
            const float up = copysignf(__uint_as_float((uint32_t)(127 + 10 - e) << 23), a.scale);
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                const float x = v[i] * up;
                const __half hi = __float2half_rn(x);
                sq[row * S::kQStride + lane + 32 * i] = hi;
                if (TERMS == 2)
                    sq[(kRows + row) * S::kQStride + lane + 32 * i] = __float2half_rn(x - __half2float(hi));
            }
            if (lane == 0) {
                // scores count in powers of two; the factor as a float and, for
                // float32 calls, its rest
                const float ks = a.k_scale ? a.k_scale[h] : 1.f, down = __uint_as_float((uint32_t)(127 + e - 10) << 23);
                if (TERMS == 2) {
                    const double f = fabs((double)a.scale) * 1.44269504088896340736 * ks * down;
                    sc[row] = make_float2((float)f, (float)(f - (float)f));
                } else {
                    sc[row] = make_float2(fabsf(a.scale) * kLog2e * ks * down, 0.f);
                }
            }
        }
        __syncthreads();
        auto query = [&](int m, int st, uint32_t (&f)[4]) {
            const int d = (st / SP) * 128 + t4 * KD + 4 * (st % SP);
            const uint2 x = *reinterpret_cast<const uint2 *>(sq + (m * kRows + g) * S::kQStride + d);
            const uint2 y = *reinterpret_cast<const uint2 *>(sq + (m * kRows + g + 8) * S::kQStride + d);
            f[0] = x.x;
            f[1] = y.x;
            f[2] = x.y;
            f[3] = y.y;
        };
        uint32_t qf[kQRegs ? TERMS : 1][kQRegs ? STEPS : 1][4];
        if constexpr (kQRegs) {
#pragma unroll
            for (int m = 0; m < TERMS; ++m)
#pragma unroll
                for (int st = 0; st < STEPS; ++st) query(m, st, qf[m][st]);
        }
        const float2 cr[2] = {sc[g], sc[g + 8]};
        // the last token that each of the lane's two rows sees
        int pos[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) pos[i] = s.len - s.n + (s.rb * kRows + g + 8 * i) / G;

        float o[NT][4], mx[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f};
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[j][e] = 0.f;

        for (int k = 0; k < n; ++k) {
            const int id = __shfl_sync(0xffffffffu, ids, k & 31);
            const int kn = k + NS - 1;
            const int id_n = __shfl_sync(0xffffffffu, (kn >> 5) == (k >> 5) ? ids : ids_next, kn & 31);
            copy_wait<NS - 2>();
            __syncwarp();
            fetch(kn, kn < n ? id_n : -1);
            if ((k & 31) == 31) {
                ids = ids_next;
                ids_next = pages_from(k + 33);
            }
            if (id < 0) continue;
            const int tok0 = first_tok + k * kChunk;
            const unsigned char *kc = ring + (k % NS) * S::kTileBytes, *ks = kc + kTile * D / 2;
            const unsigned char *vc = ks + kTile * D / 16, *vs = vc + kTile * D / 2;
            // ------------------------------------------------ S = Q K^T
            float x[2][4] = {};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int row = 8 * i + (g >> 1) + 4 * (g & 1);
#pragma unroll
                for (int pc = 0; pc < NP; ++pc) {
                    uint32_t w[KD / 8], sc2;
                    const unsigned char *src = kc + row * (D / 2) + pc * 64 + t4 * (KD / 2);
                    const unsigned char *scp = ks + row * (D / 16) + pc * 8 + t4 * (KD / 16);
                    if constexpr (KD == 32) {
                        const uint4 r = *reinterpret_cast<const uint4 *>(src);
                        w[0] = r.x;
                        w[1] = r.y;
                        w[2] = r.z;
                        w[3] = r.w;
                        sc2 = *reinterpret_cast<const uint16_t *>(scp);
                    } else {
                        const uint2 r = *reinterpret_cast<const uint2 *>(src);
                        w[0] = r.x;
                        w[1] = r.y;
                        sc2 = *scp;
                    }
                    const uint32_t both = e4m3x2_to_f16(sc2);
#pragma unroll
                    for (int kk = 0; kk < KD / 8; ++kk) {
                        uint32_t hw[4];
                        e2m1x8_to_f16(w[kk], hw);
                        const uint32_t f = __byte_perm(both, both, kk / 2 ? 0x3232 : 0x1010);
#pragma unroll
                        for (int q = 0; q < 4; q += 2) {
                            const int st = pc * SP + 2 * kk + q / 2;
                            const uint32_t b0 = hmul2(hw[q], f), b1 = hmul2(hw[q + 1], f);
                            if constexpr (TERMS == 1) {
                                if constexpr (kQRegs) {
                                    mma_f16(x[i], qf[0][st], b0, b1);
                                } else {
                                    uint32_t fr[4];
                                    query(0, st, fr);
                                    mma_f16(x[i], fr, b0, b1);
                                }
                            } else {
                                // the tensor cores cut their sums off, so long ones are added here
                                float y[4] = {};
                                uint32_t fr[4];
                                if constexpr (kQRegs) {
                                    mma_f16(y, qf[1][st], b0, b1);
                                    mma_f16(y, qf[0][st], b0, b1);
                                } else {
                                    query(1, st, fr);
                                    mma_f16(y, fr, b0, b1);
                                    query(0, st, fr);
                                    mma_f16(y, fr, b0, b1);
                                }
#pragma unroll
                                for (int e = 0; e < 4; ++e) x[i][e] += y[e];
                            }
                        }
                    }
                }
            }
            // ------------------------------------------------ softmax
            const bool edge = tok0 < s.lo_all || tok0 + kTile > s.hi_all;
            float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (edge) {
                        const int tok = tok0 + 8 * i + t4 + 4 * (e & 1), q = pos[e >> 1];
                        if (tok > q || (a.window > 0 && tok <= q - a.window)) x[i][e] = -INFINITY;
                    }
                    top[e >> 1] = fmaxf(top[e >> 1], x[i][e]);
                }
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 1));
                top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 2));
                // (a row that sees nothing here, whatever its factor)
                top[r] = top[r] == -INFINITY ? -INFINITY : top[r] * cr[r].x;
            }
            if (__any_sync(0xffffffffu, top[0] > mx[0] + kSlack<T> || top[1] > mx[1] + kSlack<T>)) {
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float to = fmaxf(mx[r], top[r]);
                    const float f = to == -INFINITY ? 1.f : exp2f(mx[r] - to);
                    mx[r] = to;
                    sum[r] *= f;
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        o[j][2 * r] *= f;
                        o[j][2 * r + 1] *= f;
                    }
                }
            }
            uint32_t pa[TERMS][4];
            const float off[2] = {mx[0] == -INFINITY ? 0.f : mx[0] - kBoost<T>, mx[1] == -INFINITY ? 0.f : mx[1] - kBoost<T>};
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    float pr[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float v = x[i][2 * r + e];
                        const float u = TERMS == 2 ? fmaf(v, cr[r].x, fmaf(v, cr[r].y, -off[r])) : fmaf(v, cr[r].x, -off[r]);
                        pr[e] = ex2f(edge && v == -INFINITY ? -INFINITY : u);
                    }
                    sum[r] += pr[0] + pr[1];
                    const __half2 hi = __floats2half2_rn(pr[0], pr[1]);
                    pa[0][2 * i + r] = *reinterpret_cast<const uint32_t *>(&hi);
                    if (TERMS == 2) {
                        const float2 f = __half22float2(hi);
                        pa[TERMS - 1][2 * i + r] = pack2<__half>(pr[0] - f.x, pr[1] - f.y);
                    }
                }
            // ------------------------------------------------ O += P V
            uint32_t vw[4][VD / 8], vf[2][(VD + 15) / 16];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                uint32_t sb[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int row = 8 * i + t4 + 4 * e;
                    const unsigned char *src = vc + row * (D / 2) + g * (VD / 2);
                    if constexpr (VD == 8) {
                        vw[2 * i + e][0] = *reinterpret_cast<const uint32_t *>(src);
                    } else if constexpr (VD == 16) {
                        const uint2 r = *reinterpret_cast<const uint2 *>(src);
                        vw[2 * i + e][0] = r.x;
                        vw[2 * i + e][1] = r.y;
                    } else {
                        const uint4 r = *reinterpret_cast<const uint4 *>(src);
                        vw[2 * i + e][0] = r.x;
                        vw[2 * i + e][1] = r.y;
                        vw[2 * i + e][2] = r.z;
                        vw[2 * i + e][3] = r.w;
                    }
                    const unsigned char *scp = vs + row * (D / 16) + g * VD / 16;
                    if constexpr (VD == 32) sb[e] = *reinterpret_cast<const uint16_t *>(scp);
                    else sb[e] = *scp;
                    // (a token that no row sees may hold anything)
                    if (edge && (tok0 + row < s.lo || tok0 + row >= s.hi)) sb[e] = 0;
                }
#pragma unroll
                for (int w = 0; w < (VD + 15) / 16; ++w) vf[i][w] = e4m3x2_to_f16(__byte_perm(sb[0], sb[1], w ? 0x4451 : 0x4440));
            }
#pragma unroll
            for (int v8 = 0; v8 < VD / 8; ++v8) {  // eight channels at a time
                uint32_t h0[2][4], h1[2][4];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t wa = vw[2 * i][v8], wb = vw[2 * i + 1][v8], f = vf[i][v8 / 2];
                    e2m1x8_to_f16((wa & 0x0f0f0f0fu) | ((wb << 4) & 0xf0f0f0f0u), h0[i]);
                    e2m1x8_to_f16(((wa >> 4) & 0x0f0f0f0fu) | (wb & 0xf0f0f0f0u), h1[i]);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        h0[i][q] = hmul2(h0[i][q], f);
                        h1[i][q] = hmul2(h1[i][q], f);
                    }
                }
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint32_t b0 = e ? h1[0][q] : h0[0][q], b1 = e ? h1[1][q] : h0[1][q];
                        float (&acc)[4] = o[8 * v8 + 2 * q + e];
                        if constexpr (TERMS == 1) {
                            mma_f16(acc, pa[0], b0, b1);
                        } else {
                            float y[4] = {};
                            mma_f16(y, pa[TERMS - 1], b0, b1);
                            mma_f16(y, pa[0], b0, b1);
#pragma unroll
                            for (int c = 0; c < 4; ++c) acc[c] += y[c];
                        }
                    }
            }
        }
        copy_wait<0>();
        __syncthreads();  // the rings are free for the warps' O

        // ------------------------------------------------ the warps' parts joined
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 1);
            sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 2);
            const int row = warp * kRows + g + 8 * r;
            if (t4 == 0) {
                sm[row] = mx[r];
                sl[row] = sum[r];
            }
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int j = 0; j < NT; j += 4)
                    *reinterpret_cast<float4 *>(so + row * S::kOStride + (2 * t4 + e) * VD + j) =
                        make_float4(o[j][2 * r + e], o[j + 1][2 * r + e], o[j + 2][2 * r + e], o[j + 3][2 * r + e]);
        }
        __syncthreads();
        {
            constexpr int PER = D / 8;  // eight threads per row
            const int row = tid / 8, d0 = (tid % 8) * PER;
            float m = -INFINITY, l = 0.f, acc[PER];
#pragma unroll
            for (int w = 0; w < kWarps; ++w) m = fmaxf(m, sm[w * kRows + row]);
#pragma unroll
            for (int i = 0; i < PER; ++i) acc[i] = 0.f;
            if (m == -INFINITY) m = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = exp2f(sm[w * kRows + row] - m);
                l += f * sl[w * kRows + row];
#pragma unroll
                for (int i = 0; i < PER; ++i) acc[i] += f * so[(w * kRows + row) * S::kOStride + d0 + i];
            }
            if (row < s.rows) {
                if (c0 == 0 && c1 == s.chunks) {
                    const float vs = a.v_scale ? a.v_scale[h] : 1.f;
                    write_row<T>(a, s, h, row, d0, acc, PER, l == 0.f ? 0.f : vs / l, m, l);
                } else {
                    float *ws = partial(a.workspace, D, 2 * blockIdx.x + (first ? 0 : 1));
#pragma unroll
                    for (int i = 0; i < PER; i += 4)
                        *reinterpret_cast<float4 *>(ws + row * D + d0 + i) =
                            make_float4(acc[i], acc[i + 1], acc[i + 2], acc[i + 3]);
                    if (d0 == 0) {
                        ws[kRows * D + row] = m;
                        ws[kRows * (D + 1) + row] = l;
                    }
                }
            }
        }
        __syncthreads();
        first = false;
    }
}

// Joins the parts of a unit that several blocks worked on: a block per query
// row, each of its warps every eighth part.
constexpr int kJoinWarps = 8;
template <typename T, int D>
__global__ void __launch_bounds__(32 * kJoinWarps)
attend_join_kernel(const AttendArgs a, int pairs, int row_blocks, int rows, int blocks) {
    constexpr int PER = D / 32;
    __shared__ float sm[kJoinWarps], sl[kJoinWarps], so[kJoinWarps][D];
    pdl_trigger();
    pdl_wait();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int u = blockIdx.x / rows, row = blockIdx.x - u * rows;
    const int p = u / a.H, h = u - p * a.H;
    const int64_t *base = reinterpret_cast<const int64_t *>(a.workspace);
    const int64_t begin = base[p], chunks = (base[p + 1] - begin) / a.H, W = base[pairs];
    if (chunks == 0) return;
    const int64_t N = parts_of(W, blocks);
    const int64_t x0 = begin + h * chunks, x1 = x0 + chunks;
    const int b0 = (int)part_of(x0, W, N), b1 = (int)part_of(x1 - 1, W, N);
    if (b0 == b1) return;  // written whole
    const Span s = span_of(a, p, row_blocks);
    if (row >= s.rows) return;
    const int later = part_begin(b0, W, N) < x0;  // the unit is not the first of block b0
    float m = -INFINITY, l = 0.f, acc[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) acc[i] = 0.f;
    for (int q = b0 + warp; q <= b1; q += kJoinWarps) {
        const float *ws = partial(a.workspace, D, 2 * q + (q == b0 ? later : 0));
        const float pm = ws[kRows * D + row], pl = ws[kRows * (D + 1) + row];
        float v[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) v[i] = ws[row * D + lane + 32 * i];
        if (pl == 0.f) continue;  // (it saw nothing)
        const float to = fmaxf(m, pm), f = exp2f(m - to), g = exp2f(pm - to);
        m = to;
        l = l * f + pl * g;
#pragma unroll
        for (int i = 0; i < PER; ++i) acc[i] = acc[i] * f + v[i] * g;
    }
    if (lane == 0) {
        sm[warp] = m;
        sl[warp] = l;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) so[warp][lane + 32 * i] = acc[i];
    __syncthreads();
    m = -INFINITY;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) m = fmaxf(m, sm[w]);
    if (m == -INFINITY) m = 0.f;
    float f[kJoinWarps];
    l = 0.f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
        f[w] = exp2f(sm[w] - m);
        l += f[w] * sl[w];
    }
    const float vs = a.v_scale ? a.v_scale[h] : 1.f;
    if (tid < D) {
        float o = 0.f;
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w) o += f[w] * so[w][tid];
        write_row<T>(a, s, h, row, tid, &o, 1, l == 0.f ? 0.f : vs / l, m, l);
    }
}

int64_t row_blocks_of(int64_t T, int64_t G) { return (T * G + kRows - 1) / kRows; }

// A call is cut along its tokens while its units would not fill the GPU by
// themselves several times over.
bool cut(int64_t pairs, int64_t H) { return pairs <= kMaxPairs && pairs * H < 8 * kGrid; }

template <typename T, int D>
cudaError_t launch_td(const AttendArgs &a, cudaStream_t s) {
    const int64_t rb = row_blocks_of(a.T, a.Hq / a.H), pairs = a.B * rb, units = pairs * a.H;
    constexpr size_t smem = Smem<T, D>::kBytes;
    cudaError_t e = cudaFuncSetAttribute(attend_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    if (!cut(pairs, a.H)) {
        if (units > INT32_MAX) return cudaErrorInvalidConfiguration;
        return launch_dependent(attend_kernel<T, D>, (unsigned)units, kThreads, smem, s, a, (int)pairs, (int)rb, true);
    }
    // as many blocks as are resident at a time
    const int blocks = D == 256 ? kGrid / 3 * 2 : kGrid;
    e = launch_dependent(attend_kernel<T, D>, (unsigned)blocks, kThreads, smem, s, a, (int)pairs, (int)rb, false);
    if (e != cudaSuccess) return e;
    const int rows = (int)std::min<int64_t>(a.T * (a.Hq / a.H), kRows);
    return launch_dependent(attend_join_kernel<T, D>, (unsigned)(units * rows), 32 * kJoinWarps, 0, s, a, (int)pairs,
                            (int)rb, rows, blocks);
}

template <typename T>
cudaError_t launch_t(const AttendArgs &a, cudaStream_t s) {
    switch (a.D) {
    case 64: return launch_td<T, 64>(a, s);
    case 128: return launch_td<T, 128>(a, s);
    case 256: return launch_td<T, 256>(a, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

int64_t attend_workspace_bytes(int64_t B, int64_t T, int64_t Hq, int64_t H, int64_t D) {
    int64_t rows, pairs;
    if (__builtin_mul_overflow(T, Hq / H, &rows) || rows > INT32_MAX - kRows ||
        __builtin_mul_overflow(B, row_blocks_of(T, Hq / H), &pairs) || pairs > INT32_MAX)
        return -1;
    return cut(pairs, H) ? ((int64_t)2 * kGrid * partial_floats((int)D) + kBaseFloats) * 4 : 0;
}

cudaError_t launch_kv_attend(DType dt, const AttendArgs &a, cudaStream_t s) {
    switch (dt) {
    case DType::F32: return launch_t<float>(a, s);
    case DType::BF16: return launch_t<__nv_bfloat16>(a, s);
    case DType::F16: return launch_t<__half>(a, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace gdn
