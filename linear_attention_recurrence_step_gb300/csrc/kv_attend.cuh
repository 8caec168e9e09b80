// kv_attend.cuh -- attention over the 4-bit paged cache.
//
// A unit is up to 8 or 16 query rows (draft tokens times query heads of one
// key head) of one sequence and key head.  Each warp takes 32 tokens at a time
// through S^T = K Q^T, the softmax, and O^T += V^T P^T on mma.sync (m16n8k16, f16
// operands, f32 sums), and keeps its own reference, sum and O until the end of
// its part of the unit.  Tokens and channels are the products' wide side (16),
// query rows the narrow one (8), so that a single token's few rows waste
// little; a transposition of 8 x 8 f16 pairs turns S^T's accumulator into P^T.
//
// Operands.  Codes times scales are exact in f16 (fp4.cuh).  A query row is
// scaled by a power of two and split into f16 terms: one for f16 and bf16
// inputs (exact to 2^-24 of the row's largest), two for f32 (2^-23 of an
// element).  Probabilities are rounded to one f16 term (2^-12, against 2^-9 of a
// bf16 output and 2^-12 of an f16 one), two for f32.
//
// Softmax.  2^(x - reference) needs no maximum as long as the reference is near:
// it moves (and sum and O with it) only when some x is 2^slack above it, which
// one vote per tile finds, so most tiles take no reduction over tokens at all.
// x - reference is one operation on a score and its factor.  Where x can reach 2^26, and
// a float32 reference can be off by more than the slack, a warp rounds scores to x
// first, as the reference is.
//
// Layout.  The order of the contracted index is free as long as both operands
// use it: a lane's four elements of a k-step are neighbours in its row of the
// cache, so it reads its row in 16-byte pieces; row r of S^T's eight is token
// 4 (r % 2) + r / 2, and row r of O^T's m-tile j is channel (r % 8) D/8 + 2j + r/8,
// so a lane reads a run of D/8 channels of each of its tokens and interleaves
// the codes of two tokens with logic on whole words.
//
// The tokens of all units, in chunks of 128, form one line that is cut in
// equal parts, one per block; the parts of a unit that is cut are joined by a
// second kernel in the order of the line, so results do not change from run
// to run.  Units that fill the GPU by themselves are taken whole, one by a block.
//
// Bound by issue (62 % of the slots; half of the instructions dequantise), then by
// memory: one token of 8 sequences of 131072 (8 key heads of 128, 1.2 GB) 223 us, 5.4
// TB/s; of 32 sequences of up to 8192 (189 MB) 51 us, 52 with cold caches; float32 calls
// 321 and 69.  With query rows on the wide side of the products, as usual, the first took
// 371 us.
#pragma once

#include <algorithm>
#include <cfloat>

#include "attend.h"
#include "fp4.cuh"
#include "pieces.cuh"

namespace gdn {

namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kTile = 32;                    // tokens of a warp at a time, in halves of 16
constexpr int kChunk = kTile * kWarps;       // tokens of a block at a time
constexpr int kSms = 152;                    // a call that is cut along its tokens has as many blocks as these hold
constexpr int kMaxPairs = 512;               // (sequence, row block) pairs of such a call
constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.693147180559945309f;
// Probabilities carry a factor 2^boost, so that small ones keep their bits in
// f16 (whose steps end at 2^-24); boost + slack stay below f16's 2^16.
template <typename T> constexpr float kBoost = sizeof(T) == 4 ? 14.f : 6.f;
template <typename T> constexpr float kSlack = sizeof(T) == 4 ? 1.f : 8.f;
// The tensor cores cut a sum off where they add to it, so sums of terms of one sign fall
// short by half a unit of their last place per 16 tokens of a warp: by 1.6e-4 of them over
// 131072 tokens of a block.  Where a block can have more (of f16 calls; of bf16 calls 8
// times as many), that would pass half of y's rounding, and products are added outside
// (LONG).
template <typename T> constexpr int64_t kLongTokens = 131072;
template <> constexpr int64_t kLongTokens<__nv_bfloat16> = 1048576;
constexpr float kNoScore = -FLT_MAX;         // the reference of a row that has seen nothing
// Whether scores of a factor can reach 2^26 in powers of two: products of queries below
// 2^11 and keys of up to 2688, times D.
__device__ __forceinline__ bool far_scores(float factor, int D) { return factor * (float)D >= 0x1p26f / (2048.f * 2688.f); }

// Eights of query rows per unit (four would take 255 registers: 32 rows, heads of 128, of
// 16 sequences of up to 8192 tokens 75 us, two units of 16 rows 70), and the blocks of
// such units that an SM holds, by registers and shared memory.
constexpr int eights_of(int64_t rows) { return rows <= 8 ? 1 : 2; }
constexpr int resident(int NB, int D, bool f32) {
    return (NB == 1 ? (D == 64 ? 6 : D == 128 ? 5 : 3) : D == 64 ? 4 : D == 128 ? 3 : 2) - (f32 && !(NB > 1 && D > 64));
}

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

// The 8 x 8 pairs of a warp, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(d) : "r"(v));
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
__device__ __forceinline__ Span span_of(const AttendArgs &a, int p, int row_blocks, int unit_rows) {
    Span s;
    s.b = p / row_blocks;
    s.rb = p - s.b * row_blocks;
    const int G = a.Hq / a.H, T = (int)a.T;
    s.n = a.fresh ? min(max(a.fresh[s.b], 0), T) : T;
    s.len = (int)min((int64_t)max(a.lengths[s.b], 0), (int64_t)a.width << a.page_shift);
    const int r0 = s.rb * unit_rows;
    s.rows = min(max(s.n * G - r0, 0), unit_rows);
    s.lo = s.hi = s.lo_all = s.hi_all = s.chunk0 = s.chunks = 0;
    if (s.rows == 0) return s;
    const int pos0 = s.len - s.n + r0 / G, pos1 = s.len - s.n + (r0 + s.rows - 1) / G;
    s.hi = max(pos1 + 1, 0);
    s.hi_all = max(pos0 + 1, 0);
    if (a.window > 0) {
        // (positions before the first token are below 0: no difference that leaves 32 bits)
        s.lo = pos0 >= a.window ? pos0 - a.window + 1 : 0;
        s.lo_all = pos1 >= a.window ? pos1 - a.window + 1 : 0;
    }
    s.chunk0 = s.lo / kChunk;
    s.chunks = max((s.hi + kChunk - 1) / kChunk - s.chunk0, 1);  // (a row that sees nothing is written too)
    return s;
}

template <typename T, int D, int NB> struct Smem {
    static constexpr int kTerms = sizeof(T) == 4 ? 2 : 1;
    static constexpr int kRows = 8 * NB;
    static constexpr int kQStride = D + 8;                                 // f16 per query row
    static constexpr size_t kQ = (size_t)kTerms * kRows * kQStride * 2;
    // each warp's ring of tiles (K codes, K scales, V codes, V scales of 16
    // tokens, twice), under the warps' O at the end of a unit
    static constexpr int kHalfBytes = 16 * D * 9 / 8, kTileBytes = 2 * kHalfBytes;
    static constexpr int kStages = NB == 1 ? 2 : 3;
    static constexpr int kOStride = D + 4;                                 // f32 per row of O
    static constexpr size_t kRing = (size_t)kWarps * kStages * kTileBytes;
    static constexpr size_t kO = (size_t)kWarps * kRows * kOStride * 4;
    static constexpr size_t kBig = kRing > kO ? kRing : kO;
    static constexpr size_t kBytes = kQ + kBig + (size_t)kWarps * kRows * 8 + kRows * 8;
    static_assert(kQ % 16 == 0 && kHalfBytes % 16 == 0, "16-byte pieces");
};

__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N> __device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
}

// A line of W chunks is cut in as many parts as there are blocks (a constant: the
// quotient is a product), or in chunks if there are fewer: the first index of block
// c's part; the block of index x.
template <int BLOCKS> __device__ __forceinline__ int64_t part_begin(int c, int64_t W) {
    return W < BLOCKS ? min((int64_t)c, W) : (int64_t)((uint64_t)c * (uint64_t)W / BLOCKS);
}
template <int BLOCKS> __device__ __forceinline__ int part_of(int64_t x, int64_t W) {
    return W < BLOCKS ? (int)x : (int)(((x + 1) * BLOCKS - 1) / W);
}

// The workspace: where each pair begins in the line, then two partial results
// per block (O, the reference and the sum of each row).
constexpr int partial_floats(int rows, int D) { return rows * (D + 2); }
constexpr int kBaseFloats = 2 * (kMaxPairs + 8);
__device__ __forceinline__ float *partial(float *workspace, int rows, int D, int i) {
    return workspace + kBaseFloats + (int64_t)i * partial_floats(rows, D);
}

// N channels of row r of y from d0 on, o times inv, and its log-sum-exp.
template <typename T, int N>
__device__ __forceinline__ void write_row(const AttendArgs &a, const Span &s, int h, int r, int d0, const float (&o)[N],
                                          float inv, float ref, float l) {
    const int G = a.Hq / a.H, t = r / G, hq = h * G + r - t * G;
    const int64_t tok = (int64_t)s.b * a.T + t;
    T *y = static_cast<T *>(a.y) + (tok * a.Hq + hq) * a.D + d0;
    constexpr int VEC = 16 / (int)sizeof(T);
    if (N % VEC == 0 && a.vec_y) {
#pragma unroll
        for (int i = 0; i < N / VEC; ++i) {
            float v[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) v[e] = o[(i * VEC + e) % N] * inv;
            store_piece<T, VEC>(y + i * VEC, v);
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) st_from_f32(y + i, o[i] * inv);
    }
    if (d0 == 0 && a.lse) a.lse[tok * a.Hq + hq] = l == 0.f ? -INFINITY : (ref + log2f(l)) * kLn2;
}

template <typename T, int D, int NB, bool LONG>
__global__ void __launch_bounds__(kThreads, resident(NB, D, sizeof(T) == 4))
attend_kernel(const AttendArgs a, int pairs, int row_blocks, bool whole) {
    using S = Smem<T, D, NB>;
    constexpr int TERMS = S::kTerms, STEPS = D / 16, NS = S::kStages, ROWS = S::kRows;
    constexpr int KD = D < 128 ? D / 4 : 32, SP = KD / 4;   // a lane's neighbouring channels of K, k-steps that they fill
    constexpr int NP = D / (4 * KD);                        // such pieces per row
    constexpr int VD = D / 8, MT = VD / 2;                  // a lane's channels of V, m-tiles of O^T
    constexpr int VS = (VD + 15) / 16;                      // scales that they have
    constexpr bool kQRegs = TERMS * STEPS * 2 * NB <= 32;   // query fragments stay in registers
    extern __shared__ __align__(16) unsigned char smem[];
    __half *sq = reinterpret_cast<__half *>(smem);
    float *so = reinterpret_cast<float *>(smem + S::kQ);
    float *sm = reinterpret_cast<float *>(smem + S::kQ + S::kBig), *sl = sm + kWarps * ROWS;
    float2 *sc = reinterpret_cast<float2 *>(sl + kWarps * ROWS);
    __shared__ int64_t base[kMaxPairs + 1];
    __shared__ int64_t part[kWarps];
    // (the kernel that joins is let in when this one ends: its blocks, waiting beside
    // this one's, cost 7 of 60 us over 32 x 8192 tokens)
    pdl_wait();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
    const int page = 1 << a.page_shift, G = a.Hq / a.H;
    const int64_t block_bytes = kv_block_bytes(page, D);
    const unsigned char *ring = smem + S::kQ + warp * NS * S::kTileBytes;
    const uint32_t ring_s = static_cast<uint32_t>(__cvta_generic_to_shared(ring));

    int64_t at, end;
    if (!whole) {
        int64_t carry = 0;
        for (int p0 = 0; p0 < pairs; p0 += kThreads) {
            const int p = p0 + tid;
            const int64_t mine = p < pairs ? (int64_t)span_of(a, p, row_blocks, ROWS).chunks * a.H : 0;
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
        const int64_t W = carry;
        constexpr int BLOCKS = kSms * resident(NB, D, sizeof(T) == 4);
        at = part_begin<BLOCKS>((int)blockIdx.x, W);
        end = part_begin<BLOCKS>((int)blockIdx.x + 1, W);
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
            s = span_of(a, p, row_blocks, ROWS);
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
            s = span_of(a, p, row_blocks, ROWS);
            const int64_t off = at - base[p];
            h = (int)(off / s.chunks);
            c0 = (int)(off - (int64_t)h * s.chunks);
            c1 = (int)min((int64_t)s.chunks, c0 + (end - at));
            at += c1 - c0;
        }

        // ------------------------------------------------ this warp's tiles
        const int n = c1 - c0, first_tok = (s.chunk0 + c0) * kChunk + warp * kTile;
        const int32_t *row_table = a.table + (int64_t)s.b * a.width;
        // the table's entry for half `lane` of the tiles from k on, -1: nothing of it
        // is seen
        auto pages_from = [&](int k) {
            const int kk = k + (lane >> 1), tok = first_tok + kk * kChunk + 16 * (lane & 1);
            int id = -1;
            if (kk < n && tok < s.hi && tok + 16 > s.lo) id = row_table[tok >> a.page_shift];
            return id;  // (checked where it is used, later: here the warp would wait for it)
        };
        int ids = pages_from(0), ids_next = pages_from(16);
        // pages divide a chunk, so a warp's tiles start at the same row of their
        // pages.  Sources of the lane's 16-byte pieces in page 0, for either half:
        // keys' codes, values' codes, and the piece of scales that is its own
        constexpr int CODES = 8 * D, HALF = 9 * D;   // bytes of 16 tokens: codes; codes and scales
        constexpr int SPS = D / 16;                  // pieces of 16 tokens' scales, of keys or of values
        const uint32_t page_bytes = (uint32_t)(a.H * block_bytes), pool = (uint32_t)a.pages;
        const unsigned char *k_src[2], *v_src[2];
        const int values = page * (D / 2 + D / 16), row0 = first_tok & (page - 1);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            k_src[i] = a.cache + h * block_bytes + ((row0 + 16 * i) & (page - 1)) * (D / 2) + 16 * lane;
            v_src[i] = k_src[i] + values;
        }
        constexpr int SCOPIES = (4 * SPS + 31) / 32;
        const unsigned char *s_src[SCOPIES];
        uint32_t s_dst[SCOPIES];
#pragma unroll
        for (int j = 0; j < SCOPIES; ++j) {
            const int q = lane + 32 * j, i = q / (2 * SPS), v = q / SPS & 1, o = 16 * (q % SPS);
            s_src[j] = a.cache + h * block_bytes + page * (D / 2) + ((row0 + 16 * i) & (page - 1)) * (D / 16) + v * values + o;
            s_dst[j] = i * S::kHalfBytes + v * HALF + CODES + o;
        }
        // the halves of a tile into a slot of the ring; `from` holds their pages in
        // lanes at and at + 1.  Returns which of them are there.
        auto fetch = [&](uint32_t dst, int from, int at) {
            int id0 = __shfl_sync(0xffffffffu, from, at & 31), id1 = __shfl_sync(0xffffffffu, from, (at + 1) & 31);
            if ((uint32_t)id0 >= pool) id0 = -1;
            if ((uint32_t)id1 >= pool) id1 = -1;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int id = i ? id1 : id0;
                if (id >= 0) {
                    const unsigned char *kp = k_src[i] + (uint64_t)(uint32_t)id * page_bytes;
                    const unsigned char *vp = v_src[i] + (uint64_t)(uint32_t)id * page_bytes;
                    const uint32_t d = dst + i * S::kHalfBytes + 16 * lane;
#pragma unroll
                    for (int j = 0; j < CODES / 512; ++j) {
                        copy16(d + 512 * j, kp + 512 * j);
                        copy16(d + HALF + 512 * j, vp + 512 * j);
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < SCOPIES; ++j) {
                const int q = lane + 32 * j, id = q / (2 * SPS) ? id1 : id0;
                if ((4 * SPS % 32 == 0 || q < 4 * SPS) && id >= 0)
                    copy16(dst + s_dst[j], s_src[j] + (uint64_t)(uint32_t)id * page_bytes);
            }
            copy_commit();
            return (id0 >= 0 ? 1 : 0) | (id1 >= 0 ? 2 : 0);
        };
        uint32_t slot_in = ring_s;
        int slot = 0, there = 0;  // two bits per tile in flight
        auto next_in = [&]() {
            slot_in += S::kTileBytes;
            if (slot_in == ring_s + NS * S::kTileBytes) slot_in = ring_s;
        };
#pragma unroll
        for (int k = 0; k < NS - 1; ++k) {
            there |= fetch(slot_in, ids, 2 * k) << (2 * k);
            next_in();
        }

        // ------------------------------------------------ queries to f16 terms
        for (int row = warp; row < ROWS; row += kWarps) {
            const int r = s.rb * ROWS + row, t = r / G;
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
            // scale's sign; a NaN if it is infinite, for scores of -inf would count as
            // masked ones (NaNs are passed on as they are)
            const bool finite = top < INFINITY;
            const int e = finite ? max((int)(__float_as_uint(top) >> 23) - 127, -100) : 10;
            const float up = copysignf(__uint_as_float(finite ? (uint32_t)(127 + 10 - e) << 23 : 0x7fc00000u), a.scale);
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                const float x = v[i] * up;
                const __half hi = __float2half_rn(x);
                sq[row * S::kQStride + lane + 32 * i] = hi;
                if (TERMS == 2)
                    sq[(ROWS + row) * S::kQStride + lane + 32 * i] = __float2half_rn(x - __half2float(hi));
            }
            if (lane == 0) {
                // scores count in powers of two; the factor (never 0: what is masked
                // is -inf times it) as a float and, for float32 calls, its rest
                const float ks = a.k_scale ? a.k_scale[h] : 1.f, down = __uint_as_float((uint32_t)(127 + e - 10) << 23);
                if (TERMS == 2) {
                    const double f = fabs((double)a.scale) * 1.44269504088896340736 * ks * down;
                    sc[row] = make_float2(fmaxf((float)f, FLT_MIN), (float)(f - (float)f));
                } else {
                    sc[row] = make_float2(fmaxf(fabsf(a.scale) * kLog2e * ks * down, FLT_MIN), 0.f);
                }
            }
        }
        __syncthreads();
        // fragment of k-step st for the query rows 8b + g
        auto query = [&](int m, int b, int st) {
            const int d = (st / SP) * 128 + t4 * KD + 4 * (st % SP);
            return *reinterpret_cast<const uint2 *>(sq + (m * ROWS + 8 * b + g) * S::kQStride + d);
        };
        uint2 qf[kQRegs ? TERMS : 1][kQRegs ? NB : 1][kQRegs ? STEPS : 1];
        if constexpr (kQRegs) {
#pragma unroll
            for (int m = 0; m < TERMS; ++m)
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int st = 0; st < STEPS; ++st) qf[m][b][st] = query(m, b, st);
        }
        // of the lane's query rows 8b + 2 t4 + e: the score's factor, the last
        // token seen, the reference less the boost, the sum
        float2 cr[NB][2];
        bool rounded = false;  // the warp's scores are: their factor is 1 then, which is far itself
        int pos[NB][2];
        float off[NB][2], sum[NB][2];
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = 8 * b + 2 * t4 + e;
                cr[b][e] = sc[row];
                rounded = rounded || far_scores(cr[b][e].x, D);
                pos[b][e] = s.len - s.n + (s.rb * ROWS + row) / G;
                off[b][e] = kNoScore;
                sum[b][e] = 0.f;
            }
        rounded = __any_sync(0xffffffffu, rounded);
        if (rounded) {
#pragma unroll
            for (int b = 0; b < NB; ++b) cr[b][0] = cr[b][1] = make_float2(1.f, 0.f);
        }
        float o[NB][MT][4];
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int j = 0; j < MT; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[b][j][e] = 0.f;

        for (int k = 0; k < n; ++k) {
            const bool in0 = there & 1, in1 = there & 2;
            copy_wait<NS - 2>();
            __syncwarp();
            const int kn = k + NS - 1;
            there = (there >> 2) | fetch(slot_in, (kn >> 4) == (k >> 4) ? ids : ids_next, 2 * kn) << (2 * (NS - 2));
            next_in();
            if ((k & 15) == 15) {
                ids = ids_next;
                ids_next = pages_from(k + 17);
            }
            const unsigned char *tile = ring + slot * S::kTileBytes;
            slot = slot == NS - 1 ? 0 : slot + 1;
            if (!in0 && !in1) continue;
            const int tok0 = first_tok + k * kChunk;
            const bool edge = tok0 < s.lo_all || tok0 + kTile > s.hi_all || !in0 || !in1;
            // ------------------------------------------------ S^T = K Q^T
            float x[2][NB][4] = {};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const unsigned char *kc = tile + i * S::kHalfBytes, *ks = kc + CODES;
#pragma unroll
                for (int pc = 0; pc < NP; ++pc) {
                    uint32_t w[2][KD / 8], both[2];
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const int row = 8 * r + (g >> 1) + 4 * (g & 1);
                        const unsigned char *src = kc + row * (D / 2) + pc * 64 + t4 * (KD / 2);
                        const unsigned char *scp = ks + row * (D / 16) + pc * 8 + t4 * (KD / 16);
                        uint32_t sc2;
                        if constexpr (KD == 32) {
                            const uint4 q = *reinterpret_cast<const uint4 *>(src);
                            w[r][0] = q.x;
                            w[r][1] = q.y;
                            w[r][2] = q.z;
                            w[r][3] = q.w;
                            sc2 = *reinterpret_cast<const uint16_t *>(scp);
                        } else {
                            const uint2 q = *reinterpret_cast<const uint2 *>(src);
                            w[r][0] = q.x;
                            w[r][1] = q.y;
                            sc2 = *scp;
                        }
                        both[r] = e4m3x2_to_f16(sc2);
                    }
#pragma unroll
                    for (int kk = 0; kk < KD / 8; ++kk) {
                        uint32_t hw[2][4];
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            e2m1x8_to_f16(w[r][kk], hw[r]);
                            const uint32_t f = __byte_perm(both[r], both[r], kk / 2 ? 0x3232 : 0x1010);
#pragma unroll
                            for (int q = 0; q < 4; ++q) hw[r][q] = hmul2(hw[r][q], f);
                        }
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            const int st = pc * SP + 2 * kk + q;
                            const uint32_t af[4] = {hw[0][2 * q], hw[1][2 * q], hw[0][2 * q + 1], hw[1][2 * q + 1]};
#pragma unroll
                            for (int b = 0; b < NB; ++b) {
                                const uint2 q0 = kQRegs ? qf[0][kQRegs ? b : 0][kQRegs ? st : 0] : query(0, b, st);
                                if constexpr (TERMS == 1) {
                                    mma_f16(x[i][b], af, q0.x, q0.y);
                                } else {
                                    // (the tensor cores cut their sums off, so long ones are added here)
                                    const uint2 q1 = kQRegs ? qf[TERMS - 1][kQRegs ? b : 0][kQRegs ? st : 0] : query(TERMS - 1, b, st);
                                    float y[4] = {};
                                    mma_f16(y, af, q1.x, q1.y);
                                    mma_f16(y, af, q0.x, q0.y);
#pragma unroll
                                    for (int e = 0; e < 4; ++e) x[i][b][e] += y[e];
                                }
                            }
                        }
                    }
                }
            }
            // ------------------------------------------------ softmax
            if (edge) {
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int tok = tok0 + 16 * i + 8 * (e >> 1) + (g >> 1) + 4 * (g & 1);
#pragma unroll
                        for (int b = 0; b < NB; ++b)
                            if (!(i ? in1 : in0) || tok > pos[b][e & 1] ||
                                (a.window > 0 && tok <= pos[b][e & 1] - a.window))
                                x[i][b][e] = -INFINITY;
                    }
            }
            if (cr[0][0].x == 1.f) {
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 f = sc[8 * b + 2 * t4 + (e & 1)];
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            if (x[i][b][e] != -INFINITY) x[i][b][e] = fmaf(x[i][b][e], f.x, x[i][b][e] * f.y);
                    }
            }
            auto power = [&](float v, int b, int e) {
                if constexpr (TERMS == 2) return v == -INFINITY ? v : fmaf(v, cr[b][e].x, fmaf(v, cr[b][e].y, -off[b][e]));
                else return fmaf(v, cr[b][e].x, -off[b][e]);
            };
            bool far = false;
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                float top = -INFINITY;
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) top = fmaxf(top, power(x[i][b][e], b, e & 1));
                far = far || top > kBoost<T> + kSlack<T>;
            }
            if (__any_sync(0xffffffffu, far)) {
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float top = fmaxf(fmaxf(x[0][b][e], x[0][b][e + 2]), fmaxf(x[1][b][e], x[1][b][e + 2]));
#pragma unroll
                        for (int d = 4; d < 32; d *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                        // (a row that sees nothing here keeps its reference)
                        const float to = top == -INFINITY ? off[b][e] : fmaxf(off[b][e], top * cr[b][e].x - kBoost<T>);
                        const float f = exp2f(off[b][e] - to);
                        off[b][e] = to;
                        sum[b][e] *= f;
#pragma unroll
                        for (int j = 0; j < MT; ++j) {
                            o[b][j][e] *= f;
                            o[b][j][e + 2] *= f;
                        }
                    }
            }
            uint32_t pb[TERMS][2][NB][2];
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const float p0 = ex2f(power(x[i][b][2 * r], b, 0)), p1 = ex2f(power(x[i][b][2 * r + 1], b, 1));
                        sum[b][0] += p0;
                        sum[b][1] += p1;
                        const __half2 hi = __floats2half2_rn(p0, p1);
                        pb[0][i][b][r] = transpose8(*reinterpret_cast<const uint32_t *>(&hi));
                        if (TERMS == 2) {
                            const float2 f = __half22float2(hi);
                            pb[TERMS - 1][i][b][r] = transpose8(pack2<__half>(p0 - f.x, p1 - f.y));
                        }
                    }
            // ------------------------------------------------ O^T += V^T P^T
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const unsigned char *vc = tile + i * S::kHalfBytes + HALF, *vs = vc + CODES;
                uint32_t vw[4][VD / 8], vf[2][VS], sb[2][2];
#pragma unroll
                for (int r = 0; r < 2; ++r)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int row = 8 * r + t4 + 4 * e;
                        const unsigned char *src = vc + row * (D / 2) + g * (VD / 2);
                        if constexpr (VD == 8) {
                            vw[2 * r + e][0] = *reinterpret_cast<const uint32_t *>(src);
                        } else if constexpr (VD == 16) {
                            const uint2 q = *reinterpret_cast<const uint2 *>(src);
                            vw[2 * r + e][0] = q.x;
                            vw[2 * r + e][1] = q.y;
                        } else {
                            const uint4 q = *reinterpret_cast<const uint4 *>(src);
                            vw[2 * r + e][0] = q.x;
                            vw[2 * r + e][1] = q.y;
                            vw[2 * r + e][2] = q.z;
                            vw[2 * r + e][3] = q.w;
                        }
                        const unsigned char *scp = vs + row * (D / 16) + g * VD / 16;
                        if constexpr (VD == 32) sb[r][e] = *reinterpret_cast<const uint16_t *>(scp);
                        else sb[r][e] = *scp;
                    }
                if (edge) {  // (a token that no row sees may hold anything)
#pragma unroll
                    for (int r = 0; r < 2; ++r)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int tok = tok0 + 16 * i + 8 * r + t4 + 4 * e;
                            if (!(i ? in1 : in0) || tok < s.lo || tok >= s.hi) sb[r][e] = 0;
                        }
                }
#pragma unroll
                for (int r = 0; r < 2; ++r)
#pragma unroll
                    for (int w = 0; w < VS; ++w)
                        vf[r][w] = e4m3x2_to_f16(__byte_perm(sb[r][0], sb[r][1], w ? 0x0051 : 0x0040));
#pragma unroll
                for (int v8 = 0; v8 < VD / 8; ++v8) {  // eight channels at a time
                    uint32_t h0[2][4], h1[2][4];
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const uint32_t wa = vw[2 * r][v8], wb = vw[2 * r + 1][v8], f = vf[r][v8 / 2];
                        e2m1x8_to_f16((wa & 0x0f0f0f0fu) | ((wb << 4) & 0xf0f0f0f0u), h0[r]);
                        e2m1x8_to_f16(((wa >> 4) & 0x0f0f0f0fu) | (wb & 0xf0f0f0f0u), h1[r]);
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            h0[r][q] = hmul2(h0[r][q], f);
                            h1[r][q] = hmul2(h1[r][q], f);
                        }
                    }
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const uint32_t af[4] = {h0[0][q], h1[0][q], h0[1][q], h1[1][q]};
#pragma unroll
                        for (int b = 0; b < NB; ++b) {
                            float (&acc)[4] = o[b][4 * v8 + q];
                            if constexpr (TERMS == 1 && !LONG) {
                                mma_f16(acc, af, pb[0][i][b][0], pb[0][i][b][1]);
                            } else {
                                float y[4] = {};
                                if (TERMS == 2) mma_f16(y, af, pb[TERMS - 1][i][b][0], pb[TERMS - 1][i][b][1]);
                                mma_f16(y, af, pb[0][i][b][0], pb[0][i][b][1]);
#pragma unroll
                                for (int c = 0; c < 4; ++c) acc[c] += y[c];
                            }
                        }
                    }
                }
            }
        }
        copy_wait<0>();
        __syncthreads();  // the rings are free for the warps' O

        // ------------------------------------------------ the warps' parts joined
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int d = 4; d < 32; d *= 2) sum[b][e] += __shfl_xor_sync(0xffffffffu, sum[b][e], d);
                const int row = warp * ROWS + 8 * b + 2 * t4 + e;
                if (g == 0) {
                    sm[row] = off[b][e];
                    sl[row] = sum[b][e];
                }
#pragma unroll
                for (int j = 0; j < MT; j += 2)
                    *reinterpret_cast<float4 *>(so + row * S::kOStride + g * VD + 2 * j) =
                        make_float4(o[b][j][e], o[b][j][2 + e], o[b][j + 1][e], o[b][j + 1][2 + e]);
            }
        __syncthreads();
        {
            constexpr int TPR = kThreads / ROWS, PER = D / TPR;  // threads per row, channels of each
            const int row = tid / TPR, d0 = (tid % TPR) * PER;
            float m = sm[row], l = 0.f, acc[PER];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) m = fmaxf(m, sm[w * ROWS + row]);
#pragma unroll
            for (int i = 0; i < PER; ++i) acc[i] = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = exp2f(sm[w * ROWS + row] - m);
                l += f * sl[w * ROWS + row];
#pragma unroll
                for (int i = 0; i < PER; i += 4) {
                    const float4 v = *reinterpret_cast<const float4 *>(so + (w * ROWS + row) * S::kOStride + d0 + i);
                    acc[i] += f * v.x;
                    acc[i + 1] += f * v.y;
                    acc[i + 2] += f * v.z;
                    acc[i + 3] += f * v.w;
                }
            }
            if (row < s.rows) {
                if (c0 == 0 && c1 == s.chunks) {
                    const float vs = a.v_scale ? a.v_scale[h] : 1.f;
                    write_row<T, PER>(a, s, h, s.rb * ROWS + row, d0, acc, l == 0.f ? 0.f : vs / l, m, l);
                } else {
                    float *ws = partial(a.workspace, ROWS, D, 2 * blockIdx.x + (first ? 0 : 1));
#pragma unroll
                    for (int i = 0; i < PER; i += 4)
                        *reinterpret_cast<float4 *>(ws + row * D + d0 + i) =
                            make_float4(acc[i], acc[i + 1], acc[i + 2], acc[i + 3]);
                    if (d0 == 0) {
                        ws[ROWS * D + row] = m;
                        ws[ROWS * (D + 1) + row] = l;
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
template <typename T, int D, int NB>
__global__ void __launch_bounds__(32 * kJoinWarps)
attend_join_kernel(const AttendArgs a, int pairs, int row_blocks, int rows) {
    constexpr int PER = D / 32, unit_rows = 8 * NB, BLOCKS = kSms * resident(NB, D, sizeof(T) == 4);
    __shared__ float sm[kJoinWarps], sl[kJoinWarps], so[kJoinWarps][D];
    pdl_trigger();
    pdl_wait();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int u = blockIdx.x / rows, row = blockIdx.x - u * rows;
    const int p = u / a.H, h = u - p * a.H;
    const int64_t *base = reinterpret_cast<const int64_t *>(a.workspace);
    const int64_t begin = base[p], chunks = (base[p + 1] - begin) / a.H, W = base[pairs];
    if (chunks == 0) return;
    const int64_t x0 = begin + h * chunks, x1 = x0 + chunks;
    const int b0 = part_of<BLOCKS>(x0, W), b1 = part_of<BLOCKS>(x1 - 1, W);
    if (b0 == b1) return;  // written whole
    const Span s = span_of(a, p, row_blocks, unit_rows);
    if (row >= s.rows) return;
    const int later = part_begin<BLOCKS>(b0, W) < x0;  // the unit is not the first of block b0
    float m = kNoScore, l = 0.f, acc[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) acc[i] = 0.f;
    for (int q = b0 + warp; q <= b1; q += kJoinWarps) {
        const float *ws = partial(a.workspace, unit_rows, D, 2 * q + (q == b0 ? later : 0));
        const float pm = ws[unit_rows * D + row], pl = ws[unit_rows * (D + 1) + row];
        const float to = fmaxf(m, pm), f = exp2f(m - to), g = exp2f(pm - to);
        m = to;
        l = l * f + pl * g;
#pragma unroll
        for (int i = 0; i < PER; ++i) acc[i] = acc[i] * f + ws[row * D + lane + 32 * i] * g;
    }
    if (lane == 0) {
        sm[warp] = m;
        sl[warp] = l;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) so[warp][lane + 32 * i] = acc[i];
    __syncthreads();
    m = sm[0];
#pragma unroll
    for (int w = 1; w < kJoinWarps; ++w) m = fmaxf(m, sm[w]);
    float f[kJoinWarps];
    l = 0.f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
        f[w] = exp2f(sm[w] - m);
        l += f[w] * sl[w];
    }
    const float vs = a.v_scale ? a.v_scale[h] : 1.f;
    if (tid < D) {
        float o[1] = {0.f};
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w) o[0] += f[w] * so[w][tid];
        write_row<T, 1>(a, s, h, s.rb * unit_rows + row, tid, o, l == 0.f ? 0.f : vs / l, m, l);
    }
}

// A call is cut along its tokens while its units do not fill the GPU by themselves:
// then equal parts are worth the second kernel.  That is so for lengths that differ by
// four times or so; a call that is not cut takes as long as its longest unit: 94 sequences
// of 1000 tokens and one of 131072, one new token each, 850 us, and 76 with one sequence
// less, which is cut.  Tokens of 1024 to 4096, 8 key heads of 128:
// 512 units of 8 rows 57 us cut, 64 whole; 1024 100 and 97; 2048 180 and 157; 384 units
// of 16 rows 90 and 101; 512 94 and 78; 1024 161 and 127.
bool cut(int64_t pairs, int64_t H, int blocks) { return pairs <= kMaxPairs && pairs * H < blocks; }

template <typename T, int D, int NB>
cudaError_t launch_tdn(const AttendArgs &a, cudaStream_t s) {
    using S = Smem<T, D, NB>;
    constexpr int ROWS = S::kRows;
    const int64_t all = a.T * (a.Hq / a.H), rb = (all + ROWS - 1) / ROWS, pairs = a.B * rb, units = pairs * a.H;
    constexpr size_t smem = S::kBytes;
    const int blocks = kSms * resident(NB, D, sizeof(T) == 4);
    const bool whole = !cut(pairs, a.H, blocks);
    // the most tokens of a unit that a block can have, of a part where units are cut (in the
    // mean over the blocks, which have equal parts)
    const int64_t row = (int64_t)a.width << a.page_shift;
    const int64_t tokens = whole ? row : std::min<int64_t>(row, units * (row / kChunk + 1) / blocks * kChunk);
    const auto kernel = sizeof(T) == 2 && tokens > kLongTokens<T> ? attend_kernel<T, D, NB, sizeof(T) == 2> : attend_kernel<T, D, NB, false>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    if (whole) {
        if (units > INT32_MAX) return cudaErrorInvalidConfiguration;
        return launch_dependent(kernel, (unsigned)units, kThreads, smem, s, a, (int)pairs, (int)rb, true);
    }
    e = launch_dependent(kernel, (unsigned)blocks, kThreads, smem, s, a, (int)pairs, (int)rb, false);
    if (e != cudaSuccess) return e;
    const int rows = (int)std::min<int64_t>(all, ROWS);
    return launch_dependent(attend_join_kernel<T, D, NB>, (unsigned)(units * rows), 32 * kJoinWarps, 0, s, a, (int)pairs,
                            (int)rb, rows);
}

template <typename T, int D>
cudaError_t launch_td(const AttendArgs &a, cudaStream_t s) {
    return eights_of(a.T * (a.Hq / a.H)) == 1 ? launch_tdn<T, D, 1>(a, s) : launch_tdn<T, D, 2>(a, s);
}

template <typename T>
cudaError_t launch_attend(const AttendArgs &a, cudaStream_t s) {
    switch (a.D) {
    case 64: return launch_td<T, 64>(a, s);
    case 128: return launch_td<T, 128>(a, s);
    case 256: return launch_td<T, 256>(a, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

}  // namespace gdn
