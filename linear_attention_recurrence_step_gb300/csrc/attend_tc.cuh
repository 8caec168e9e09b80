// attend_tc.cuh -- attention of many query rows over the 4-bit paged cache
// (prompts), on tcgen05.
//
// A unit is up to 256 query rows (two tiles of 128; one tile for heads of 256, and
// where a sequence has no more rows) of one sequence and key head.  A CTA takes a unit,
// or, where there are few, an equal part of its tokens (a second kernel joins the parts,
// in order), TN = 128 tokens (64 for heads of 256) at a time.  Roles:
//   dequant warps  codes from global memory, a step ahead in registers, to exact
//                  f16 (code times scale, fp4.cuh) in shared memory: K and V as
//                  panels of 64 channels x TN tokens, 128-byte rows, 128-byte
//                  swizzle.  The same layout is K's K-major operand of S = Q K^T
//                  and V's N-major operand of O += P V.  Two stages.
//   issuer         S of a tile into tensor memory; then, when its probabilities
//                  are there, O += P V with P from tensor memory.  While one
//                  tile's softmax runs, the other tile's products do.
//   softmax warps  thread r owns row r of its tile: a step's scores from tensor
//                  memory to registers, their maximum, 2^(x - reference) as f16
//                  over the columns of S.  O is rescaled, by the row's thread, only
//                  when a probability would pass 2^14.
// With one tile S has two buffers instead, and S of the next step is issued
// before O += P V of this one.
//
// Per 128 x 128 x 128 step of a tile: 2 x 512 cycles of products, 16384
// exponentials and 64 KB through shared memory by the products (512 + 256
// cycles), 32 KB of operands written (256 cycles, no bank conflicts).  Measured:
// 2048 tokens over 8192, 32 heads of 128 on 8 of the cache, in 191 us (1.26
// PFLOP/s of products, 0.66 of a library product's rate), 197 with cold caches, 369 over
// 16384: 1.4 us a step of two tiles, and 9 us a unit for its queries, first step and
// output.  The products and the dequant warps share the shared memory, which is what
// bounds the steps.
//
// Registers: 192 for a softmax thread, so that a step's 128 scores stay in them.
// Spills there cost most of all (106 bytes of them: 249 us for 193).
//
// Operands and softmax are those of kv_attend.cuh; sums stay in tensor memory in
// float32, for 16384 tokens at a time (kTcCarry).  Every wait is bounded; when one runs
// out, the unit's rows are written as NaN and the library's wait flag is raised.
#pragma once

#include <algorithm>
#include <cfloat>

#include "attend.h"
#include "fp4.cuh"
#include "pieces.cuh"
#include "tma.cuh"

namespace gdn {

namespace {

constexpr int kTcThreads = 512;   // warpgroups: softmax, softmax (or dequant), dequant, issuer (one warp of it)
constexpr int kTcTile = 128;                              // query rows of a tile
constexpr uint32_t kTmemCols = 512, kTmemO = 256;         // S buffers at 0 and 128, O from 256 on
constexpr int kTcSms = 152;
constexpr long long kDrainCycles = 2000000000ll;
// A row's largest probability when its reference is set is 2^6; the reference
// moves when one passes 2^14.  f16 steps end at 2^-24: weights are off by 2^-12 of
// themselves, or by 2^-31 of the row's largest.
constexpr float kTcBoost = 6.f, kTcMost = 14.f;
// The tensor cores cut a sum off where they add to it, so an O whose terms have one sign
// falls short by half a unit of its last place per 16 tokens: 7.8e-4 of it over 131072.
// After every so many tokens the rows' threads take the larger part of O out of the
// tensor memory, which leaves 7e-5.  That code is in kernels of its own (LONG), for calls
// whose parts can be so long: without ever running, it takes 197 us of 191 for 2048 tokens
// over 8192; over 65536 they take 1589 us for 1535.
constexpr int kTcCarry = 16384;
constexpr float kTcNoScore = -FLT_MAX;  // the reference of a row that has seen nothing
// Whether scores of a factor can reach 2^26 in powers of two: they are rounded then before
// the reference is taken off (kv_attend.cuh).
__device__ __forceinline__ bool far_scores(float factor, int D) { return factor * (float)D >= 0x1p26f / (2048.f * 2688.f); }

template <int D, int TILES> struct Tc {
    static constexpr int kTiles = TILES;
    static constexpr int kRows = kTiles * kTcTile;
    static constexpr int kTok = D == 256 ? 64 : 128;       // tokens per step
    static constexpr int kDqWarps = 12 - 4 * TILES;
    static constexpr uint32_t kQBytes = kRows * D * 2, kOpBytes = kTok * D * 2;  // K or V of a step
    static constexpr uint32_t kQ = 0, kK = kQBytes, kV = kK + 2 * kOpBytes, kBars = kV + 2 * kOpBytes;
    static constexpr uint32_t kFactors = kBars + 256;      // f32 per row, where scores are rounded
    static constexpr uint32_t kHeld = kFactors + 4 * kRows;  // f32 per row: the factor of what is held outside O, 0: nothing
    static constexpr size_t kSmem = kHeld + 4 * kRows + 1024;  // (1024: alignment)
};
enum Bar { kKFull = 0, kVFull = 2, kKFree = 4, kVFree = 6, kSFull = 8, kPFull = 10, kODone = 12, kDrain = 14, kNever = 15, kBarCount = 16 };

// Operand descriptors of 128-byte swizzled panels: the low word (address and
// leading offset) and the high one, the same for all (8-row groups 1024 bytes
// apart, version 1, the swizzle).
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_low(uint32_t addr, uint32_t lbo) {
    return ((addr >> 4) & 0x3fffu) | ((lbo >> 4) << 16);
}
// kind::f16: f16 A and B, f32 accumulator, M = 128, N = n; B K-major or N-major.
constexpr uint32_t op_desc(int n, bool n_major) {
    return (1u << 4) | (n_major ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24);
}
// One thread of the warp issues (`one`), so that the warp stays together and
// descriptors are uniform: a branch around each product costs 100 cycles in
// moves to uniform registers.
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t r;
    asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
    return r;
}
__device__ __forceinline__ void mma_ss(uint32_t one, uint32_t d, uint32_t a, uint32_t b, uint32_t op, uint32_t add) {
    asm volatile("{\n.reg .pred p, q;\n.reg .b64 a, b;\nsetp.ne.b32 p, %4, 0;\nsetp.ne.b32 q, %5, 0;\n"
                 "mov.b64 a, {%1, %6};\nmov.b64 b, {%2, %6};\n"
                 "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n}\n" ::"r"(d),
                 "r"(a), "r"(b), "r"(op), "r"(add), "r"(one), "r"(kDescHigh)
                 : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t one, uint32_t d, uint32_t a, uint32_t b, uint32_t op, uint32_t add) {
    asm volatile("{\n.reg .pred p, q;\n.reg .b64 b;\nsetp.ne.b32 p, %4, 0;\nsetp.ne.b32 q, %5, 0;\n"
                 "mov.b64 b, {%2, %6};\n"
                 "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n}\n" ::"r"(d),
                 "r"(a), "r"(b), "r"(op), "r"(add), "r"(one), "r"(kDescHigh)
                 : "memory");
}
__device__ __forceinline__ void commit_to(uint32_t one, uint32_t bar) {
    asm volatile("{\n.reg .pred q;\nsetp.ne.b32 q, %1, 0;\n"
                 "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(bar), "r"(one)
                 : "memory");
}
__device__ __forceinline__ void tm_before() { asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory"); }
__device__ __forceinline__ void tm_after() { asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory"); }
__device__ __forceinline__ void tm_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory"); }
__device__ __forceinline__ void tm_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }
// 32 columns of the thread's lane; 32 and 16 columns written.
__device__ __forceinline__ void tm_ld32(uint32_t t, float *v) {  // (valid after tm_wait_ld)
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(t));
#pragma unroll
    for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(r[e]);
}
__device__ __forceinline__ void tm_st32(uint32_t t, const float (&v)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};\n" ::"r"(t),
        "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]), "f"(v[9]),
        "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15]), "f"(v[16]), "f"(v[17]), "f"(v[18]),
        "f"(v[19]), "f"(v[20]), "f"(v[21]), "f"(v[22]), "f"(v[23]), "f"(v[24]), "f"(v[25]), "f"(v[26]), "f"(v[27]),
        "f"(v[28]), "f"(v[29]), "f"(v[30]), "f"(v[31])
        : "memory");
}
__device__ __forceinline__ void tm_st16(uint32_t t, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(t),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ uint32_t times2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;\n" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ void st_shared16(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};\n" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// Whether the phase of this parity is complete (without the clock that a bounded
// wait starts by reading).
__device__ __forceinline__ bool passed(uint32_t bar, uint32_t parity) {
    uint32_t done;
    asm volatile("{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}\n"
                 : "=r"(done)
                 : "r"(bar), "r"(parity)
                 : "memory");
    return done != 0;
}
template <int N> __device__ __forceinline__ void more_registers() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(N));
}
template <int N> __device__ __forceinline__ void less_registers() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(N));
}

struct TcArgs {
    AttendArgs a;
    int parts;              // of a unit's tokens
    int part_rows;          // rows of a partial result
    unsigned *wait_flag;
    long long wait_cycles;
    int inject_expiry;
};

// The first token that a query at position pos sees.  (Positions before the first
// token count as -1: that less a window of up to 2^31 - 1 stays in 32 bits.)
__device__ __forceinline__ int first_seen(const AttendArgs &a, int pos) {
    return a.window > 0 ? max(max(pos, -1) - a.window + 1, 0) : 0;
}

// Row block rb of sequence b: the tokens [lo, hi) that any of its rows sees, and the
// steps over them (one at least where there are rows: those that see nothing are
// written too).
struct TcSpan {
    int r0, rows, n, len, lo, hi, step0, steps;
};
template <int D, int TILES> __device__ __forceinline__ TcSpan tc_span(const AttendArgs &a, int b, int rb) {
    using L = Tc<D, TILES>;
    TcSpan s;
    const int G = a.Hq / a.H;
    s.n = a.fresh ? min(max(a.fresh[b], 0), (int)a.T) : (int)a.T;
    s.len = (int)min((int64_t)max(a.lengths[b], 0), (int64_t)a.width << a.page_shift);
    s.r0 = rb * L::kRows;
    s.rows = min(max(s.n * G - s.r0, 0), L::kRows);
    const int first = s.len - s.n + s.r0 / G, last = s.len - s.n + (s.r0 + max(s.rows, 1) - 1) / G;
    s.hi = max(last + 1, 0);
    s.lo = first_seen(a, first);
    s.step0 = s.lo / L::kTok;
    s.steps = s.rows == 0 ? 0 : max((s.hi + L::kTok - 1) / L::kTok - s.step0, 1);
    return s;
}

template <typename T, int D, int TILES, bool LONG>
__global__ void __launch_bounds__(kTcThreads, 1) attend_tc_kernel(const TcArgs ta) {
    using L = Tc<D, TILES>;
    constexpr int TN = L::kTok;
    const AttendArgs &a = ta.a;
    extern __shared__ unsigned char smem_raw[];
    const uint32_t base = (sh_addr(smem_raw) + 1023u) & ~1023u;
    auto bar = [&](int i) { return base + L::kBars + 8u * (uint32_t)i; };
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem_raw + (base - sh_addr(smem_raw)) + L::kBars + 8 * kBarCount);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(sh_addr(tmem_slot)),
                     "r"(kTmemCols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n");
    }
    if (tid == 0) {
        for (int i = 0; i < kBarCount; ++i)
            mbar_init(bar(i), i < kKFree ? L::kDqWarps : i == kPFull || i == kPFull + 1 ? 4 : 1);
        mbar_init_fence();
    }
    tm_before();
    __syncthreads();
    tm_after();
    const uint32_t tmem = *tmem_slot;
    pdl_trigger();
    pdl_wait();

    // ------------------------------------------------ the unit, and this part of it
    const int G = a.Hq / a.H, page = 1 << a.page_shift;
    // later row blocks see more tokens: those first
    const int ordered = (int)(gridDim.x - 1 - blockIdx.x), u = ordered / ta.parts, part = ordered - u * ta.parts;
    const int h = u % a.H, b = u / a.H % (int)a.B, rb = u / a.H / (int)a.B;
    const TcSpan span = tc_span<D, TILES>(a, b, rb);
    const int n = span.n, len = span.len, r0 = span.r0, rows = span.rows, lo = span.lo, hi = span.hi;
    const int tiles = rows > kTcTile ? 2 : 1;
    const int j0 = (int)((int64_t)part * span.steps / ta.parts);
    const int step0 = span.step0 + j0, steps = (int)((int64_t)(part + 1) * span.steps / ta.parts) - j0;
    const int32_t *table = a.table + (int64_t)b * a.width;
    // the table's entry for the 16 tokens `lane` (of TN) of step j, -1: none of them
    // is seen.  (Whether it names a page is asked where it is used, a step later:
    // here the warp would wait for it.)
    const uint32_t pool = (uint32_t)a.pages;
    auto pages_of = [&](int j) {
        const int tok = (step0 + j) * TN + 16 * lane;
        int id = -1;
        if (j < steps && lane < TN / 16 && tok < hi && tok + 16 > lo) id = table[tok >> a.page_shift];
        return id;
    };
    bool ok = true;
    // by a whole warp: all of it goes on, or none
    auto wait = [&](int i, uint32_t parity) {
        if (ok && !__all_sync(0xffffffffu, passed(bar(i), parity & 1u)))
            ok = __all_sync(0xffffffffu, mbar_wait_bounded(bar(i), parity & 1u, ta.wait_cycles));
        return ok;
    };
    if (ta.inject_expiry) wait(kNever, 0);

    const bool softmax_warp = warp < 4 * L::kTiles;
    float sum = 0.f, off = kTcNoScore;
    // registers where they are used: 4 x 128 at launch, as many or fewer in all
    if (softmax_warp) {
        more_registers<192>();  // (192 + 192 + 88 + 40, or 192 + 120 + 120 + 40)
        // ================================================ softmax warps
        const int t = warp >> 2, row = tid & 127, r = r0 + t * kTcTile + row;  // tile, row in it, row of the sequence
        const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);  // this warp's 32 lanes
        const int pos = len - n + r / G;
        // D/8 lanes share a row of q or y, eight channels each
        constexpr int LR = D / 8, RI = 32 / LR;
        const int piece = lane % LR, warp_row = t * kTcTile + (row & ~31);
        auto place = [&](int at_row) {  // of the piece, in the panels of 64 channels x kRows rows
            return base + L::kQ + (uint32_t)(piece / 8) * (L::kRows * 128) + at_row * 128 + (((piece & 7) ^ (at_row & 7)) << 4);
        };
        float c = FLT_MIN;
        if (t < tiles && steps > 0) {
            // the warp's 32 rows to f16, each scaled by a power of two, with the scale's
            // sign; eight loads in flight
            const T *const q = static_cast<const T *>(a.q) + b * a.q_sb + 8 * piece;
            const float factor = fabsf(a.scale) * 1.44269504088896341f * (a.k_scale ? a.k_scale[h] : 1.f);
#pragma unroll 1
            for (int i0 = 0; i0 < LR; i0 += 8) {
                RawPiece<T, 8> raw[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int at_row = warp_row + (i0 + i) * RI + lane / LR, qr = r0 + at_row, qt = qr / G;
                    const T *from = q + qt * a.q_st + (int64_t)(h * G + qr - qt * G) * D;
                    raw[i].w = make_uint4(0, 0, 0, 0);
                    if (at_row < rows) {
                        if (a.vec_q) {
                            raw[i] = load_raw<T, 8>(from);
                        } else {
                            const uint16_t *e = reinterpret_cast<const uint16_t *>(from);
                            raw[i].w = make_uint4(e[0] | (uint32_t)e[1] << 16, e[2] | (uint32_t)e[3] << 16,
                                                  e[4] | (uint32_t)e[5] << 16, e[6] | (uint32_t)e[7] << 16);
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float v[8], top = 0.f;
                    widen<T, 8>(v, raw[i]);
#pragma unroll
                    for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(v[e]));
#pragma unroll
                    for (int d = 1; d < LR; d *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                    // (an infinite row is made NaN: scores of -inf would count as masked ones)
                    const bool finite = top < INFINITY;
                    const int e2 = finite ? max((int)(__float_as_uint(top) >> 23) - 127, -100) : 10;
                    const float up = copysignf(__uint_as_float(finite ? (uint32_t)(127 + 10 - e2) << 23 : 0x7fc00000u), a.scale);
                    st_shared16(place(warp_row + (i0 + i) * RI + lane / LR), pack2<__half>(v[0] * up, v[1] * up),
                                pack2<__half>(v[2] * up, v[3] * up), pack2<__half>(v[4] * up, v[5] * up),
                                pack2<__half>(v[6] * up, v[7] * up));
                    // the factor of the scores to the row's own thread
                    const int mine = __shfl_sync(0xffffffffu, e2, lane % RI * LR);
                    if (lane / RI == i0 + i) c = fmaxf(factor * __uint_as_float((uint32_t)(127 + mine - 10) << 23), FLT_MIN);
                }
            }
        }
        asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
        named_bar_sync(1, 32 * (4 * L::kTiles + 1));  // with the issuer: the queries are there

        // visible tokens of the row: [row_lo, row_hi)
        const int row_hi = min(pos + 1, hi), row_lo = first_seen(a, pos);
        // tokens that every row of the tile sees
        const int tr0 = r0 + t * kTcTile, tr1 = r0 + min(rows, (t + 1) * kTcTile) - 1;
        const int all_hi = len - n + tr0 / G + 1, all_lo = first_seen(a, len - n + tr1 / G);
        // What is held of O is, in a unit that is written whole, the row's y, rounded to its
        // type below a power of two (the rest stays in O); in a part its partial result.
        auto held_at = [&]() { return base + L::kHeld + 4u * threadIdx.x; };
        auto held_factor = [&]() {
            float f;
            asm volatile("ld.shared.f32 %0, [%1];\n" : "=f"(f) : "r"(held_at()));
            return f;
        };
        auto hold_factor = [&](float f) { asm volatile("st.shared.f32 [%0], %1;\n" ::"r"(held_at()), "f"(f) : "memory"); };
        const auto y_row = [&]() {
            const int qt = r / G;
            return static_cast<T *>(a.y) + (((int64_t)b * a.T + qt) * a.Hq + h * G + r - qt * G) * D;
        };
        // (channel d of row i at [d][i], so that a warp's stores are whole lines)
        const auto part_row = [&]() {
            return a.workspace + ((int64_t)u * ta.parts + part) * ((D + 2) * (int64_t)ta.part_rows) + t * kTcTile + row;
        };
        auto add_held = [&](int k, float f, float (&v)[32]) {  // 32 channels from 32 k on
            if (ta.parts == 1) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const T *y = y_row() + 32 * k + 8 * i;
                    float x[8];
                    if (a.vec_y) {
                        load_piece<T, 8>(x, y);
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e) x[e] = ld_f32(y + e);
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[8 * i + e] = fmaf(x[e], f, v[8 * i + e]);
                }
            } else {
#pragma unroll
                for (int e = 0; e < 32; ++e) v[e] = fmaf(part_row()[(32 * k + e) * ta.part_rows], f, v[e]);
            }
        };
        auto carry = [&]() {
            const float f = held_factor();
            // a power of two above the sum of the weights: O is below 2688 of it
            const uint32_t two = ta.parts == 1 ? (__float_as_uint(fmaxf(sum, 0x1p-100f)) & 0x7f800000u) + 0x00800000u : 0x3f800000u;
            const float to = __uint_as_float(two), inv = __uint_as_float(0x7f000000u - two);
            const bool there = t * kTcTile + row < rows;
#pragma unroll 1
            for (int k = 0; k < D / 32; ++k) {
                float w[32];
                const uint32_t o_at = lanes + kTmemO + (uint32_t)(t * D + 32 * k);
                tm_ld32(o_at, w);
                tm_wait_ld();
                if (there) {
                    if (f != 0.f) add_held(k, f, w);
                    if (ta.parts == 1) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            T *y = y_row() + 32 * k + 8 * i;
                            float x[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) x[e] = w[8 * i + e] * inv;
                            const RawPiece<T, 8> piece8 = narrow_piece<T, 8>(x);
                            widen<T, 8>(x, piece8);
                            if (a.vec_y) {
                                store_raw<T, 8>(y, piece8);
                            } else {
#pragma unroll
                                for (int e = 0; e < 8; ++e) st_from_f32(y + e, x[e]);
                            }
#pragma unroll
                            for (int e = 0; e < 8; ++e) w[8 * i + e] = fmaf(-x[e], to, w[8 * i + e]);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            part_row()[(32 * k + e) * ta.part_rows] = w[e];
                            w[e] = 0.f;
                        }
                    }
                }
                __syncwarp();
                tm_st32(o_at, w);
            }
            tm_wait_st();
            hold_factor(to);
        };
        if (LONG) hold_factor(0.f);
        int ids = t < tiles ? pages_of(0) : -1;
        // the warp's scores are rounded: their factor is 1 then, which is far itself
        auto factor_at = [&]() { return base + L::kFactors + 4u * threadIdx.x; };
        if (__any_sync(0xffffffffu, far_scores(c, D))) {
            asm volatile("st.shared.f32 [%0], %1;\n" ::"r"(factor_at()), "f"(c) : "memory");
            c = 1.f;
        }
        for (int j = 0; j < steps && t < tiles; ++j) {
            const int buf = tiles == 2 ? t : j & 1;
            const uint32_t s_at = lanes + 128u * (uint32_t)buf;
            const unsigned present = __ballot_sync(0xffffffffu, (uint32_t)ids < pool);  // bit i: tokens 16 i on
            ids = pages_of(j + 1);
            if (!wait(kSFull + buf, tiles == 2 ? j : j >> 1)) break;
            if (t * kTcTile + (row & ~31) >= rows) {  // none of the warp's rows: what S holds is no one's P
                if (lane == 0) mbar_arrive(bar(kPFull + buf));
                continue;
            }
            tm_after();
            if (LONG && j > 0 && j % (kTcCarry / TN) == 0) {
                if (!wait(kODone + t, j - 1)) break;
                tm_after();
                carry();
            }
            const int tok0 = (step0 + j) * TN;
            const bool edge = tok0 < all_lo || tok0 + TN > all_hi || present != (1u << (TN / 16)) - 1u;
            const int c_lo = row_lo - tok0, c_hi = row_hi - tok0;
            float v[TN];
#pragma unroll
            for (int k = 0; k < TN / 32; ++k) tm_ld32(s_at + 32u * k, v + 32 * k);
            tm_wait_ld();
            if (edge) {
#pragma unroll
                for (int q = 0; q < TN / 32; ++q) {
                    const int from = min(max(c_lo - 32 * q, 0), 32), to = min(max(c_hi - 32 * q, 0), 32);
                    uint32_t seen = (uint32_t)((1ull << to) - 1) & ~(uint32_t)((1ull << from) - 1);
                    if (!((present >> (2 * q)) & 1u)) seen &= 0xffff0000u;
                    if (!((present >> (2 * q + 1)) & 1u)) seen &= 0x0000ffffu;
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (!((seen >> i) & 1u)) v[32 * q + i] = -INFINITY;
                }
            }
            if (c == 1.f) {
                float f;
                asm volatile("ld.shared.f32 %0, [%1];\n" : "=f"(f) : "r"(factor_at()));
#pragma unroll
                for (int e = 0; e < TN; ++e) v[e] = __fmul_rn(v[e], f);
            }
            float tops[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
            for (int e = 4; e < TN; ++e) tops[e % 4] = fmaxf(tops[e % 4], v[e]);
            const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
            // the reference moves, and sum and O with it
            if (__any_sync(0xffffffffu, fmaf(top, c, -off) > kTcMost)) {
                const float to = top == -INFINITY ? off : fmaxf(off, top * c - kTcBoost);
                const float f = exp2f(off - to);
                off = to;
                sum *= f;
                if (j > 0) {
                    if (!wait(kODone + t, j - 1)) break;
                    tm_after();
#pragma unroll 1
                    for (int k = 0; k < D / 32; ++k) {
                        float w[32];
                        const uint32_t o_at = lanes + kTmemO + (uint32_t)(t * D + 32 * k);
                        tm_ld32(o_at, w);
                        tm_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) w[e] *= f;
                        tm_st32(o_at, w);
                    }
                    tm_wait_st();
                    if (LONG) hold_factor(held_factor() * f);
                }
            }
            const float2 c2 = make_float2(c, c), off2 = make_float2(-off, -off);
            float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
            for (int k = 0; k < TN / 32; ++k) {
                uint32_t p[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float2 x = ffma2(make_float2(v[32 * k + 2 * e], v[32 * k + 2 * e + 1]), c2, off2);
                    const float2 y = make_float2(ex2f(x.x), ex2f(x.y));
                    acc[e & 1] = __fadd2_rn(acc[e & 1], y);
                    p[e] = pack2<__half>(y.x, y.y);
                }
                tm_st16(s_at + 16u * k, p);
            }
            acc[0] = __fadd2_rn(acc[0], acc[1]);
            sum += acc[0].x + acc[0].y;
            tm_wait_st();
            // (one tile's S runs ahead of its O: O's phases are followed step by step, for
            // a phase can only be told from the one before it)
            if (tiles == 1 && j > 0 && !wait(kODone + t, j - 1)) break;
            tm_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kPFull + buf));
        }

        // ------------------------------------------------ the row's output
        if (t < tiles && t * kTcTile + (row & ~31) < rows) {
            if (steps > 0) wait(kODone + t, steps - 1);
            tm_after();
            const bool there = t * kTcTile + row < rows;
            const float bad = __int_as_float(0x7fc00000), held = LONG && steps > 0 ? held_factor() : 0.f;
            if (ta.parts == 1) {
                const float vs = a.v_scale ? a.v_scale[h] : 1.f;
                const float inv = !ok ? bad : sum == 0.f ? 0.f : vs / sum;
#pragma unroll 1
                for (int k = 0; k < D / 32; ++k) {
                    float v[32];
                    tm_ld32(lanes + kTmemO + (uint32_t)(t * D + 32 * k), v);
                    tm_wait_ld();
                    if (LONG && held != 0.f && there) add_held(k, held, v);
                    // (where the queries were: their last product is done)
                    const uint32_t at_row = base + L::kQ + (uint32_t)(k / 2) * (L::kRows * 128) + (t * kTcTile + row) * 128;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float w[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) w[e] = ok ? v[8 * i + e] * inv : bad;
                        const RawPiece<T, 8> x = narrow_piece<T, 8>(w);
                        st_shared16(at_row + (((k % 2 * 4 + i) ^ (row & 7)) << 4), x.w.x, x.w.y, x.w.z, x.w.w);
                    }
                }
                __syncwarp();
#pragma unroll 4
                for (int i = 0; i < LR; ++i) {  // whole rows, from the lanes that share them
                    const int at_row = warp_row + i * RI + lane / LR, yr = r0 + at_row, yt = yr / G;
                    uint4 w;
                    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                                 : "r"(place(at_row)));
                    if (at_row >= rows) continue;
                    T *y = static_cast<T *>(a.y) + (((int64_t)b * a.T + yt) * a.Hq + h * G + yr - yt * G) * D + 8 * piece;
                    if (a.vec_y) {
                        *reinterpret_cast<uint4 *>(y) = w;
                    } else {
                        uint16_t *e = reinterpret_cast<uint16_t *>(y);
                        const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                        for (int j = 0; j < 8; ++j) e[j] = (uint16_t)(x[j / 2] >> (16 * (j % 2)));
                    }
                }
                if (there && a.lse) {
                    const int qt = r / G;
                    a.lse[((int64_t)b * a.T + qt) * a.Hq + h * G + r - qt * G] =
                        !ok ? bad : sum == 0.f ? -INFINITY : (off + log2f(sum)) * 0.693147180559945309f;
                }
            } else {
                float *ws = a.workspace + ((int64_t)u * ta.parts + part) * ((D + 2) * (int64_t)ta.part_rows);
                const int i = t * kTcTile + row;
                if (steps > 0) {
#pragma unroll 1
                    for (int k = 0; k < D / 32; ++k) {
                        float v[32];
                        tm_ld32(lanes + kTmemO + (uint32_t)(t * D + 32 * k), v);
                        tm_wait_ld();
                        if (there) {
                            if (LONG && held != 0.f) add_held(k, held, v);
#pragma unroll
                            for (int e = 0; e < 32; ++e) ws[(32 * k + e) * ta.part_rows + i] = v[e];
                        }
                        __syncwarp();
                    }
                }
                if (there) {
                    ws[D * ta.part_rows + i] = off;
                    ws[(D + 1) * ta.part_rows + i] = ok ? sum : bad;
                }
            }
        }
    } else if (warp < 12) {
        less_registers<TILES == 1 ? 120 : 88>();
        // ================================================ dequant warps
        // A job is 32 neighbouring channels of a token: 16 bytes of codes, two
        // scales.  D/32 lanes share a token; a warp's jobs are neighbouring tokens,
        // those of 16 tokens in one page.
        constexpr int LPR = D / 32, RPI = 32 / LPR, JOBS = TN / (RPI * L::kDqWarps);
        constexpr int PAGES = JOBS * RPI >= 16 ? JOBS * RPI / 16 : 1, JPP = JOBS / PAGES;
        const int w = warp - 4 * L::kTiles, piece = lane % LPR, sub = lane / LPR, panel = piece >> 1;
        const int first = w * JOBS * RPI + sub;  // the token of job 0, in the step
        // the order of a job's four words, so that eight lanes write distinct banks
        const int order = D == 256 ? panel : D == 128 ? 2 * panel : 0;
        const uint32_t page_bytes = (uint32_t)(a.H * kv_block_bytes(page, D));
        const unsigned char *cache = a.cache + h * kv_block_bytes(page, D) + 16 * piece;
        const unsigned char *scales = a.cache + h * kv_block_bytes(page, D) + page * (D / 2) + 2 * piece;
        const int values = page * (D / 2 + D / 16);
        const uint32_t pick[2] = {order & 2 ? 0x3232u : 0x1010u, order & 2 ? 0x1010u : 0x3232u};
        uint32_t chunk[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            chunk[k] = (uint32_t)panel * (TN * 128) + first * 128 + ((((piece & 1) * 4 + (k ^ order)) ^ (first & 7)) << 4);
        // steps read ahead: two where a warp's share of one is few registers
        constexpr int AHEAD = JOBS <= 2 ? 2 : 1;
        uint2 kq[AHEAD][JOBS][2], vq[AHEAD][JOBS][2];
        uint32_t ks[AHEAD][JOBS], vs[AHEAD][JOBS];
        auto load = [&](int j, int ids, int at, uint2 (&q)[JOBS][2], uint32_t (&sc)[JOBS]) {
            const int t0 = (step0 + j) * TN;
            const bool full = t0 >= lo && t0 + TN <= hi;
#pragma unroll
            for (int p = 0; p < PAGES; ++p) {
                const int id = __shfl_sync(0xffffffffu, ids, (w * JOBS * RPI + 16 * p) >> 4);
                const int in = first + 16 * p, row = (t0 + in) & (page - 1);
                const uint64_t off = (uint64_t)(uint32_t)id * page_bytes + (uint32_t)at;
                const unsigned char *c = cache + off + row * (D / 2), *s = scales + off + row * (D / 16);
#pragma unroll
                for (int i = 0; i < JPP; ++i) {
                    const int job = p * JPP + i, tok = t0 + in + i * RPI;
                    q[job][0] = q[job][1] = make_uint2(0, 0);
                    sc[job] = 0;
                    if ((uint32_t)id < pool && (full || (tok >= lo && tok < hi))) {
                        // (the halves in the order that they are written in)
                        q[job][0] = *reinterpret_cast<const uint2 *>(c + i * RPI * (D / 2) + 4 * (order & 2));
                        q[job][1] = *reinterpret_cast<const uint2 *>(c + i * RPI * (D / 2) + 8 - 4 * (order & 2));
                        sc[job] = *reinterpret_cast<const uint16_t *>(s + i * RPI * (D / 16));
                    }
                }
            }
        };
        auto store = [&](uint32_t dst, const uint2 (&q)[JOBS][2], const uint32_t (&sc)[JOBS]) {
#pragma unroll
            for (int i = 0; i < JOBS; ++i) {
                const uint32_t both = e4m3x2_to_f16(sc[i]);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint32_t x = k % 2 ? q[i][k / 2].y : q[i][k / 2].x;
                    if (D == 256 && (order & 1)) x = k % 2 ? q[i][k / 2].x : q[i][k / 2].y;
                    const uint32_t f = __byte_perm(both, both, pick[k / 2]);
                    uint32_t e[4];
                    e2m1x8_to_f16(x, e);
                    st_shared16(dst + (chunk[k] ^ (((i * RPI) & 7) << 4)) + i * RPI * 128, times2(e[0], f), times2(e[1], f),
                                times2(e[2], f), times2(e[3], f));
                }
            }
            asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
            __syncwarp();
        };
#pragma unroll
        for (int p = 0; p < AHEAD; ++p) {
            const int ids = pages_of(p);
            load(p, ids, 0, kq[p], ks[p]);
            load(p, ids, values, vq[p], vs[p]);
        }
        int ids_next = pages_of(AHEAD);
        for (int j0 = 0; j0 < steps && ok; j0 += AHEAD) {
#pragma unroll
            for (int p = 0; p < AHEAD; ++p) {
                const int j = j0 + p, st = j & 1, ids = ids_next;
                if (j >= steps) break;
                ids_next = pages_of(j + AHEAD + 1);
                if (j >= 2 && !wait(kKFree + st, (j >> 1) - 1)) break;
                store(base + L::kK + st * L::kOpBytes, kq[p], ks[p]);
                if (lane == 0) mbar_arrive(bar(kKFull + st));
                load(j + AHEAD, ids, 0, kq[p], ks[p]);
                if (j >= 2 && !wait(kVFree + st, (j >> 1) - 1)) break;
                store(base + L::kV + st * L::kOpBytes, vq[p], vs[p]);
                if (lane == 0) mbar_arrive(bar(kVFull + st));
                load(j + AHEAD, ids, values, vq[p], vs[p]);
            }
        }
    } else {
        less_registers<40>();
        // ================================================ issuer
        if (warp == 12) {
            named_bar_sync(1, 32 * (4 * L::kTiles + 1));
            constexpr uint32_t op_s = op_desc(TN, false), op_o = op_desc(D, true);
            const uint32_t one = elect_one(), tm = __shfl_sync(0xffffffffu, tmem, 0);
            const uint32_t sbase = __shfl_sync(0xffffffffu, base, 0);
            auto issue_s = [&](int j, int t) {
                const int buf = tiles == 2 ? t : j & 1;
                if (!wait(kKFull + (j & 1), j >> 1)) return;
                tm_after();
                const uint32_t q = desc_low(sbase + L::kQ + t * kTcTile * 128, 16);
                const uint32_t k = desc_low(sbase + L::kK + (j & 1) * L::kOpBytes, 16);
#pragma unroll
                for (int s = 0; s < D / 16; ++s)
                    mma_ss(one, tm + 128u * buf, q + ((s >> 2) * (L::kRows * 128) + (s & 3) * 32) / 16,
                           k + ((s >> 2) * (TN * 128) + (s & 3) * 32) / 16, op_s, s > 0);
                commit_to(one, bar(kSFull + buf));
                if (t == tiles - 1) commit_to(one, bar(kKFree + (j & 1)));
            };
            auto issue_o = [&](int j, int t) {
                const int buf = tiles == 2 ? t : j & 1;
                if (!wait(kVFull + (j & 1), j >> 1) || !wait(kPFull + buf, tiles == 2 ? j : j >> 1)) return;
                tm_after();
                const uint32_t v = desc_low(sbase + L::kV + (j & 1) * L::kOpBytes, TN * 128);
#pragma unroll
                for (int s = 0; s < TN / 16; ++s)
                    mma_ts(one, tm + kTmemO + (uint32_t)(t * D), tm + 128u * buf + 8u * s, v + s * 2048 / 16, op_o, j > 0 || s > 0);
                commit_to(one, bar(kODone + t));
                if (t == tiles - 1) commit_to(one, bar(kVFree + (j & 1)));
            };
            if (steps > 0)
                for (int t = 0; t < tiles; ++t) issue_s(0, t);
            for (int j = 0; j < steps && ok; ++j) {
                if (tiles == 1 && j + 1 < steps) issue_s(j + 1, 0);
                for (int t = 0; t < tiles; ++t) {
                    issue_o(j, t);
                    if (tiles == 2 && j + 1 < steps) issue_s(j + 1, t);
                }
            }
            // nothing is in flight when the tensor memory goes
            commit_to(one, bar(kDrain));
            if (!mbar_wait_bounded(bar(kDrain), 0, kDrainCycles)) ok = false;
        }
    }
    if (!ok) *ta.wait_flag = 1u;
    tm_before();
    __syncthreads();
    tm_after();
    if (warp == 0)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(kTmemCols));
}

// Joins a unit's parts: a block per eight of its rows.
template <typename T, int D, int TILES>
__global__ void __launch_bounds__(256) attend_tc_join_kernel(const AttendArgs a, int parts, int part_rows, int groups) {
    __shared__ float so[D][9];
    pdl_trigger();
    pdl_wait();
    const int u = blockIdx.x / groups, i0 = (blockIdx.x - u * groups) * 8, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int h = u % a.H, b = u / a.H % (int)a.B, rb = u / a.H / (int)a.B, G = a.Hq / a.H;
    const TcSpan s = tc_span<D, TILES>(a, b, rb);
    if (i0 >= s.rows) return;
    // eight neighbouring rows of a channel are 32 bytes: the lane of channel
    // lane / 8 of the warp's four and row lane % 8 adds them up
    const int i = i0 + lane % 8;
    const bool there = i < s.rows;
    float ref = kTcNoScore, sum = 0.f, acc[D / 32];
#pragma unroll
    for (int k = 0; k < D / 32; ++k) acc[k] = 0.f;
#pragma unroll 2
    for (int q = 0; q < parts; ++q) {
        const float *ws = a.workspace + ((int64_t)u * parts + q) * ((D + 2) * (int64_t)part_rows);
        const float pr = there ? ws[D * part_rows + i] : 0.f, ps = there ? ws[(D + 1) * part_rows + i] : 0.f;
        if (ps == 0.f) continue;  // (it had no steps, or saw nothing)
        const float to = fmaxf(ref, pr), f = exp2f(ref - to), g = exp2f(pr - to);
        ref = to;
        sum = sum * f + ps * g;
#pragma unroll
        for (int k = 0; k < D / 32; ++k) acc[k] = acc[k] * f + ws[(32 * k + 4 * warp + lane / 8) * part_rows + i] * g;
    }
    const float vs = a.v_scale ? a.v_scale[h] : 1.f, inv = sum == 0.f ? 0.f : vs / sum;
#pragma unroll
    for (int k = 0; k < D / 32; ++k) so[32 * k + 4 * warp + lane / 8][lane % 8] = acc[k] * inv;
    auto place = [&](int row) {
        const int r = s.r0 + row, t = r / G;
        return ((int64_t)b * a.T + t) * a.Hq + h * G + r - t * G;
    };
    if (threadIdx.x < 8 && there && a.lse)
        a.lse[place(i)] = sum == 0.f ? -INFINITY : (ref + log2f(sum)) * 0.693147180559945309f;
    __syncthreads();
    if (i0 + warp < s.rows) {
        T *y = static_cast<T *>(a.y) + place(i0 + warp) * D;
        for (int d = lane; d < D; d += 32) st_from_f32(y + d, so[d][warp]);
    }
}

// Tiles of a unit: one where a sequence has no more rows (the second tile's warps
// then help to dequantise).
int tc_tiles(int64_t rows, int64_t D) { return D == 256 || rows <= kTcTile ? 1 : 2; }
// How a call is laid out: units, and in how many parts each is cut.
struct TcPlan {
    int64_t units, workspace;
    int parts, part_rows;
};
TcPlan tc_plan(int64_t B, int64_t rows, int64_t H, int64_t D) {
    const int64_t unit_rows = tc_tiles(rows, D) * kTcTile;
    TcPlan p{B * ((rows + unit_rows - 1) / unit_rows) * H, 0, 1, (int)((std::min(rows, unit_rows) + 7) / 8 * 8)};
    // Units of 1.5 times the SMs on are left whole: cut, they would be dealt out
    // little more evenly (256 over 152 SMs: 112 steps instead of 118), and have to
    // be joined.  (So for lengths that differ by four times or so; whole units take as long
    // as the longest: 64 rows of 15 sequences of 1000 tokens and of one of 131072 1165 us,
    // of 3 and one, which are cut, 224.)  Fewer are cut, into one part an SM in all, or two
    // of two tiles: 256
    // rows of one sequence of 8192 tokens and 8 heads 54 us whole, 23 cut; 32 to 128
    // rows of 16 sequences of up to 8192 tokens 79 us whole, 81 in two parts each and
    // 88 in four.
    if (2 * p.units < 3 * kTcSms) p.parts = (int)std::min<int64_t>(tc_tiles(rows, D) * kTcSms / p.units, 64);
    if (p.parts > 1) p.workspace = p.units * p.parts * (D + 2) * p.part_rows * 4;
    else p.parts = 1;
    return p;
}

template <typename T, int D, int TILES>
cudaError_t launch_tc(const AttendArgs &a, cudaStream_t s) {
    using L = Tc<D, TILES>;
    unsigned *flag = nullptr;
    cudaError_t e = attend_tc_wait_flag(&flag);
    if (e != cudaSuccess) return e;
    const TcPlan p = tc_plan(a.B, a.T * (a.Hq / a.H), a.H, D);
    if (p.units * p.parts > INT32_MAX) return cudaErrorInvalidConfiguration;
    // a part's first step, queries and output cost as much as six steps
    const int64_t steps = ((int64_t)a.width << a.page_shift) / L::kTok;
    const int parts = (int)std::max<int64_t>(std::min<int64_t>(p.parts, steps / 6), 1);
    // whether a part can have more than kTcCarry tokens
    const int64_t most = a.window > 0 ? std::min(steps, (a.window + a.T) / L::kTok + 2) : steps;
    const bool carries = (most + parts - 1) / parts > kTcCarry / L::kTok;
    const auto kernel = carries ? attend_tc_kernel<T, D, TILES, true> : attend_tc_kernel<T, D, TILES, false>;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)L::kSmem);
    if (e != cudaSuccess) return e;
    TcArgs ta{a, parts, p.part_rows, flag, wait_bound_cycles(), inject_wait_expiry()};
    e = launch_dependent(kernel, (unsigned)(p.units * parts), kTcThreads, L::kSmem, s, ta);
    if (e != cudaSuccess || parts == 1) return e;
    const int groups = p.part_rows / 8;
    return launch_dependent(attend_tc_join_kernel<T, D, TILES>, (unsigned)(p.units * groups), 256, 0, s, a, parts, p.part_rows, groups);
}

template <typename T>
cudaError_t launch_attend_tc(const AttendArgs &a, cudaStream_t s) {
    const bool one = tc_tiles(a.T * (a.Hq / a.H), a.D) == 1;
    switch (a.D) {
    case 64: return one ? launch_tc<T, 64, 1>(a, s) : launch_tc<T, 64, 2>(a, s);
    case 128: return one ? launch_tc<T, 128, 1>(a, s) : launch_tc<T, 128, 2>(a, s);
    case 256: return launch_tc<T, 256, 1>(a, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

}  // namespace gdn
