// attend_tc.cu -- attention of many query rows over the 4-bit paged cache
// (prompts), on tcgen05.
//
// A CTA takes one unit: up to 256 query rows (two tiles of 128; one tile for
// heads of 256) of one sequence and key head, and the tokens that they see,
// TN = 128 (64 for heads of 256) at a time.  Roles:
//   dequant warps  codes from global memory, a step ahead in registers, to exact
//                  f16 (code times scale, fp4.cuh) in shared memory: K and V as
//                  panels of 64 channels x TN tokens, 128-byte rows, 128-byte
//                  swizzle.  The same layout is K's K-major operand of S = Q K^T
//                  and V's N-major operand of O += P V.  Two stages.
//   issuer         S of a tile into tensor memory; then, when its probabilities
//                  are there, O += P V with P from tensor memory.  While one
//                  tile's softmax runs, the other tile's products do.
//   softmax warps  thread r owns row r of its tile: S from tensor memory to
//                  registers, 2^(x - reference), P as f16 over S's columns.  Only
//                  where a step's sum says that a probability may be too large
//                  for f16 are the maximum taken and O rescaled, by the row's
//                  thread.
// With one tile S has two buffers instead, and S of the next step is issued
// before O += P V of this one.
//
// Per 128 x 128 x 128 step of a tile: 2 x 512 cycles of products, 16384
// exponentials and 64 KB through shared memory by the products (512 + 256
// cycles), 32 KB of operands written (256 cycles, no bank conflicts).
//
// Operands and softmax are those of kv_attend.cuh; sums stay in tensor memory
// in float32.  Every wait is bounded; when one runs out, the unit's rows are
// written as NaN and the library's wait flag is raised.
#include <algorithm>
#include <cfloat>
#include <type_traits>

#include "attend.h"
#include "fp4.cuh"
#include "pieces.cuh"
#include "tma.cuh"

namespace gdn {

namespace {

__device__ unsigned g_attend_tc_wait_flag;

constexpr int kTcThreads = 512;   // warpgroups: softmax, softmax (or dequant), dequant, issuer (a warp of it) and dequant
constexpr int kTcTile = 128;                              // query rows of a tile
constexpr uint32_t kTmemCols = 512, kTmemO = 256;         // S buffers at 0 and 128, O from 256 on
constexpr long long kDrainCycles = 2000000000ll;
// A row's largest probability when its reference is set, at least (the wider the
// scores spread, the lower, by kTcRoom at most), and what a step's may add up to.
// f16 steps end at 2^-24: weights are off by 2^-12 of themselves, or by 2^-22 of
// the row's largest (2^-16 if the scores spread over 24 bits or more).
constexpr float kTcLow = 3.f, kTcRoom = 6.f, kTcMost = 32768.f;

template <int D> struct Tc {
    static constexpr int kTiles = D == 256 ? 1 : 2;
    static constexpr int kRows = kTiles * kTcTile;
    static constexpr int kTok = D == 256 ? 64 : 128;       // tokens per step
    // Dequantisation, in units of 32/(D/32) tokens of K or V: the warps of whole
    // warpgroups take kKUnits and kVUnits of them each; the three warps beside the
    // issuer kXUnits of V, behind those.
    static constexpr int kDqWarps = D == 256 ? 8 : 4;
    static constexpr int kUnitTok = 1024 / D, kUnits = kTok / kUnitTok;
    static constexpr int kKUnits = kUnits / kDqWarps, kVUnits = D == 256 ? 2 : D == 128 ? 1 : 0;
    static constexpr int kXUnits = (kUnits - kDqWarps * kVUnits + 2) / 3;
    static constexpr int kVWarps = (kVUnits > 0 ? kDqWarps : 0) + (kXUnits > 0 ? 3 : 0);
    static constexpr int kSoftmaxRegs = 168, kDqRegs = 88;  // 128 threads of each: 2 and 2, or 1 and 3
    static constexpr uint32_t kQBytes = kRows * D * 2, kOpBytes = kTok * D * 2;  // K or V of a step
    static constexpr uint32_t kQ = 0, kK = kQBytes, kV = kK + 2 * kOpBytes, kBars = kV + 2 * kOpBytes;
    static constexpr size_t kSmem = kBars + 256 + 1024;    // (1024: alignment)
};
// Barriers: of a stage of K or V (written, free), of an S buffer (S there, part 0
// and part 1 of P there), of a tile (O with part 0, O of the step).
enum Bar {
    kKFull = 0, kVFull = 2, kKFree = 4, kVFree = 6, kSFull = 8, kPFull = 10, kOPart = 14, kODone = 16, kDrain = 18,
    kNever = 19, kBarCount = 20
};

__device__ __forceinline__ uint64_t operand_desc(uint32_t addr, uint32_t lbo, uint32_t sbo) {  // 128-byte swizzle
    return (uint64_t)((addr >> 4) & 0x3fffu) | ((uint64_t)((lbo >> 4) & 0x3fffu) << 16) |
           ((uint64_t)((sbo >> 4) & 0x3fffu) << 32) | (1ull << 46) | (2ull << 61);
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
__device__ __forceinline__ void mma_ss(uint32_t one, uint32_t d, uint64_t a, uint64_t b, uint32_t op, uint32_t add) {
    asm volatile("{\n.reg .pred p, q;\nsetp.ne.b32 p, %4, 0;\nsetp.ne.b32 q, %5, 0;\n"
                 "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
                 "l"(a), "l"(b), "r"(op), "r"(add), "r"(one)
                 : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t one, uint32_t d, uint32_t a, uint64_t b, uint32_t op, uint32_t add) {
    asm volatile("{\n.reg .pred p, q;\nsetp.ne.b32 p, %4, 0;\nsetp.ne.b32 q, %5, 0;\n"
                 "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
                 "r"(a), "l"(b), "r"(op), "r"(add), "r"(one)
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
__device__ __forceinline__ void tm_st16(uint32_t t, const uint32_t *r) {
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

template <int N> __device__ __forceinline__ void more_registers() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(N));
}
template <int N> __device__ __forceinline__ void less_registers() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(N));
}

struct TcArgs {
    AttendArgs a;
    int row_blocks;
    unsigned *wait_flag;
    long long wait_cycles;
    int inject_expiry;
};

template <typename T, int D>
__global__ void __launch_bounds__(kTcThreads, 1) attend_tc_kernel(const TcArgs ta) {
    using L = Tc<D>;
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
            mbar_init(bar(i), i < kVFull ? L::kDqWarps : i < kKFree ? L::kVWarps : i >= kPFull && i < kOPart ? 4 : 1);
        mbar_init_fence();
    }
    tm_before();
    __syncthreads();
    tm_after();
    const uint32_t tmem = *tmem_slot;
    pdl_trigger();
    pdl_wait();

    // ------------------------------------------------ the unit
    const int G = a.Hq / a.H, page = 1 << a.page_shift;
    // later row blocks see more tokens: those first
    const int u = (int)(gridDim.x - 1 - blockIdx.x), h = u % a.H, b = u / a.H % (int)a.B, rb = u / a.H / (int)a.B;
    const int n = a.fresh ? min(max(a.fresh[b], 0), (int)a.T) : (int)a.T;
    const int len = (int)min((int64_t)max(a.lengths[b], 0), (int64_t)a.width << a.page_shift);
    const int r0 = rb * L::kRows, rows = min(max(n * G - r0, 0), L::kRows);
    const int tiles = rows > kTcTile ? 2 : 1;
    // the tokens that any row sees, and steps over them
    const int first_pos = len - n + r0 / G, last_pos = len - n + (r0 + max(rows, 1) - 1) / G;
    const int hi = max(last_pos + 1, 0), lo = a.window > 0 ? max(first_pos - a.window + 1, 0) : 0;
    const int step0 = lo / TN, steps = rows == 0 ? 0 : max((hi + TN - 1) / TN - step0, 0);
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
        if (ok) ok = __all_sync(0xffffffffu, mbar_wait_bounded(bar(i), parity & 1u, ta.wait_cycles));
        return ok;
    };
    if (ta.inject_expiry) wait(kNever, 0);

    const bool softmax_warp = warp < 4 * L::kTiles;
    float sum = 0.f, off = -1e30f;
    // registers where they are used: 4 x 128 at launch, as many or fewer in all
    if (softmax_warp) {
        more_registers<L::kSoftmaxRegs>();
        // ================================================ softmax warps
        const int t = warp >> 2, row = tid & 127, r = r0 + t * kTcTile + row;  // tile, row in it, row of the sequence
        const bool there = t * kTcTile + row < rows;
        const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);  // this warp's 32 lanes
        const int qt = r / G, pos = len - n + qt;
        float c = FLT_MIN;
        if (t < tiles && steps > 0) {
            // the row to f16, scaled by a power of two, with the scale's sign
            const T *q = static_cast<const T *>(a.q) + b * a.q_sb + qt * a.q_st + (int64_t)(h * G + r - qt * G) * D;
            RawPiece<T, 8> raw[D / 8];  // all of the row in flight at once
            if (there && a.vec_q) {
#pragma unroll
                for (int i = 0; i < D / 8; ++i) raw[i] = load_raw<T, 8>(q + 8 * i);
            } else {
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    uint32_t w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint16_t *at = reinterpret_cast<const uint16_t *>(q) + 8 * i + 2 * e;
                        w[e] = there ? at[0] | (uint32_t)at[1] << 16 : 0u;
                    }
                    raw[i].w = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
            float top = 0.f;
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                float v[8];
                widen<T, 8>(v, raw[i]);
#pragma unroll
                for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(v[e]));
            }
            const int e2 = top < INFINITY ? max((int)(__float_as_uint(top) >> 23) - 127, -100) : 10;
            const float up = copysignf(__uint_as_float((uint32_t)(127 + 10 - e2) << 23), a.scale);
            const float ks = a.k_scale ? a.k_scale[h] : 1.f;
            c = fmaxf(fabsf(a.scale) * 1.44269504088896341f * ks * __uint_as_float((uint32_t)(127 + e2 - 10) << 23), FLT_MIN);
            const uint32_t sq = base + L::kQ + t * kTcTile * 128 + row * 128;  // panels of 64 channels x kRows rows
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                float v[8];
                widen<T, 8>(v, raw[i]);
                st_shared16(sq + (i >> 3) * (L::kRows * 128) + (((i & 7) ^ (row & 7)) << 4), pack2<__half>(v[0] * up, v[1] * up),
                            pack2<__half>(v[2] * up, v[3] * up), pack2<__half>(v[4] * up, v[5] * up),
                            pack2<__half>(v[6] * up, v[7] * up));
            }
        }
        asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
        named_bar_sync(1, 32 * (4 * L::kTiles + 1));  // with the issuer: the queries are there

        // visible tokens of the row: [row_lo, row_hi)
        const int row_hi = min(pos + 1, hi), row_lo = a.window > 0 ? max(pos - a.window + 1, 0) : 0;
        // tokens that every row of the tile sees
        const int tr0 = r0 + t * kTcTile, tr1 = r0 + min(rows, (t + 1) * kTcTile) - 1;
        const int all_hi = len - n + tr0 / G + 1, all_lo = a.window > 0 ? max(len - n + tr1 / G - a.window + 1, 0) : 0;
        constexpr int PN = 64, PARTS = TN / PN;  // P is handed over in parts
        int ids = t < tiles ? pages_of(0) : -1;
        for (int j = 0; j < steps && t < tiles; ++j) {
            const int buf = tiles == 2 ? t : j & 1;
            const uint32_t s_at = lanes + 128u * (uint32_t)buf;
            const unsigned present = __ballot_sync(0xffffffffu, (uint32_t)ids < pool);  // bit i: tokens 16 i on
            ids = pages_of(j + 1);
            if (!wait(kSFull + buf, tiles == 2 ? j : j >> 1)) break;
            tm_after();
            const int tok0 = (step0 + j) * TN;
            const bool edge = tok0 < all_lo || tok0 + TN > all_hi || present != (1u << (TN / 16)) - 1u;
            const int c_lo = row_lo - tok0, c_hi = row_hi - tok0;
            // columns [64 part, 64 part + PN) of S
            auto scores = [&](int part, float (&v)[PN]) {
#pragma unroll
                for (int k = 0; k < PN / 32; ++k) tm_ld32(s_at + (uint32_t)(PN * part + 32 * k), v + 32 * k);
            };
            auto mask = [&](int part, float (&v)[PN]) {
                if (edge) {
#pragma unroll
                    for (int i = 0; i < PN; ++i) {
                        const int e = PN * part + i;
                        if (e < c_lo || e >= c_hi || !((present >> (e / 16)) & 1u)) v[i] = -INFINITY;
                    }
                }
            };
            // the probabilities to f16, and their sum
            uint32_t p[PN / 2];
            auto powers = [&](const float (&v)[PN]) {
                const float2 c2 = make_float2(c, c), off2 = make_float2(-off, -off);
                float2 part[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                for (int e = 0; e < PN / 2; ++e) {
                    const float2 x = ffma2(make_float2(v[2 * e], v[2 * e + 1]), c2, off2);
                    const float2 y = make_float2(ex2f(x.x), ex2f(x.y));
                    part[e & 1] = __fadd2_rn(part[e & 1], y);
                    p[e] = pack2<__half>(y.x, y.y);
                }
                part[0] = __fadd2_rn(part[0], part[1]);
                return part[0].x + part[0].y;
            };
            float v[PARTS][PN];
#pragma unroll
            for (int part = 0; part < PARTS; ++part) scores(part, v[part]);
            tm_wait_ld();
#pragma unroll
            for (int part = 0; part < PARTS; ++part) {
                mask(part, v[part]);
                float now = powers(v[part]);
                // A sum below 2^15 has no term above it: every one fits f16, and no maximum
                // was needed.  Else (the first step, and when the scores rise) the reference
                // moves to the maximum, and sum and O with it; and above it, the more the
                // wider the scores spread: then later ones rise higher, and small
                // probabilities matter less.
                if (__any_sync(0xffffffffu, now > kTcMost)) {
                    float w[PN], top = -INFINITY, all = 0.f;
                    scores(part, w);
                    tm_wait_ld();
                    mask(part, w);
                    int count = 0;
#pragma unroll
                    for (int e = 0; e < PN; ++e) {
                        top = fmaxf(top, w[e]);
                        all += w[e] == -INFINITY ? 0.f : w[e];
                        count += w[e] == -INFINITY ? 0 : 1;
                    }
                    const float spread = count > 0 ? fminf(0.25f * c * (top - all / (float)count), kTcRoom) : 0.f;
                    const float to = top == -INFINITY ? off : fmaxf(off, top * c + kTcLow + fmaxf(spread, 0.f));
                    const float f = exp2f(off - to);
                    off = to;
                    sum *= f;
                    now = powers(w);
                    if (j > 0 || part > 0) {
                        if (!(part > 0 ? wait(kOPart + t, j) : wait(kODone + t, j - 1))) break;
                        tm_after();
#pragma unroll 1
                        for (int k = 0; k < D / 32; ++k) {
                            float o[32];
                            const uint32_t o_at = lanes + kTmemO + (uint32_t)(t * D + 32 * k);
                            tm_ld32(o_at, o);
                            tm_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] *= f;
                            tm_st32(o_at, o);
                        }
                    }
                }
                sum += now;
                // (over columns of S that are in registers, all of them)
#pragma unroll
                for (int k = 0; k < PN / 32; ++k) tm_st16(s_at + (uint32_t)(PN / 2 * part + 16 * k), p + 16 * k);
                tm_wait_st();
                tm_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(kPFull + 2 * part + buf));
            }
            if (!ok) break;
        }

        // ------------------------------------------------ the row's output
        if (t < tiles) {
            if (steps > 0) wait(kODone + t, steps - 1);
            tm_after();
            const float vs = a.v_scale ? a.v_scale[h] : 1.f;
            const float inv = !ok ? __int_as_float(0x7fc00000) : sum == 0.f ? 0.f : vs / sum;
            const int64_t at = ((int64_t)b * a.T + qt) * a.Hq + h * G + r - qt * G;
            T *y = static_cast<T *>(a.y) + at * D;
#pragma unroll 1
            for (int k = 0; k < D / 32; ++k) {
                float v[32];
                if (steps > 0 && ok) {
                    tm_ld32(lanes + kTmemO + (uint32_t)(t * D + 32 * k), v);
                    tm_wait_ld();
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] = 0.f;
                }
                if (there && a.vec_y) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float w[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) w[e] = v[8 * i + e] * inv;
                        store_piece<T, 8>(y + 32 * k + 8 * i, w);
                    }
                } else if (there) {
#pragma unroll
                    for (int e = 0; e < 32; ++e) st_from_f32(y + 32 * k + e, v[e] * inv);
                }
                __syncwarp();
            }
            if (there && a.lse)
                a.lse[at] = !ok ? inv : sum == 0.f ? -INFINITY : (off + log2f(sum)) * 0.693147180559945309f;
        }
    } else if (warp != 12) {
        less_registers<L::kDqRegs>();
        // ================================================ dequant warps
        // A lane's part of a unit is 32 neighbouring channels of a token: 16 bytes of
        // codes, two scales.  D/32 lanes share a token; a unit's tokens are in a page.
        constexpr int LPR = D / 32, UT = L::kUnitTok;
        const bool extra = warp > 12;
        const int w = extra ? warp - 13 : warp - 4 * L::kTiles, piece = lane % LPR, sub = lane / LPR, panel = piece >> 1;
        // the order of the four words, so that eight lanes write distinct banks
        const int order = D == 256 ? panel : D == 128 ? 2 * panel : 0;
        const uint32_t page_bytes = (uint32_t)(a.H * kv_block_bytes(page, D));
        const unsigned char *cache = a.cache + h * kv_block_bytes(page, D) + 16 * piece;
        const unsigned char *scales = a.cache + h * kv_block_bytes(page, D) + page * (D / 2) + 2 * piece;
        const int values = page * (D / 2 + D / 16);
        const uint32_t pick[2] = {order & 2 ? 0x3232u : 0x1010u, order & 2 ? 0x1010u : 0x3232u};
        uint32_t chunk[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            chunk[k] = (uint32_t)panel * (TN * 128) + sub * 128 + ((((piece & 1) * 4 + (k ^ order)) ^ (sub & 7)) << 4);
        auto load = [&](int j, int ids, int at, int unit, uint2 (&q)[2], uint32_t &sc) {
            const int t0 = (step0 + j) * TN, in = unit * UT + sub, tok = t0 + in, row = tok & (page - 1);
            const int id = __shfl_sync(0xffffffffu, ids, (unit * UT) >> 4);
            q[0] = q[1] = make_uint2(0, 0);
            sc = 0;
            if ((uint32_t)id < pool && tok >= lo && tok < hi) {
                const uint64_t off = (uint64_t)(uint32_t)id * page_bytes + (uint32_t)at;
                const unsigned char *c = cache + off + row * (D / 2);
                // (the halves in the order that they are written in)
                q[0] = *reinterpret_cast<const uint2 *>(c + 4 * (order & 2));
                q[1] = *reinterpret_cast<const uint2 *>(c + 8 - 4 * (order & 2));
                sc = *reinterpret_cast<const uint16_t *>(scales + off + row * (D / 16));
            }
        };
        auto store = [&](uint32_t dst, int unit, const uint2 (&q)[2], uint32_t sc) {
            const uint32_t both = e4m3x2_to_f16(sc), at = dst + unit * UT * 128;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                uint32_t x = k % 2 ? q[k / 2].y : q[k / 2].x;
                if (D == 256 && (order & 1)) x = k % 2 ? q[k / 2].x : q[k / 2].y;
                const uint32_t f = __byte_perm(both, both, pick[k / 2]);
                uint32_t e[4];
                e2m1x8_to_f16(x, e);
                // (units of four tokens: the odd ones' rows are 4 to 7 of the swizzle's eight)
                st_shared16(at + (UT == 4 ? chunk[k] ^ ((unit & 1) << 6) : chunk[k]), times2(e[0], f), times2(e[1], f),
                            times2(e[2], f), times2(e[3], f));
            }
        };
        auto stored = [&](int i) {
            asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(i));
        };
        // NK units of K from k0 on and NV of V from v0 on, a step ahead in registers
        auto run = [&](auto nk, auto nv, int k0, int v0) {
            constexpr int NK = decltype(nk)::value, NV = decltype(nv)::value;
            uint2 kq[NK > 0 ? NK : 1][2], vq[NV > 0 ? NV : 1][2];
            uint32_t ks[NK > 0 ? NK : 1], vs[NV > 0 ? NV : 1];
            int ids = pages_of(0), ids_next = pages_of(1);
            auto load_k = [&](int j) {
#pragma unroll
                for (int i = 0; i < NK; ++i) load(j, ids, 0, k0 + i, kq[i], ks[i]);
            };
            auto load_v = [&](int j) {
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    if (v0 + i < L::kUnits) load(j, ids, values, v0 + i, vq[i], vs[i]);
            };
            load_k(0);
            load_v(0);
            for (int j = 0; j < steps; ++j) {
                const int st = j & 1;
                ids = ids_next;
                ids_next = pages_of(j + 2);
                if (NK > 0) {
                    if (j >= 2 && !wait(kKFree + st, (j >> 1) - 1)) break;
#pragma unroll
                    for (int i = 0; i < NK; ++i) store(base + L::kK + st * L::kOpBytes, k0 + i, kq[i], ks[i]);
                    stored(kKFull + st);
                }
                if (NV > 0) {
                    if (j >= 2 && !wait(kVFree + st, (j >> 1) - 1)) break;
#pragma unroll
                    for (int i = 0; i < NV; ++i)
                        if (v0 + i < L::kUnits) store(base + L::kV + st * L::kOpBytes, v0 + i, vq[i], vs[i]);
                    stored(kVFull + st);
                }
                // (a fence waits for loads in flight: so none before the step's last one)
                load_k(j + 1);
                load_v(j + 1);
            }
        };
        if (!extra)
            run(std::integral_constant<int, L::kKUnits>(), std::integral_constant<int, L::kVUnits>(), w * L::kKUnits,
                w * L::kVUnits);
        else if (L::kXUnits > 0)
            run(std::integral_constant<int, 0>(), std::integral_constant<int, L::kXUnits>(), 0,
                L::kDqWarps * L::kVUnits + w * L::kXUnits);
    } else {
        less_registers<L::kDqRegs>();
        // ================================================ issuer
        {
            named_bar_sync(1, 32 * (4 * L::kTiles + 1));
            constexpr uint32_t op_s = op_desc(TN, false), op_o = op_desc(D, true);
            const uint32_t one = elect_one(), tm = __shfl_sync(0xffffffffu, tmem, 0);
            const uint32_t sbase = __shfl_sync(0xffffffffu, base, 0);
            auto issue_s = [&](int j, int t) {
                const int buf = tiles == 2 ? t : j & 1;
                if (t == 0 && !wait(kKFull + (j & 1), j >> 1)) return;
                tm_after();
                const uint64_t q = operand_desc(sbase + L::kQ + t * kTcTile * 128, 16, 1024);
                const uint64_t k = operand_desc(sbase + L::kK + (j & 1) * L::kOpBytes, 16, 1024);
#pragma unroll
                for (int s = 0; s < D / 16; ++s)
                    mma_ss(one, tm + 128u * buf, q + ((s >> 2) * (L::kRows * 128) + (s & 3) * 32) / 16,
                           k + ((s >> 2) * (TN * 128) + (s & 3) * 32) / 16, op_s, s > 0);
                commit_to(one, bar(kSFull + buf));
                if (t == tiles - 1) commit_to(one, bar(kKFree + (j & 1)));
            };
            auto issue_o = [&](int j, int t) {
                const int buf = tiles == 2 ? t : j & 1;
                if (t == 0 && !wait(kVFull + (j & 1), j >> 1)) return;
                const uint64_t v = operand_desc(sbase + L::kV + (j & 1) * L::kOpBytes, TN * 128, 1024);
#pragma unroll
                for (int part = 0; part < TN / 64; ++part) {
                    if (!wait(kPFull + 2 * part + buf, tiles == 2 ? j : j >> 1)) return;
                    tm_after();
#pragma unroll
                    for (int s = 4 * part; s < 4 * part + 4; ++s)
                        mma_ts(one, tm + kTmemO + (uint32_t)(t * D), tm + 128u * buf + 8u * s, v + s * 2048 / 16, op_o, j > 0 || s > 0);
                    if (part < TN / 64 - 1) commit_to(one, bar(kOPart + t));
                }
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

template <typename T, int D>
cudaError_t launch_tc(const AttendArgs &a, cudaStream_t s) {
    using L = Tc<D>;
    void *flag = nullptr;
    cudaError_t e = cudaGetSymbolAddress(&flag, g_attend_tc_wait_flag);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(attend_tc_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)L::kSmem);
    if (e != cudaSuccess) return e;
    const int64_t rb = (a.T * (a.Hq / a.H) + L::kRows - 1) / L::kRows, units = a.B * rb * a.H;
    if (units > INT32_MAX) return cudaErrorInvalidConfiguration;
    TcArgs ta{a, (int)rb, static_cast<unsigned *>(flag), wait_bound_cycles(), inject_wait_expiry()};
    return launch_dependent(attend_tc_kernel<T, D>, (unsigned)units, kTcThreads, L::kSmem, s, ta);
}

template <typename T>
cudaError_t launch_t(const AttendArgs &a, cudaStream_t s) {
    switch (a.D) {
    case 64: return launch_tc<T, 64>(a, s);
    case 128: return launch_tc<T, 128>(a, s);
    case 256: return launch_tc<T, 256>(a, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

bool attend_takes_tc(DType dt, const AttendArgs &a) {
    return dt != DType::F32 && a.T * (a.Hq / a.H) >= 64;
}

cudaError_t launch_attend_tc(DType dt, const AttendArgs &a, cudaStream_t s) {
    return dt == DType::BF16 ? launch_t<__nv_bfloat16>(a, s) : launch_t<__half>(a, s);
}

cudaError_t attend_tc_take_wait_flag(unsigned *was_set) {
    unsigned v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_attend_tc_wait_flag, sizeof v);
    if (e != cudaSuccess) return e;
    *was_set = v;
    if (v) {
        const unsigned zero = 0;
        e = cudaMemcpyToSymbol(g_attend_tc_wait_flag, &zero, sizeof zero);
    }
    return e;
}

}  // namespace gdn
