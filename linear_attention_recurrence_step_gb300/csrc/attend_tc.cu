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
// A row's largest probability when its reference is set is 2^6, or, the wider the
// scores spread, down to 2^0; a step's may add up to 2^15.  f16 steps end at
// 2^-24: weights are off by 2^-12 of themselves, or by 2^-31 of the row's largest
// (2^-25 if the scores spread over 24 bits or more).
constexpr float kTcBoost = 6.f, kTcRoom = 6.f, kTcMost = 32768.f;
constexpr int kTcMaxPairs = 512;   // (sequence, row block) pairs of a call that is cut along its tokens
constexpr int kTcParts = 152;      // blocks of such a call: one per SM
constexpr int kTcAhead = 4;

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
    static constexpr int kSoftmaxRegs = 152, kDqRegs = 104;  // 128 threads of each: 2 and 2, or 1 and 3
    static constexpr uint32_t kQBytes = kRows * D * 2, kOpBytes = kTok * D * 2;  // K or V of a step
    static constexpr uint32_t kQ = 0, kK = kQBytes, kV = kK + 2 * kOpBytes, kBars = kV + 2 * kOpBytes;
    static constexpr uint32_t kLine = kBars + 256;         // where the pairs begin in the line
    static constexpr size_t kSmem = kLine + 4 * (kTcMaxPairs + 8) + 1024;  // (1024: alignment)
    // the workspace: a note per block on the unit that it cuts, then two partial
    // results per block (O, the reference and the sum of each row)
    static constexpr int kNoteFloats = 4 * kTcParts, kPartFloats = kRows * (D + 2);
    static constexpr int64_t kWorkspace = 4 * ((int64_t)kNoteFloats + 2ll * kTcParts * kPartFloats);
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
    int pairs, row_blocks;
    unsigned *wait_flag;
    long long wait_cycles;
    int inject_expiry;
    bool whole;             // a block takes one whole unit
};

// A (sequence, row block) pair: the tokens [lo, hi) that any of its rows sees,
// and the steps over them.
struct TcSpan {
    int b, r0, rows, n, len, lo, hi, step0, steps;
};
template <int D> __device__ __forceinline__ TcSpan tc_span(const AttendArgs &a, int p, int row_blocks) {
    using L = Tc<D>;
    TcSpan s;
    s.b = p / row_blocks;
    const int G = a.Hq / a.H;
    s.n = a.fresh ? min(max(a.fresh[s.b], 0), (int)a.T) : (int)a.T;
    s.len = (int)min((int64_t)max(a.lengths[s.b], 0), (int64_t)a.width << a.page_shift);
    s.r0 = (p - s.b * row_blocks) * L::kRows;
    s.rows = min(max(s.n * G - s.r0, 0), L::kRows);
    const int first = s.len - s.n + s.r0 / G, last = s.len - s.n + (s.r0 + max(s.rows, 1) - 1) / G;
    s.hi = max(last + 1, 0);
    s.lo = a.window > 0 ? max(first - a.window + 1, 0) : 0;
    s.step0 = s.lo / L::kTok;
    // (rows that see nothing are written too)
    s.steps = s.rows == 0 ? 0 : max((s.hi + L::kTok - 1) / L::kTok - s.step0, 1);
    return s;
}
// All units stand on a line: kTcAhead places for what a unit costs beside its
// steps (queries, the first step, its output: some 12000 cycles, a step 3000),
// then its steps; W places in all, fewer than 2^31.  It is cut in kTcParts parts, or
// in places if there are fewer: where block c's begins, and the block of place x.  (The quotients are below 153 and no nearer to the next integer than
// 2^-31: doubles give them exactly.)
__device__ __forceinline__ int tc_begin(int c, int W) {
    return W < kTcParts ? min(c, W) : (int)((uint64_t)(uint32_t)c * (uint32_t)W / kTcParts);
}
__device__ __forceinline__ int tc_part_of(int x, int W) {
    return W < kTcParts ? x : (int)((((double)x + 1) * kTcParts - 1) / (double)W);
}

template <typename T, int D>
__global__ void __launch_bounds__(kTcThreads, 1) attend_tc_kernel(const TcArgs ta) {
    using L = Tc<D>;
    constexpr int TN = L::kTok;
    const AttendArgs &a = ta.a;
    extern __shared__ unsigned char smem_raw[];
    const uint32_t base = (sh_addr(smem_raw) + 1023u) & ~1023u;
    unsigned char *const gbase = smem_raw + (base - sh_addr(smem_raw));
    auto bar = [&](int i) { return base + L::kBars + 8u * (uint32_t)i; };
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(gbase + L::kBars + 8 * kBarCount);
    int *line = reinterpret_cast<int *>(gbase + L::kLine);
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

    // ------------------------------------------------ this block's part of the line
    const int G = a.Hq / a.H, page = 1 << a.page_shift;
    int begin = 0, end = 1;
    auto places = [](int steps) { return steps > 0 ? steps + kTcAhead : 0; };
    if (!ta.whole) {
        for (int p = tid; p <= ta.pairs; p += kTcThreads) line[p] = p < ta.pairs ? places(tc_span<D>(a, p, ta.row_blocks).steps) * a.H : 0;
        __syncthreads();
        if (warp == 0) {  // to sums of those before
            int carry = 0;
            for (int p0 = 0; p0 <= ta.pairs; p0 += 32) {
                const int mine = p0 + lane <= ta.pairs ? line[p0 + lane] : 0;
                int v = mine;
#pragma unroll
                for (int d = 1; d < 32; d *= 2) {
                    const int o = __shfl_up_sync(0xffffffffu, v, d);
                    if (lane >= d) v += o;
                }
                if (p0 + lane <= ta.pairs) line[p0 + lane] = carry + v - mine;
                carry += __shfl_sync(0xffffffffu, v, 31);
            }
        }
        __syncthreads();
        begin = tc_begin((int)blockIdx.x, line[ta.pairs]);
        end = tc_begin((int)blockIdx.x + 1, line[ta.pairs]);
    }
    // the pair, head and first step of the line's place x (below 0: ahead of the steps)
    auto find = [&](int x, int &p, int &h, int &j0) {
        if (ta.whole) {  // (later row blocks see more tokens: those first)
            const int u = (int)(gridDim.x - 1 - blockIdx.x), q = u / a.H, nb = ta.pairs / ta.row_blocks;
            h = u - q * a.H;
            p = q % nb * ta.row_blocks + q / nb;
            j0 = 0;
            return tc_span<D>(a, p, ta.row_blocks);
        }
        int lo = 0, hi = ta.pairs;
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (line[mid] <= x) lo = mid;
            else hi = mid;
        }
        p = lo;
        const TcSpan s = tc_span<D>(a, p, ta.row_blocks);
        const uint32_t off = (uint32_t)(x - line[p]), n = (uint32_t)places(s.steps);
        h = (int)(off / n);
        j0 = (int)(off - (uint32_t)h * n) - kTcAhead;
        return s;
    };
    if (!ta.whole && tid == 0) {
        // where a unit is cut first, a note for the kernel that joins its parts
        int4 note = make_int4(-1, 0, 0, 0);
        if (begin < end) {
            int p, h, j0;
            const TcSpan s = find(begin, p, h, j0);
            const int W = line[ta.pairs], x0 = begin - j0, c0 = tc_part_of(x0, W);  // (x0: its first step)
            if (j0 > 0 && c0 == (int)blockIdx.x - 1)
                note = make_int4(p, h, 2 * c0 + (tc_begin(c0, W) < x0 - kTcAhead ? 1 : 0), tc_part_of(x0 + s.steps - 1, W));
        }
        reinterpret_cast<int4 *>(a.workspace)[blockIdx.x] = note;
    }
    const uint32_t pool = (uint32_t)a.pages;
    bool ok = true;
    // by a whole warp: all of it goes on, or none
    auto wait = [&](int i, uint32_t parity) {
        if (ok) ok = __all_sync(0xffffffffu, mbar_wait_bounded(bar(i), parity & 1u, ta.wait_cycles));
        return ok;
    };
    if (ta.inject_expiry) wait(kNever, 0);

    // A part of a unit: steps [j0, j0 + steps) of it (none, if this block's part of
    // the line ends ahead of its first); `next`: where the next one begins.
    struct Segment {
        TcSpan s;
        int h, j0, steps, tiles, next;
    };
    auto segment = [&](int at) {
        Segment g;
        int p;
        g.s = find(at, p, g.h, g.j0);
        const int ahead = max(-g.j0, 0);
        g.j0 = max(g.j0, 0);
        g.steps = ta.whole ? g.s.steps : max(min(g.s.steps - g.j0, end - at - ahead), 0);
        g.next = ta.whole ? 1 : at + ahead + g.steps;
        g.tiles = g.s.rows > kTcTile ? 2 : 1;
        return g;
    };
    // How often each S buffer, and each tile's O, was used up to a segment: their
    // barriers' phases.  (One tile uses both S buffers in turn.)
    struct Uses {
        int step = 0, s0 = 0, s1 = 0, o1 = 0;  // (tile 0's O: at every step)
        __device__ int s(int buf) const { return buf ? s1 : s0; }
        __device__ int o(int t) const { return t ? o1 : step; }
    };
    auto after = [](Uses &u, const Segment &g) {
        u.step += g.steps;
        u.s0 += g.tiles == 2 ? g.steps : (g.steps + 1) / 2;
        u.s1 += g.tiles == 2 ? g.steps : g.steps / 2;
        u.o1 += g.tiles == 2 ? g.steps : 0;
    };
    // A segment's tokens, from its first step's on.
    struct Tokens {
        const int32_t *table;   // the sequence's row
        int tok0, lo, hi, steps;
    };
    auto tokens = [&](const Segment &g) {
        return Tokens{a.table + (int64_t)g.s.b * a.width, (g.s.step0 + g.j0) * TN, g.s.lo, g.s.hi, g.steps};
    };
    // the table's entry for the 16 tokens `lane` (of TN) of step j of a segment, -1:
    // none of them is seen.  (Whether it names a page is asked where it is used, a
    // step later: here the warp would wait for it.)
    auto pages_of = [&](const Tokens &k, int j) {
        const int tok = k.tok0 + j * TN + 16 * lane;
        int id = -1;
        if (j < k.steps && lane < TN / 16 && tok < k.hi && tok + 16 > k.lo) id = k.table[tok >> a.page_shift];
        return id;
    };
    Uses use;

    const bool softmax_warp = warp < 4 * L::kTiles;
    // registers where they are used: 4 x 128 at launch, as many or fewer in all
    if (softmax_warp) {
        more_registers<L::kSoftmaxRegs>();
        // ================================================ softmax warps
        const int t = warp >> 2, row = tid & 127;                    // tile, row in it
        const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);  // this warp's 32 lanes
        constexpr int PARTS = TN / 64;                               // P is handed over in parts
        bool first = true;
        for (int at = begin; at < end;) {
            float sum = 0.f, off = -1e30f, c = FLT_MIN;
            // what the steps need; the rest of the segment is found again at its end,
            // for the registers that it would hold
            Tokens k;
            int tiles, row_lo, row_hi, all_lo, all_hi;  // tokens that the row sees, and that every row of the tile does
            bool on;
            {
            const Segment g = segment(at);
            if (g.steps == 0) break;
            on = t < g.tiles;
            const int pos = g.s.len - g.s.n + (g.s.r0 + t * kTcTile + row) / G;
            k = tokens(g);
            tiles = g.tiles;
            row_hi = min(pos + 1, g.s.hi) - k.tok0;
            row_lo = (a.window > 0 ? max(pos - a.window + 1, 0) : 0) - k.tok0;
            const int tr0 = g.s.r0 + t * kTcTile, tr1 = g.s.r0 + min(g.s.rows, (t + 1) * kTcTile) - 1;
            all_hi = g.s.len - g.s.n + tr0 / G + 1 - k.tok0;
            all_lo = (a.window > 0 ? max(g.s.len - g.s.n + tr1 / G - a.window + 1, 0) : 0) - k.tok0;
            if (on) {
                // the warp's 32 rows to f16, each scaled by a power of two, with the scale's
                // sign; D/8 lanes take a row, eight channels each, four rows in flight
                constexpr int LR = D / 8, RI = 32 / LR;
                const int piece = lane % LR, base_row = t * kTcTile + (row & ~31);
                const T *const q = static_cast<const T *>(a.q) + g.s.b * a.q_sb + 8 * piece;
                auto load = [&](int i, RawPiece<T, 8> &raw) {
                    const int at_row = base_row + i * RI + lane / LR, r = g.s.r0 + at_row, qt = r / G;
                    const T *from = q + qt * a.q_st + (int64_t)(g.h * G + r - qt * G) * D;
                    raw.w = make_uint4(0, 0, 0, 0);
                    if (at_row < g.s.rows) {
                        if (a.vec_q) {
                            raw = load_raw<T, 8>(from);
                        } else {
                            const uint16_t *e = reinterpret_cast<const uint16_t *>(from);
                            raw.w = make_uint4(e[0] | (uint32_t)e[1] << 16, e[2] | (uint32_t)e[3] << 16,
                                               e[4] | (uint32_t)e[5] << 16, e[6] | (uint32_t)e[7] << 16);
                        }
                    }
                };
                const float factor = fabsf(a.scale) * 1.44269504088896341f * (a.k_scale ? a.k_scale[g.h] : 1.f);
                constexpr int AT_ONCE = 4;
#pragma unroll 1
                for (int i0 = 0; i0 < LR; i0 += AT_ONCE) {
                    RawPiece<T, 8> raw[AT_ONCE];
#pragma unroll
                    for (int i = 0; i < AT_ONCE; ++i) load(i0 + i, raw[i]);
#pragma unroll
                    for (int i = 0; i < AT_ONCE; ++i) {
                        float v[8], top = 0.f;
                        widen<T, 8>(v, raw[i]);
#pragma unroll
                        for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(v[e]));
#pragma unroll
                        for (int d = 1; d < LR; d *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                        const int e2 = top < INFINITY ? max((int)(__float_as_uint(top) >> 23) - 127, -100) : 10;
                        const float up = copysignf(__uint_as_float((uint32_t)(127 + 10 - e2) << 23), a.scale);
                        const int at_row = base_row + (i0 + i) * RI + lane / LR;
                        st_shared16(base + L::kQ + (uint32_t)(piece / 8) * (L::kRows * 128) + at_row * 128 +
                                        (((piece & 7) ^ (at_row & 7)) << 4),
                                    pack2<__half>(v[0] * up, v[1] * up), pack2<__half>(v[2] * up, v[3] * up),
                                    pack2<__half>(v[4] * up, v[5] * up), pack2<__half>(v[6] * up, v[7] * up));
                        // the factor of the scores to the row's own thread
                        const int mine = __shfl_sync(0xffffffffu, e2, lane % RI * LR);
                        if (lane / RI == i0 + i)
                            c = fmaxf(factor * __uint_as_float((uint32_t)(127 + mine - 10) << 23), FLT_MIN);
                    }
                }
            }
            }
            int ids = on ? pages_of(k, 0) : -1;
            asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
            named_bar_sync(1, 32 * (4 * L::kTiles + 1));  // with the issuer: the queries are there

            for (int j = 0; j < k.steps && on; ++j) {
                const int buf = tiles == 2 ? t : j & 1, nth = use.s(buf) + (tiles == 2 ? j : j >> 1);
                const uint32_t s_at = lanes + 128u * (uint32_t)buf;
                const unsigned present = __ballot_sync(0xffffffffu, (uint32_t)ids < pool);  // bit i: tokens 16 i on
                ids = pages_of(k, j + 1);
                if (!wait(kSFull + buf, nth)) break;
                tm_after();
                const bool edge = j * TN < all_lo || (j + 1) * TN > all_hi || present != (1u << (TN / 16)) - 1u;
                const int c_lo = row_lo - j * TN, c_hi = row_hi - j * TN;
                // A step goes by chunks of 32 columns of S (the next one on its way while
                // one is worked on); P is handed over in parts of two.
                auto mask = [&](int chunk, float (&v)[32]) {
                    if (edge) {
                        const int from = min(max(c_lo - 32 * chunk, 0), 32), to = min(max(c_hi - 32 * chunk, 0), 32);
                        uint32_t seen = (uint32_t)((1ull << to) - 1) & ~(uint32_t)((1ull << from) - 1);
                        if (!((present >> (2 * chunk)) & 1u)) seen &= 0xffff0000u;
                        if (!((present >> (2 * chunk + 1)) & 1u)) seen &= 0x0000ffffu;
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (!((seen >> i) & 1u)) v[i] = -INFINITY;
                    }
                };
                uint32_t p[32];
                float2 acc;
                // a chunk's probabilities to f16, and onto the part's sum
                auto powers = [&](int q, const float (&v)[32]) {
                    const float2 c2 = make_float2(c, c), off2 = make_float2(-off, -off);
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float2 x = ffma2(make_float2(v[2 * e], v[2 * e + 1]), c2, off2);
                        const float2 y = make_float2(ex2f(x.x), ex2f(x.y));
                        acc = __fadd2_rn(acc, y);
                        p[16 * q + e] = pack2<__half>(y.x, y.y);
                    }
                };
                float v[2][32];
                tm_ld32(s_at, v[0]);
#pragma unroll
                for (int part = 0; part < PARTS; ++part) {
                    acc = make_float2(0.f, 0.f);
                    const bool start = part == 0 && j == 0;  // (there is no reference yet)
                    if (!start) {
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            tm_wait_ld();
                            if (q == 0) tm_ld32(s_at + 32u * (2 * part + 1), v[1]);
                            mask(2 * part + q, v[q]);
                            powers(q, v[q]);
                        }
                    }
                    // A sum below 2^15 has no term above it: every one fits f16, and no maximum
                    // was needed.  Else (the first step, and when the scores rise) the reference
                    // moves to the maximum, and sum and O with it; and above it, the more the
                    // wider the scores spread: then later ones rise higher, and small
                    // probabilities matter less.
                    if (start || __any_sync(0xffffffffu, acc.x + acc.y > kTcMost)) {
                        float top = -INFINITY, all = 0.f;
                        int count = 0;
#pragma unroll 1
                        for (int q = 0; q < 2; ++q) {
                            float w[32];
                            tm_ld32(s_at + 32u * (2 * part + q), w);
                            tm_wait_ld();
                            mask(2 * part + q, w);
#pragma unroll
                            for (int e = 0; e < 32; ++e) {
                                top = fmaxf(top, w[e]);
                                all += w[e] == -INFINITY ? 0.f : w[e];
                                count += w[e] == -INFINITY ? 0 : 1;
                            }
                        }
                        const float spread = count > 0 ? fminf(0.25f * c * (top - all / (float)count), kTcRoom) : 0.f;
                        const float to = top == -INFINITY ? off : fmaxf(off, top * c - kTcBoost + fmaxf(spread, 0.f));
                        const float f = exp2f(off - to);
                        off = to;
                        sum *= f;
                        acc = make_float2(0.f, 0.f);
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            float w[32];
                            tm_ld32(s_at + 32u * (2 * part + q), w);
                            tm_wait_ld();
                            mask(2 * part + q, w);
                            powers(q, w);
                        }
                        if (j > 0 || part > 0) {
                            if (!(part > 0 ? wait(kOPart + t, use.o(t) + j) : wait(kODone + t, use.o(t) + j - 1))) break;
                            tm_after();
#pragma unroll 1
                            for (int d = 0; d < D; d += 32) {
                                float o[32];
                                const uint32_t o_at = lanes + kTmemO + (uint32_t)(t * D + d);
                                tm_ld32(o_at, o);
                                tm_wait_ld();
#pragma unroll
                                for (int e = 0; e < 32; ++e) o[e] *= f;
                                tm_st32(o_at, o);
                            }
                        }
                    }
                    sum += acc.x + acc.y;
                    // (over columns of S that were read: part i's go to [32 i, 32 i + 32))
#pragma unroll
                    for (int q = 0; q < 2; ++q) tm_st16(s_at + (uint32_t)(32 * part + 16 * q), p + 16 * q);
                    if (part + 1 < PARTS) tm_ld32(s_at + 32u * (2 * part + 2), v[0]);
                    tm_wait_st();
                    tm_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(kPFull + 2 * part + buf));
                }
                if (!ok) break;
            }

            // ------------------------------------------------ the row's output
            const Segment g = segment(at);
            at = g.next;
            if (on) {
                wait(kODone + t, use.o(t) + g.steps - 1);
                tm_after();
                const bool there = t * kTcTile + row < g.s.rows;
                const int r = g.s.r0 + t * kTcTile + row, qt = r / G;
                const float bad = __int_as_float(0x7fc00000);
                if (g.steps == g.s.steps) {
                    const float vs = a.v_scale ? a.v_scale[g.h] : 1.f;
                    const float inv = !ok ? bad : sum == 0.f ? 0.f : vs / sum;
                    const int64_t out = ((int64_t)g.s.b * a.T + qt) * a.Hq + g.h * G + r - qt * G;
#pragma unroll 1
                    for (int k = 0; k < D / 32; ++k) {
                        float v[32];
                        tm_ld32(lanes + kTmemO + (uint32_t)(t * D + 32 * k), v);
                        tm_wait_ld();
                        // (where the queries were: their last product is done)
                        const uint32_t at_row = base + L::kQ + (uint32_t)(k / 2) * (L::kRows * 128) + (t * kTcTile + row) * 128;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            float w[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) w[e] = ok ? v[8 * i + e] * inv : bad;
                            const RawPiece<T, 8> n = narrow_piece<T, 8>(w);
                            st_shared16(at_row + (((k % 2 * 4 + i) ^ (row & 7)) << 4), n.w.x, n.w.y, n.w.z, n.w.w);
                        }
                    }
                    __syncwarp();
                    constexpr int LR = D / 8, RI = 32 / LR;
                    const int piece = lane % LR;
#pragma unroll 4
                    for (int i = 0; i < LR; ++i) {  // whole rows, from the lanes that share them
                        const int at_row = t * kTcTile + (row & ~31) + i * RI + lane / LR, yr = g.s.r0 + at_row, yt = yr / G;
                        uint4 w;
                        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                                     : "r"(base + L::kQ + (uint32_t)(piece / 8) * (L::kRows * 128) + at_row * 128 +
                                           (((piece & 7) ^ (at_row & 7)) << 4)));
                        if (at_row >= g.s.rows) continue;
                        T *y = static_cast<T *>(a.y) + (((int64_t)g.s.b * a.T + yt) * a.Hq + g.h * G + yr - yt * G) * D + 8 * piece;
                        if (a.vec_y) {
                            *reinterpret_cast<uint4 *>(y) = w;
                        } else {
                            uint16_t *e = reinterpret_cast<uint16_t *>(y);
                            const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                            for (int n = 0; n < 8; ++n) e[n] = (uint16_t)(x[n / 2] >> (16 * (n % 2)));
                        }
                    }
                    __syncwarp();
                    if (there && a.lse)
                        a.lse[out] = !ok ? bad : sum == 0.f ? -INFINITY : (off + log2f(sum)) * 0.693147180559945309f;
                } else {
                    // (channel d of row i at [d][i], so that a warp's stores are whole lines)
                    float *ws = a.workspace + L::kNoteFloats + (int64_t)(2 * blockIdx.x + (first ? 0 : 1)) * L::kPartFloats;
                    const int i = t * kTcTile + row;
#pragma unroll 1
                    for (int k = 0; k < D / 32; ++k) {
                        float v[32];
                        tm_ld32(lanes + kTmemO + (uint32_t)(t * D + 32 * k), v);
                        tm_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) ws[(32 * k + e) * L::kRows + i] = ok ? v[e] : bad;
                        __syncwarp();
                    }
                    ws[D * L::kRows + i] = off;
                    ws[(D + 1) * L::kRows + i] = ok ? sum : bad;
                }
            }
            after(use, g);
            first = false;
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
        const uint32_t block_bytes = (uint32_t)kv_block_bytes(page, D), page_bytes = (uint32_t)a.H * block_bytes;
        const unsigned char *const codes = a.cache + 16 * piece + 4 * (order & 2);
        const int values = page * (D / 2 + D / 16), second = 8 - 8 * (order & 2);      // from there: V's; the other half
        const int to_scale = page * (D / 2) - 14 * piece - 4 * (order & 2);            // and, of row 0, the scales
        const uint32_t pick = order & 2 ? 0x3232u : 0x1010u;
        const uint32_t chunk = (uint32_t)panel * (TN * 128) + sub * 128 + ((((piece & 1) * 4 ^ order) ^ (sub & 7)) << 4);
        // (every token of a page that is there: which of them is seen, V's scales say)
        auto load = [&](int tok0, const unsigned char *from, int ids, int unit, uint2 (&q)[2], uint32_t &sc) {
            const int row = (tok0 + unit * UT + sub) & (page - 1);
            const uint32_t id = (uint32_t)__shfl_sync(0xffffffffu, ids, (unit * UT) >> 4);
            q[0] = q[1] = make_uint2(0, 0);
            sc = 0;
            if (id < pool) {
                const unsigned char *c = from + (uint64_t)id * page_bytes + row * (D / 2);
                // (the halves in the order that they are written in)
                asm volatile("ld.global.v2.u32 {%0, %1}, [%2];" : "=r"(q[0].x), "=r"(q[0].y) : "l"(c));
                asm volatile("ld.global.v2.u32 {%0, %1}, [%2];" : "=r"(q[1].x), "=r"(q[1].y) : "l"(c + second));
                asm volatile("ld.global.u16 %0, [%1];" : "=r"(sc) : "l"(c + (to_scale - row * (D / 2 - D / 16))));
            }
        };
        auto store = [&](uint32_t dst, int unit, const uint2 (&q)[2], uint32_t sc) {
            const uint32_t both = e4m3x2_to_f16(sc), at = dst + unit * UT * 128;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                uint32_t x = k % 2 ? q[k / 2].y : q[k / 2].x;
                if (D == 256 && (order & 1)) x = k % 2 ? q[k / 2].x : q[k / 2].y;
                const uint32_t f = __byte_perm(both, both, k < 2 ? pick : pick ^ 0x2222u);
                uint32_t e[4];
                e2m1x8_to_f16(x, e);
                // (units of four tokens: the odd ones' rows are 4 to 7 of the swizzle's eight)
                st_shared16(at + (chunk ^ (k << 4) ^ (UT == 4 ? (unit & 1) << 6 : 0)), times2(e[0], f), times2(e[1], f),
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
            for (int at = begin; at < end && ok;) {
                const unsigned char *from;
                Tokens k;
                {
                    const Segment g = segment(at);
                    k = tokens(g);
                    from = codes + (uint64_t)(uint32_t)g.h * block_bytes;
                    at = g.next;
                }
                if (k.steps == 0) break;
                int ids = pages_of(k, 0), ids_next = pages_of(k, 1);
                auto load_all = [&](int j) {
#pragma unroll
                    for (int i = 0; i < NK; ++i) load(k.tok0 + j * TN, from, ids, k0 + i, kq[i], ks[i]);
#pragma unroll
                    for (int i = 0; i < NV; ++i)
                        if (v0 + i < L::kUnits) load(k.tok0 + j * TN, from + values, ids, v0 + i, vq[i], vs[i]);
                };
                load_all(0);
                for (int j = 0; j < k.steps; ++j) {
                    const int nth = use.step + j, st = nth & 1;
                    ids = ids_next;
                    ids_next = pages_of(k, j + 2);
                    if (NK > 0) {
                        if (nth >= 2 && !wait(kKFree + st, (nth >> 1) - 1)) break;
#pragma unroll
                        for (int i = 0; i < NK; ++i) store(base + L::kK + st * L::kOpBytes, k0 + i, kq[i], ks[i]);
                        stored(kKFull + st);
                    }
                    if (NV > 0) {
                        if (nth >= 2 && !wait(kVFree + st, (nth >> 1) - 1)) break;
#pragma unroll
                        for (int i = 0; i < NV; ++i) {
                            // (a token that no row sees may hold anything: no NaN of it meets a zero)
                            const int tok = k.tok0 + j * TN + (v0 + i) * UT + sub;
                            if (tok < k.lo || tok >= k.hi) vs[i] = 0;
                            if (v0 + i < L::kUnits) store(base + L::kV + st * L::kOpBytes, v0 + i, vq[i], vs[i]);
                        }
                        stored(kVFull + st);
                    }
                    // (a fence waits for loads in flight: so none before the step's last one)
                    load_all(j + 1);
                }
                use.step += k.steps;
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
        constexpr uint32_t op_s = op_desc(TN, false), op_o = op_desc(D, true);
        const uint32_t one = elect_one(), tm = __shfl_sync(0xffffffffu, tmem, 0);
        const uint32_t sbase = __shfl_sync(0xffffffffu, base, 0);
        // (after a failed wait too the warp meets the softmax warps at every segment)
        for (int at = begin; at < end;) {
            const Segment g = segment(at);
            at = g.next;
            if (g.steps == 0) break;
            const int tiles = __shfl_sync(0xffffffffu, g.tiles, 0), steps = __shfl_sync(0xffffffffu, g.steps, 0);
            named_bar_sync(1, 32 * (4 * L::kTiles + 1));
            auto issue_s = [&](int j, int t) {
                const int buf = tiles == 2 ? t : j & 1, nth = use.step + j;
                if (!ok || (t == 0 && !wait(kKFull + (nth & 1), nth >> 1))) return;
                tm_after();
                const uint64_t q = operand_desc(sbase + L::kQ + t * kTcTile * 128, 16, 1024);
                const uint64_t k = operand_desc(sbase + L::kK + (nth & 1) * L::kOpBytes, 16, 1024);
#pragma unroll
                for (int s = 0; s < D / 16; ++s)
                    mma_ss(one, tm + 128u * buf, q + ((s >> 2) * (L::kRows * 128) + (s & 3) * 32) / 16,
                           k + ((s >> 2) * (TN * 128) + (s & 3) * 32) / 16, op_s, s > 0);
                commit_to(one, bar(kSFull + buf));
                if (t == tiles - 1) commit_to(one, bar(kKFree + (nth & 1)));
            };
            auto issue_o = [&](int j, int t) {
                const int buf = tiles == 2 ? t : j & 1, nth = use.step + j;
                if (!ok || (t == 0 && !wait(kVFull + (nth & 1), nth >> 1))) return;
                const uint64_t v = operand_desc(sbase + L::kV + (nth & 1) * L::kOpBytes, TN * 128, 1024);
#pragma unroll
                for (int part = 0; part < TN / 64; ++part) {
                    if (!wait(kPFull + 2 * part + buf, use.s(buf) + (tiles == 2 ? j : j >> 1))) return;
                    tm_after();
#pragma unroll
                    for (int s = 4 * part; s < 4 * part + 4; ++s)
                        mma_ts(one, tm + kTmemO + (uint32_t)(t * D), tm + 128u * buf + 8u * s, v + s * 2048 / 16, op_o, j > 0 || s > 0);
                    if (part < TN / 64 - 1) commit_to(one, bar(kOPart + t));
                }
                commit_to(one, bar(kODone + t));
                if (t == tiles - 1) commit_to(one, bar(kVFree + (nth & 1)));
            };
            for (int t = 0; t < tiles; ++t) issue_s(0, t);
            for (int j = 0; j < steps && ok; ++j) {
                if (tiles == 1 && j + 1 < steps) issue_s(j + 1, 0);
                for (int t = 0; t < tiles; ++t) {
                    issue_o(j, t);
                    if (tiles == 2 && j + 1 < steps) issue_s(j + 1, t);
                }
            }
            after(use, g);
        }
        // nothing is in flight when the tensor memory goes
        commit_to(one, bar(kDrain));
        if (!mbar_wait_bounded(bar(kDrain), 0, kDrainCycles)) ok = false;
    }
    if (!ok) *ta.wait_flag = 1u;
    tm_before();
    __syncthreads();
    tm_after();
    if (warp == 0)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(kTmemCols));
}

// Joins the parts of the units that are cut: block (c, i) rows 8 i on of the unit
// that block c's part is the second of, if it is of any.
template <typename T, int D>
__global__ void __launch_bounds__(256) attend_tc_join_kernel(const AttendArgs a, int row_blocks, int groups) {
    using L = Tc<D>;
    __shared__ float so[D][9];
    pdl_trigger();
    pdl_wait();
    const int c = blockIdx.x / groups + 1, r0 = (blockIdx.x % groups) * 8, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int4 note = reinterpret_cast<const int4 *>(a.workspace)[c];  // pair, head, first partial result, last block
    if (note.x < 0) return;
    const TcSpan s = tc_span<D>(a, note.x, row_blocks);
    if (r0 >= s.rows) return;
    // eight neighbouring rows of a channel are 32 bytes: lane (channel lane / 8 of
    // the warp's four, row lane % 8) adds them up
    const int i = r0 + lane % 8;
    const bool there = i < s.rows;
    auto part = [&](int q) { return a.workspace + L::kNoteFloats + (int64_t)q * L::kPartFloats; };
    float ref = -1e30f, sum = 0.f, acc[D / 32];
#pragma unroll
    for (int k = 0; k < D / 32; ++k) acc[k] = 0.f;
    for (int q = c - 1; q <= note.w; ++q) {
        const float *ws = part(q == c - 1 ? note.z : 2 * q);
        const float pr = there ? ws[D * L::kRows + i] : 0.f, ps = there ? ws[(D + 1) * L::kRows + i] : 0.f;
        const float to = fmaxf(ref, pr), f = exp2f(ref - to), g = exp2f(pr - to);
        ref = to;
        sum = sum * f + ps * g;
#pragma unroll
        for (int k = 0; k < D / 32; ++k)
            acc[k] = acc[k] * f + (there ? ws[(32 * k + 4 * warp + lane / 8) * L::kRows + i] : 0.f) * g;
    }
    const float vs = a.v_scale ? a.v_scale[note.y] : 1.f, inv = sum == 0.f ? 0.f : vs / sum;
#pragma unroll
    for (int k = 0; k < D / 32; ++k) so[32 * k + 4 * warp + lane / 8][lane % 8] = acc[k] * inv;
    const int G = a.Hq / a.H;
    auto place = [&](int row) {
        const int r = s.r0 + row, t = r / G;
        return ((int64_t)s.b * a.T + t) * a.Hq + note.y * G + r - t * G;
    };
    if (threadIdx.x < 8 && there && a.lse)
        a.lse[place(i)] = sum == 0.f ? -INFINITY : (ref + log2f(sum)) * 0.693147180559945309f;
    __syncthreads();
    if (r0 + warp < s.rows) {
        T *y = static_cast<T *>(a.y) + place(r0 + warp) * D;
        for (int d = lane; d < D; d += 32) st_from_f32(y + d, so[d][warp]);
    }
}

// A call is cut along its tokens unless its units fill the GPU many times over (or
// its steps might pass 31 bits).
bool tc_cut(int64_t pairs, int64_t H, int64_t capacity) {
    return pairs <= kTcMaxPairs && pairs * H < 16 * kTcParts && pairs * H * (capacity / 64 + 1) <= INT32_MAX;
}
int64_t tc_pairs(int64_t B, int64_t rows, int64_t D) { return B * ((rows + (D == 256 ? 127 : 255)) / (D == 256 ? 128 : 256)); }

template <typename T, int D>
cudaError_t launch_tc(const AttendArgs &a, cudaStream_t s) {
    using L = Tc<D>;
    void *flag = nullptr;
    cudaError_t e = cudaGetSymbolAddress(&flag, g_attend_tc_wait_flag);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(attend_tc_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)L::kSmem);
    if (e != cudaSuccess) return e;
    const int64_t rows = a.T * (a.Hq / a.H), pairs = tc_pairs(a.B, rows, D), units = pairs * a.H;
    if (units > INT32_MAX) return cudaErrorInvalidConfiguration;
    const bool cut = tc_cut(pairs, a.H, (int64_t)a.width << a.page_shift);
    TcArgs ta{a, (int)pairs, (int)(pairs / a.B), static_cast<unsigned *>(flag), wait_bound_cycles(), inject_wait_expiry(), !cut};
    e = launch_dependent(attend_tc_kernel<T, D>, cut ? kTcParts : (unsigned)units, kTcThreads, L::kSmem, s, ta);
    if (e != cudaSuccess || !cut) return e;
    const int groups = (int)((std::min<int64_t>(rows, L::kRows) + 7) / 8);
    return launch_dependent(attend_tc_join_kernel<T, D>, (unsigned)((kTcParts - 1) * groups), 256, 0, s, a, ta.row_blocks, groups);
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

int64_t attend_tc_workspace_bytes(int64_t B, int64_t T, int64_t Hq, int64_t H, int64_t D) {
    const int64_t rows = T * (Hq / H);
    if (!attend_tc_rows(rows) || !tc_cut(tc_pairs(B, rows, D), H, 0)) return 0;
    return D == 64 ? Tc<64>::kWorkspace : D == 128 ? Tc<128>::kWorkspace : Tc<256>::kWorkspace;
}

// (up to 16 rows the other form's narrow products fit them)
bool attend_tc_rows(int64_t rows) { return rows > 16; }
bool attend_takes_tc(DType dt, const AttendArgs &a) { return dt != DType::F32 && attend_tc_rows(a.T * (a.Hq / a.H)); }

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
