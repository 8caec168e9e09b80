// sample.cu -- one token per row of logits: temperature, top-k, top-p, min-p,
// then a race on given exponential noise.
//
// With max the row's largest logit and e_i = exp((l_i - max) / T), order the
// tokens by (l descending, index ascending).  Every one of the three cuts
// keeps a prefix of that order:
//     top-k: the first k;
//     top-p: rank n while the mass of the ranks before it is below top_p
//            times the mass of the top-k tokens;
//     min-p: e_i >= min_p (the largest e is 1).
// The token is the largest e_i / noise_i of what is left (with standard
// exponential noise that draws i with probability proportional to e_i), ties
// to the lowest index.  logprob = (l - max)/T - log(sum of all e_i).
//
// A row is read from memory once, with its maximum and its mass taken on the
// way: a cluster of CTAs holds its slices in shared memory.  The cuts then go
// without a sort of the row, by a list of the tokens near the cut:
//   - top-k up to half a CTA's threads: the k-th largest of the threads' own
//     maxima bounds the k-th logit of a slice from below, and few more than k
//     tokens reach it.  One CTA takes the slices' lists and finishes the row.
//   - otherwise a histogram over bins of equal width in the logit counts the
//     tokens.  For top-p the counts bound the mass above each bin to within
//     the width of one, which leaves a bracket of one or two bins.  A second
//     pass sums the mass above the bracket and lists the tokens in it; one
//     CTA finds the exact token of the list at which the cut lies.
//   - a list is not sorted either: its tokens lie in the CTA's registers, and
//     the logit at the cut (then, among equal ones, the index) is found by
//     histograms over eight bits at a time.
//   - where a list does not fit (many equal logits), histograms over 11 bits
//     of the logit's ordered key at a time find the value at the cut, and its
//     tokens are counted in index order.
// Masses in those are integers (units of 2^-40 of the largest token's), sums
// are taken in fixed orders, and the order in which a list is filled is not
// looked at: results do not change from run to run.  The noise is read
// only for tokens that are left.
//
// What bounds it: one row of 32000 f32 with top-k 50 takes 11.6 us, about ten
// exchanges over the block and two over the cluster one after another.  128
// rows of 131072 bf16 with the three cuts take 79 us (a tenth of the copy
// rate): passes over shared memory, the list and the race of the rows with a
// top-p cut.  256 rows of 100003 uncut take 58 us (2.6 TB/s): two passes, the
// race waiting for the row's maximum.  A single pass over logits and noise in
// the log domain took 56.5 us there, at the price of registers for the cuts
// (83 us), and was not kept.
#include <cfloat>
#include <cooperative_groups.h>

#include "layer.h"
#include "pieces.cuh"

namespace gdn {

namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;         // bins of a histogram of masses
constexpr int kCountBins = 4096;    // bins of a histogram of counts alone (over count and lo)
constexpr int kMaxCluster = 8;
constexpr int kList = 1024;         // tokens near a cut that a CTA lists
constexpr int kNear = 2048;         // tokens near a cut that one CTA takes
constexpr int kOwn = kNear / kThreads;
constexpr int kMaxK = kThreads / 2; // top-k by the threads' maxima

// What is left so far: logits above `l`, and those equal to it with an index
// below `end`.  Masked tokens (-inf) are never left.
struct alignas(8) Cut {
    float l;
    uint32_t end;
    __device__ __forceinline__ bool keeps(float x, uint32_t idx) const { return x > l || (x == l && idx < end); }
};
__device__ __forceinline__ Cut no_cut() { return Cut{-FLT_MAX, 0xffffffffu}; }

// Shared memory before the row's slice, in 32-bit words, each read and written
// by itself: word offsets.  A histogram of masses holds tokens, and mass in
// two words; over the same memory lie a histogram of counts alone and, behind
// it, this CTA's list of tokens near a cut (ordered bits, then indexes).  The
// first CTA of a cluster has the lists of all behind that.
constexpr uint32_t kCount = 0, kLo = kBins, kHi = 2 * kBins;
constexpr uint32_t kListKey = kHi, kListIdx = kListKey + kList;
constexpr uint32_t kNearKey = 3 * kBins, kNearIdx = kNearKey + kNear;
constexpr uint32_t kRed = kNearIdx + kNear;                             // one word per warp, three times
constexpr uint32_t kRed2 = kRed + kWarps, kRed3 = kRed2 + kWarps;
constexpr uint32_t kWords = kRed3 + kWarps;                             // single words
constexpr uint32_t kPartMax = kWords, kPartZ = kWords + 1, kPartLeast = kWords + 2, kPartSum = kWords + 3,
                   kPartAbove = kWords + 4, kListN = kWords + 5, kTies = kWords + 6, kFoundBin = kWords + 9, kFoundLast = kWords + 10, kFoundCount = kWords + 11,
                   kFoundN = kWords + 12, kFoundMassLo = kWords + 13, kFoundMassHi = kWords + 14,
                   kFoundWLo = kWords + 15, kFoundWHi = kWords + 16, kLimit = kWords + 17, kCutL = kWords + 18,
                   kCutEnd = kWords + 19, kRace = kWords + 20, kNearN = kWords + 21, kNearAt = kWords + 22, kPartIn = kWords + 23,
                   kTightBin = kWords + 24, kTightLast = kWords + 25;
constexpr uint32_t kSharedBytes = (kWords + 28) * 4;
static_assert(kCountBins <= kHi && 2 * kList <= kBins && kSharedBytes % 16 == 0, "layout");

// Word accesses at a CTA's own shared memory, and at that of another CTA of
// the cluster (`cs` CTAs; a CTA alone takes its own).
struct Shared {
    uint32_t base;
    int cs;
    __device__ __forceinline__ uint32_t at(uint32_t w) const { return base + 4 * w; }
    __device__ __forceinline__ uint32_t get(uint32_t w) const {
        uint32_t v;
        asm volatile("ld.shared.u32 %0, [%1];\n" : "=r"(v) : "r"(at(w)) : "memory");
        return v;
    }
    __device__ __forceinline__ void put(uint32_t w, uint32_t v) const {
        asm volatile("st.shared.u32 [%0], %1;\n" ::"r"(at(w)), "r"(v) : "memory");
    }
    __device__ __forceinline__ float getf(uint32_t w) const { return __uint_as_float(get(w)); }
    __device__ __forceinline__ void putf(uint32_t w, float v) const { put(w, __float_as_uint(v)); }
    __device__ __forceinline__ uint32_t add(uint32_t w, uint32_t v) const {  // returns what was there
        uint32_t old;
        asm volatile("atom.shared.add.u32 %0, [%1], %2;\n" : "=r"(old) : "r"(at(w)), "r"(v) : "memory");
        return old;
    }
    __device__ __forceinline__ void add_only(uint32_t w, uint32_t v) const {
        asm volatile("red.shared.add.u32 [%0], %1;\n" ::"r"(at(w)), "r"(v) : "memory");
    }
    __device__ __forceinline__ void max_only(uint32_t w, uint32_t v) const {
        asm volatile("red.shared.max.u32 [%0], %1;\n" ::"r"(at(w)), "r"(v) : "memory");
    }
    __device__ __forceinline__ void min_only(uint32_t w, uint32_t v) const {
        asm volatile("red.shared.min.u32 [%0], %1;\n" ::"r"(at(w)), "r"(v) : "memory");
    }
    __device__ __forceinline__ uint32_t mapped(uint32_t w, int rank) const {
        uint32_t a;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(a) : "r"(at(w)), "r"(rank));
        return a;
    }
    __device__ __forceinline__ uint32_t get(uint32_t w, int rank) const {
        if (cs == 1) return get(w);
        uint32_t v;
        asm volatile("ld.shared::cluster.u32 %0, [%1];\n" : "=r"(v) : "r"(mapped(w, rank)) : "memory");
        return v;
    }
    __device__ __forceinline__ void put(uint32_t w, int rank, uint32_t v) const {
        if (cs == 1) return put(w, v);
        asm volatile("st.shared::cluster.u32 [%0], %1;\n" ::"r"(mapped(w, rank)), "r"(v) : "memory");
    }
    // atomic on another CTA's word; returns what was there
    __device__ __forceinline__ uint32_t add(uint32_t w, int rank, uint32_t v) const {
        if (cs == 1) return add(w, v);
        uint32_t old;
        asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;\n" : "=r"(old) : "r"(mapped(w, rank)), "r"(v) : "memory");
        return old;
    }
    // the word of every CTA, lane q of a warp taking that of CTA q (the others
    // `none`): one trip for all of them
    __device__ __forceinline__ uint32_t each_cta(uint32_t w, uint32_t none) const {
        const int lane = threadIdx.x % 32;
        return lane < cs ? get(w, lane) : none;
    }
    // sum of a float of every CTA, in the order of the CTAs
    __device__ __forceinline__ float sum_ctas(uint32_t w) const {
        const float v = __uint_as_float(each_cta(w, 0));
        float s = __shfl_sync(0xffffffffu, v, 0);
        for (int q = 1; q < cs; ++q) s += __shfl_sync(0xffffffffu, v, q);
        return s;
    }
    // the last step of a row in whose words no CTA but the first is still read:
    // that one goes on when all have come, the others do not wait for it
    __device__ __forceinline__ void leave(int rank) const {
        if (cs == 1) return;
        asm volatile("barrier.cluster.arrive.release.aligned;\n" ::: "memory");
        if (rank == 0) asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
    }
    // every CTA of the cluster in step, and its writes visible to the others
    __device__ __forceinline__ void sync() const {
        if (cs > 1) cg::this_cluster().sync();
        else __syncthreads();
    }
};

// The logit as the rules see it: NaN is masked, +inf is the largest finite
// value of its type.
template <typename T> __device__ __forceinline__ float largest();
template <> __device__ __forceinline__ float largest<float>() { return FLT_MAX; }
template <> __device__ __forceinline__ float largest<__nv_bfloat16>() { return __uint_as_float(0x7f7f0000u); }
template <> __device__ __forceinline__ float largest<__half>() { return 65504.f; }
template <typename T> __device__ __forceinline__ float logit(T x) {
    return fminf(fmaxf(Elem<T>::to_f32(x), -INFINITY), largest<T>());
}
// The same for a 16-byte piece, and its largest logit.
__device__ __forceinline__ uint4 clean(const RawPiece<float, 4> &r) {
    float v[4];
    widen<float, 4>(v, r);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = fminf(fmaxf(v[i], -INFINITY), FLT_MAX);
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
}
template <typename H2> __device__ __forceinline__ uint32_t clean2(uint32_t w, uint32_t low, uint32_t high) {
    const H2 x = __hmin2(__hmax2(*reinterpret_cast<const H2 *>(&w), *reinterpret_cast<const H2 *>(&low)),
                         *reinterpret_cast<const H2 *>(&high));
    return *reinterpret_cast<const uint32_t *>(&x);
}
__device__ __forceinline__ uint4 clean(const RawPiece<__nv_bfloat16, 8> &r) {
    constexpr uint32_t low = 0xff80ff80u, high = 0x7f7f7f7fu;
    return make_uint4(clean2<__nv_bfloat162>(r.w.x, low, high), clean2<__nv_bfloat162>(r.w.y, low, high),
                      clean2<__nv_bfloat162>(r.w.z, low, high), clean2<__nv_bfloat162>(r.w.w, low, high));
}
__device__ __forceinline__ uint4 clean(const RawPiece<__half, 8> &r) {
    constexpr uint32_t low = 0xfc00fc00u, high = 0x7bff7bffu;
    return make_uint4(clean2<__half2>(r.w.x, low, high), clean2<__half2>(r.w.y, low, high),
                      clean2<__half2>(r.w.z, low, high), clean2<__half2>(r.w.w, low, high));
}
template <typename H2> __device__ __forceinline__ float max8(const uint4 &w) {
    const H2 a = __hmax2(*reinterpret_cast<const H2 *>(&w.x), *reinterpret_cast<const H2 *>(&w.y));
    const H2 b = __hmax2(*reinterpret_cast<const H2 *>(&w.z), *reinterpret_cast<const H2 *>(&w.w));
    const H2 c = __hmax2(a, b);
    return fmaxf(__low2float(c), __high2float(c));
}
template <typename T> __device__ __forceinline__ float piece_max(const uint4 &w);
template <> __device__ __forceinline__ float piece_max<__nv_bfloat16>(const uint4 &w) { return max8<__nv_bfloat162>(w); }
template <> __device__ __forceinline__ float piece_max<__half>(const uint4 &w) { return max8<__half2>(w); }
template <> __device__ __forceinline__ float piece_max<float>(const uint4 &w) {
    return fmaxf(fmaxf(__uint_as_float(w.x), __uint_as_float(w.y)), fmaxf(__uint_as_float(w.z), __uint_as_float(w.w)));
}

__device__ __forceinline__ uint32_t order_bits(float l) {
    const uint32_t u = __float_as_uint(l + 0.f);  // -0 is 0
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float from_order_bits(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint4 piece_at(uint32_t shared_addr) {
    uint4 w;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];\n"
                 : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                 : "r"(shared_addr)
                 : "memory");
    return w;
}
// 16 bytes of a row, and one noise value; the addresses are aligned by how they
// are made, and kept so.
__device__ __forceinline__ uint4 row_piece(const void *p) {
    uint4 w;
    asm volatile("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];\n"
                 : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                 : "l"(reinterpret_cast<uint64_t>(p) & ~(uint64_t)15));
    return w;
}
__device__ __forceinline__ float noise_at(const float *p) {
    float v;
    asm volatile("ld.global.nc.f32 %0, [%1];\n" : "=f"(v) : "l"(p));
    return v;
}
__device__ __forceinline__ void put_piece(uint32_t shared_addr, const uint4 &w) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};\n" ::"r"(shared_addr), "r"(w.x), "r"(w.y), "r"(w.z),
                 "r"(w.w)
                 : "memory");
}
template <typename T> __device__ __forceinline__ float element_at(uint32_t shared_addr);
template <> __device__ __forceinline__ float element_at<float>(uint32_t shared_addr) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];\n" : "=f"(v) : "r"(shared_addr) : "memory");
    return v;
}
__device__ __forceinline__ uint16_t half_at(uint32_t shared_addr) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];\n" : "=h"(v) : "r"(shared_addr) : "memory");
    return v;
}
template <> __device__ __forceinline__ float element_at<__nv_bfloat16>(uint32_t shared_addr) {
    return unpack2<__nv_bfloat16>(half_at(shared_addr)).x;
}
template <> __device__ __forceinline__ float element_at<__half>(uint32_t shared_addr) {
    return unpack2<__half>(half_at(shared_addr)).x;
}

template <typename T, bool CACHED> struct Row {
    [[maybe_unused]] static constexpr int VE = 16 / sizeof(T);
    uint32_t pieces;     // CACHED: shared address of the slice's pieces (16-byte aligned)
    int mis;             // CACHED: elements before the slice's first in its first piece
    const T *src;        // the slice in memory
    int n;               // tokens in the slice
    uint32_t base;       // index of the first
    __device__ __forceinline__ int count() const { return (mis + n + VE - 1) / VE; }  // pieces
    // f(logit, index) for every token of the slice with a logit of at least
    // `low` (above -inf), thread by thread.  Pieces in shared memory hold
    // clean logits, and -inf around the slice; a piece without such a token
    // costs one comparison.
    template <typename F> __device__ __forceinline__ void each(float low, F &&f) const {
        if constexpr (CACHED) {
            each_piece(low, [&](const float2 (&v)[VE / 2], int i0) {
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    const float l = e % 2 ? v[e / 2].y : v[e / 2].x;
                    if (l >= low) f(l, base + (uint32_t)(i0 + e));
                }
            });
        } else {
            for (int i = threadIdx.x; i < n; i += kThreads) {
                const float l = logit(src[i]);
                if (l >= low) f(l, base + (uint32_t)i);
            }
        }
    }
    // f(logits of a piece, place of its first in the slice) for every piece of
    // a CACHED slice that has a logit of at least `low`; the first piece's
    // place may be below 0, and places outside the slice hold -inf
    template <typename F> __device__ __forceinline__ void each_piece(float low, F &&f) const {
        const int end = count();
        for (int j = threadIdx.x; j < end; j += kThreads) {
            RawPiece<T, VE> raw;
            raw.w = piece_at(pieces + 16 * j);
            if (piece_max<T>(raw.w) < low) continue;
            float2 v[VE / 2];
            widen2<T, VE>(v, raw);
            f(v, j * VE - mis);
        }
    }
    // the same, all lanes of a warp together (those without a piece get -inf)
    template <typename F> __device__ __forceinline__ void each_piece_warp(float low, F &&f) const {
        const int end = count();
        for (int j0 = threadIdx.x / 32 * 32; j0 < end; j0 += kThreads) {
            const int j = j0 + threadIdx.x % 32;
            RawPiece<T, VE> raw;
            float v1[VE];
#pragma unroll
            for (int e = 0; e < VE; ++e) v1[e] = -INFINITY;
            if (j < end) raw.w = piece_at(pieces + 16 * j);
            else raw = narrow_piece<T, VE>(v1);
            if (!__any_sync(0xffffffffu, piece_max<T>(raw.w) >= low)) continue;
            float2 v[VE / 2];
            widen2<T, VE>(v, raw);
            f(v, j * VE - mis);
        }
    }
    __device__ __forceinline__ float at(int i) const {
        return CACHED ? element_at<T>(pieces + (uint32_t)(mis + i) * (uint32_t)sizeof(T)) : logit(src[i]);
    }
};

__device__ __forceinline__ unsigned long long join64(uint32_t lo, uint32_t hi) {
    return (unsigned long long)lo | ((unsigned long long)hi << 32);
}

__device__ __forceinline__ float block_sum(float v, const Shared &sh) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if (threadIdx.x % 32 == 0) sh.putf(kRed + threadIdx.x / 32, v);
    __syncthreads();
    v = 0.f;
    for (int i = 0; i < kWarps; ++i) v += sh.getf(kRed + i);
    return v;
}

// Sums `words` counters over the CTAs: each adds up its share and hands the
// sums to all; it alone reads and writes those.
__device__ __forceinline__ void merge_bins(const Shared &sh, uint32_t first, int words, int rank) {
    const int share = words / sh.cs;
    for (int i = threadIdx.x; i < share; i += kThreads) {
        const uint32_t w = first + rank * share + i;
        uint32_t part[kMaxCluster], sum = 0;
#pragma unroll
        for (int q = 0; q < kMaxCluster; ++q) part[q] = q < sh.cs ? sh.get(w, q) : 0;
#pragma unroll
        for (int q = 0; q < kMaxCluster; ++q) sum += part[q];
#pragma unroll
        for (int q = 0; q < kMaxCluster; ++q)
            if (q < sh.cs) sh.put(w, q, sum);
    }
}

// The bin, counted from the top, of a histogram (over all CTAs of the cluster)
// in which the running count reaches `k` or the running mass reaches
// `target`; kFoundBin stays ~0 if none does.  The running values start from
// `above_count` and `above_mass`.
template <bool MASS>
__device__ __forceinline__ void find_bin(const Shared &sh, int rank, uint32_t above_count,
                                         unsigned long long above_mass, uint32_t k, double target) {
    sh.sync();
    if (sh.cs > 1) {
        // two-word masses: the CTAs' low words are summed apart from their carry
        const int share = kBins / sh.cs;
        for (int i = threadIdx.x; i < share; i += kThreads) {
            const uint32_t bin = rank * share + i;
            uint32_t c = 0;
            unsigned long long m = 0;
            for (int q = 0; q < sh.cs; ++q) {
                c += sh.get(kCount + bin, q);
                if (MASS) m += join64(sh.get(kLo + bin, q), sh.get(kHi + bin, q));
            }
            for (int q = 0; q < sh.cs; ++q) {
                sh.put(kCount + bin, q, c);
                if (MASS) {
                    sh.put(kLo + bin, q, (uint32_t)m);
                    sh.put(kHi + bin, q, (uint32_t)(m >> 32));
                }
            }
        }
        sh.sync();
    }
    // running sums from the top bin: PB bins per thread
    constexpr int PB = kBins / kThreads;
    uint32_t c[PB], ctot = 0;
    unsigned long long m[PB], mtot = 0;
#pragma unroll
    for (int j = 0; j < PB; ++j) {
        const uint32_t bin = kBins - 1 - (threadIdx.x * PB + j);
        c[j] = sh.get(kCount + bin);
        m[j] = MASS ? join64(sh.get(kLo + bin), sh.get(kHi + bin)) : 0;
        ctot += c[j];
        mtot += m[j];
    }
    uint32_t cin = ctot;
    unsigned long long min_ = mtot;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t cv = __shfl_up_sync(0xffffffffu, cin, o);
        const unsigned long long mv = MASS ? __shfl_up_sync(0xffffffffu, min_, o) : 0;
        if (lane >= o) {
            cin += cv;
            min_ += mv;
        }
    }
    if (lane == 31) {
        sh.put(kRed + warp, cin);
        sh.put(kRed2 + warp, (uint32_t)min_);
        sh.put(kRed3 + warp, (uint32_t)(min_ >> 32));
    }
    __syncthreads();
    uint32_t cbase = above_count + cin - ctot;
    unsigned long long mbase = above_mass + min_ - mtot;
    for (int i = 0; i < warp; ++i) {
        cbase += sh.get(kRed + i);
        mbase += join64(sh.get(kRed2 + i), sh.get(kRed3 + i));
    }
#pragma unroll
    for (int j = 0; j < PB; ++j) {
        const bool before = MASS ? (double)mbase < target : cbase < k;
        const bool reached = MASS ? (double)(mbase + m[j]) >= target : cbase + c[j] >= k;
        if (before && reached) {
            sh.put(kFoundBin, kBins - 1 - (threadIdx.x * PB + j));
            sh.put(kFoundCount, cbase);
            sh.put(kFoundMassLo, (uint32_t)mbase);
            sh.put(kFoundMassHi, (uint32_t)(mbase >> 32));
            sh.put(kFoundN, c[j]);
            sh.put(kFoundWLo, (uint32_t)m[j]);
            sh.put(kFoundWHi, (uint32_t)(m[j] >> 32));
        }
        cbase += c[j];
        mbase += m[j];
    }
    __syncthreads();
}

// e in units of 2^-40 added to a bin's mass.
__device__ __forceinline__ void add_mass(const Shared &sh, uint32_t bin, float e) {
    uint32_t wh = 0;
    if (e >= 0x1p-8f) {
        wh = __float2uint_rz(e * 0x1p8f);
        e -= (float)wh * 0x1p-8f;
    }
    const uint32_t wl = __float2uint_rz(e * 0x1p40f);
    const uint32_t old = sh.add(kLo + bin, wl);
    if (old + wl < old) ++wh;
    if (wh) sh.add_only(kHi + bin, wh);
}

// `cut`, narrowed to the tokens before the place where the running count
// reaches `k` (or the running mass reaches `target`), in the order (l
// descending, index ascending), among those of logit `low` or more of which
// `in(l, idx)` holds; `mass(l)` is a token's e.  For any number of tokens at
// the cut.
template <bool MASS, int ROUNDS, typename RowT, typename In, typename Mass>
__device__ __forceinline__ Cut narrow(const RowT &row, const Shared &sh, int rank, const Cut cut, uint32_t k,
                                      double target, float low, In &&in, Mass &&mass) {
    uint32_t above_count = 0, prefix = 0;
    unsigned long long above_mass = 0;
    int shift = 32;
#pragma unroll 1
    for (int round = 0; round < ROUNDS; ++round) {
        const int bits = round == 2 ? 10 : 11;
        const int next = shift - bits;
        __syncthreads();
        for (int i = threadIdx.x; i < kBins; i += kThreads) {
            sh.put(kCount + i, 0);
            if (MASS) {
                sh.put(kLo + i, 0);
                sh.put(kHi + i, 0);
            }
        }
        if (threadIdx.x == 0) sh.put(kFoundBin, 0xffffffffu);
        __syncthreads();
        row.each(low, [&](float l, uint32_t idx) {
            const uint32_t key = order_bits(l);
            if ((round > 0 && (key >> shift) != prefix) || !in(l, idx)) return;
            const uint32_t bin = (key >> next) & ((1u << bits) - 1);
            sh.add_only(kCount + bin, 1u);
            if (MASS) add_mass(sh, bin, mass(l));
        });
        find_bin<MASS>(sh, rank, above_count, above_mass, k, target);
        const uint32_t bin = sh.get(kFoundBin);
        if (bin == 0xffffffffu) return cut;  // every token that takes part is left
        prefix = (prefix << bits) | bin;
        shift = next;
        above_count = sh.get(kFoundCount);
        above_mass = join64(sh.get(kFoundMassLo), sh.get(kFoundMassHi));
    }
    // the tokens of the last bin are equal (16-bit logits have equal low bits
    // of the key): the first `want` of them stay
    const float l_eq =
        from_order_bits((prefix << shift) | (shift > 0 && prefix >> (31 - shift) == 0 ? (1u << shift) - 1 : 0));
    const uint32_t n_eq = sh.get(kFoundN);
    uint32_t want;
    if (MASS) {
        const double each = (double)join64(sh.get(kFoundWLo), sh.get(kFoundWHi)) / n_eq;
        const double q = each > 0 ? ceil((target - (double)above_mass) / each) : 1.0;
        want = q < 1 ? 1 : (q > (double)n_eq ? n_eq : (uint32_t)q);
    } else {
        want = k - above_count;
    }
    uint32_t end = 0xffffffffu;
    if (want < n_eq) {
        // index of the want-th of them: the CTAs' slices are in index order,
        // and so are the warps' parts of a slice
        const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
        const int per = ((row.n + kWarps - 1) / kWarps + 31) / 32 * 32;
        const int i0 = warp * per, i1 = i0 + per < row.n ? i0 + per : row.n;
        auto equal = [&](int i) { return i < i1 && row.at(i) == l_eq && in(l_eq, row.base + (uint32_t)i); };
        uint32_t mine = 0;
        for (int i = i0; i < i1; i += 32) mine += __popc(__ballot_sync(0xffffffffu, equal(i + lane)));
        if (lane == 0) sh.put(kRed + warp, mine);
        __syncthreads();
        if (threadIdx.x == 0) {
            uint32_t s = 0;
            for (int i = 0; i < kWarps; ++i) s += sh.get(kRed + i);
            sh.put(kTies, s);
        }
        sh.sync();
        uint32_t before = 0;
        for (int q = 0; q < rank; ++q) before += sh.get(kTies, q);
        for (int i = 0; i < warp; ++i) before += sh.get(kRed + i);
        if (before < want && want <= before + mine) {
            uint32_t left = want - before;  // the left-th of this warp's
            for (int i = i0; i < i1; i += 32) {
                const uint32_t m = __ballot_sync(0xffffffffu, equal(i + lane));
                const uint32_t c = __popc(m);
                if (left <= c) {
                    const int pos = __fns(m, 0, (int)left);
                    if (lane == 0)
                        for (int q = 0; q < sh.cs; ++q) sh.put(kLimit, q, row.base + (uint32_t)(i + pos));
                    break;
                }
                left -= c;
            }
        }
        sh.sync();
        end = sh.get(kLimit) + 1;
    }
    return Cut{l_eq, end};
}

// Appends a token to this CTA's list (past its end, only counts it).
__device__ __forceinline__ void enlist(const Shared &sh, float l, uint32_t idx) {
    const uint32_t at = sh.add(kListN, 1u);
    if (at < kList) {
        sh.put(kListKey + at, order_bits(l));
        sh.put(kListIdx + at, idx);
    }
}

// Hands this CTA's list to the first CTA, in no order.
// All CTAs' lists are there once the cluster is in step; then kNearN of the
// first CTA is their length, or above kNear if they do not fit.
__device__ __forceinline__ void send_list(const Shared &sh) {
    __syncthreads();
    const uint32_t c = sh.get(kListN);
    if (threadIdx.x == 0) sh.put(kNearAt, sh.add(kNearN, 0, c <= kList ? c : kNear + 1));
    __syncthreads();
    const uint32_t at = sh.get(kNearAt);
    if (c > kList || at > kNear || at + c > kNear) return;
    for (uint32_t i = threadIdx.x; i < c; i += kThreads) {
        sh.put(kNearKey + at + i, 0, sh.get(kListKey + i));
        sh.put(kNearIdx + at + i, 0, sh.get(kListIdx + i));
    }
}
// Their length in every CTA, or -1.
__device__ __forceinline__ int listed(const Shared &sh) {
    const uint32_t n = sh.get(kNearN, 0);
    return n <= kNear ? (int)n : -1;
}

// The lists in the first CTA, in registers: token j of a thread has key 0 if
// there is none.
struct Near {
    uint32_t key[kOwn], idx[kOwn];
    int own;  // tokens of a thread, at most
    __device__ __forceinline__ void load(const Shared &sh, int total) {
        own = (total + kThreads - 1) / kThreads;
#pragma unroll
        for (int j = 0; j < kOwn; ++j) {
            const int i = threadIdx.x + j * kThreads;
            key[j] = i < total ? sh.get(kNearKey + i) : 0;
            idx[j] = i < total ? sh.get(kNearIdx + i) : 0;
        }
    }
};

// A digit's histogram of a list: tokens, and their weight in two words of 15
// bits and the rest.  Up to seven digits (a key's and an index's) lie over the
// histograms of the row.
constexpr uint32_t kDigit = 3 * 256;
constexpr int kMostDigits = 7;
static_assert(kMostDigits * kDigit <= 3 * kBins, "layout");

// Where a list's running weight, from the largest value down, reaches
// `target`: the value, the weight before it, its tokens and their weight.
struct Place {
    uint32_t value, count;
    unsigned long long before, weight;
    bool reached;
};

// Finds it by digits of eight bits from bit `top` down to bit `low`, among the
// tokens that take part; `hist` is the first of the cleared histograms, and
// moves on.
template <bool MASS, typename Value, typename On>
__device__ __forceinline__ Place by_digits(const Shared &sh, int own, const uint32_t (&weight)[kOwn], Value &&value,
                                           On &&on, int top, int low, unsigned long long target, uint32_t &hist) {
    const int lane = threadIdx.x % 32;
    Place p{0, 0, 0, 0, true};
#pragma unroll 1
    for (int hi = top + 1; hi > low;) {
        const int lo = max(hi - 8, low);
        const uint32_t digits = (1u << (hi - lo)) - 1;
#pragma unroll
        for (int j = 0; j < kOwn; ++j)
            if (j < own && on(j)) {
                const uint32_t v = value(j);
                if (hi > top || v >> hi == p.value >> hi) {
                    const uint32_t at = hist + (v >> lo & digits);
                    sh.add_only(at, 1);
                    if (MASS) {
                        sh.add_only(at + 256, weight[j] & 0x7fffu);
                        sh.add_only(at + 512, weight[j] >> 15);
                    }
                }
            }
        __syncthreads();
        if (threadIdx.x < 32) {
            uint32_t c[8];
            unsigned long long w[8], sum = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t at = hist + 255 - (lane * 8 + i);
                c[i] = sh.get(at);
                w[i] = MASS ? sh.get(at + 256) + ((unsigned long long)sh.get(at + 512) << 15) : c[i];
                sum += w[i];
            }
            unsigned long long run = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const unsigned long long v = __shfl_up_sync(0xffffffffu, run, o);
                if (lane >= o) run += v;
            }
            const bool none = p.before + __shfl_sync(0xffffffffu, run, 31) < target;
            if (none && lane == 0) sh.put(kFoundBin, 0xffffffffu);
            run += p.before - sum;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (run < target && run + w[i] >= target) {
                    sh.put(kFoundBin, 255 - (lane * 8 + i));
                    sh.put(kFoundMassLo, (uint32_t)run);
                    sh.put(kFoundMassHi, (uint32_t)(run >> 32));
                    sh.put(kFoundN, c[i]);
                    sh.put(kFoundWLo, (uint32_t)w[i]);
                    sh.put(kFoundWHi, (uint32_t)(w[i] >> 32));
                }
                run += w[i];
            }
        }
        __syncthreads();
        const uint32_t digit = sh.get(kFoundBin);
        if (digit == 0xffffffffu) {
            p.reached = false;
            break;
        }
        p.value |= digit << lo;
        p.before = join64(sh.get(kFoundMassLo), sh.get(kFoundMassHi));
        p.count = sh.get(kFoundN);
        p.weight = join64(sh.get(kFoundWLo), sh.get(kFoundWHi));
        hist += kDigit;
        hi = lo;
        __syncthreads();
    }
    return p;
}

// The cut in a list: the first token, in the order (l descending, index
// ascending), at which the running weight reaches a target (1 or more), and
// with it all before; the last token if the weights do not reach it.  LOW: the
// key's bits below it say nothing (16-bit logits).  A token's weight is one,
// or (MASS) its e in units of 2^-30 of the largest of the list; target_of(all,
// unit) is in those too, given (with SUM) the sum of all and the unit.
template <bool MASS, bool SUM, int LOW, typename Mass, typename Target>
__device__ __forceinline__ Cut cut_near(const Shared &sh, const Near &near, Mass &&mass, Target &&target_of,
                                        int64_t V) {
    __syncthreads();
    for (int i = threadIdx.x; i < kMostDigits * (int)kDigit; i += kThreads) sh.put(kCount + i, 0);
    // the largest and the least key: their common high bits need no digits
    if (threadIdx.x == 0) {
        sh.put(kRed, 0);
        sh.put(kRed + 1, 0xffffffffu);
        sh.put(kRed + 2, 0);
        sh.put(kRed + 3, 0);
    }
    __syncthreads();
    uint32_t most = 0, least = 0xffffffffu;
#pragma unroll
    for (int j = 0; j < kOwn; ++j)
        if (j < near.own && near.key[j]) {
            most = max(most, near.key[j]);
            least = min(least, near.key[j]);
        }
    most = __reduce_max_sync(0xffffffffu, most);
    least = __reduce_min_sync(0xffffffffu, least);
    if (threadIdx.x % 32 == 0) {
        sh.max_only(kRed, most);
        sh.min_only(kRed + 1, least);
    }
    __syncthreads();
    most = sh.get(kRed);
    least = sh.get(kRed + 1);
    uint32_t weight[kOwn];
    const float largest = MASS ? fmaxf(mass(from_order_bits(most)), FLT_MIN) : 1.f;
#pragma unroll
    for (int j = 0; j < kOwn; ++j)
        weight[j] = !MASS ? 1
                    : j < near.own && near.key[j]
                        ? __float2uint_rn(mass(from_order_bits(near.key[j])) / largest * 0x1p30f)
                        : 0;
    unsigned long long all = 0;
    if constexpr (SUM) {
#pragma unroll
        for (int j = 0; j < kOwn; ++j)
            if (j < near.own) all += weight[j];
        const uint32_t lo = __reduce_add_sync(0xffffffffu, (uint32_t)all & 0x7fffu);
        const uint32_t hi = __reduce_add_sync(0xffffffffu, (uint32_t)(all >> 15));
        if (threadIdx.x % 32 == 0) {
            sh.add_only(kRed + 2, lo);
            sh.add_only(kRed + 3, hi);
        }
        __syncthreads();
        all = sh.get(kRed + 2) + ((unsigned long long)sh.get(kRed + 3) << 15);
    }
    const unsigned long long target = target_of(all, 0x1p30 / (double)largest);
    uint32_t hist = kCount;
    const int top = max(LOW, 31 - __clz(most ^ least | 1));
    const uint32_t low_bits = top == 31 ? 0xffffffffu : (2u << top) - 1;
    const Place p = by_digits<MASS>(
        sh, near.own, weight, [&](int j) { return near.key[j] & low_bits; }, [&](int j) { return near.key[j] != 0; },
        top, LOW, target, hist);
    if (!p.reached) return Cut{from_order_bits(least), 0xffffffffu};
    const uint32_t key = (most & ~low_bits) | p.value;
    // 16-bit logits have equal low bits of the key: ones below 0
    const float l = from_order_bits(LOW > 0 && key >> 31 == 0 ? key | ((1u << LOW) - 1) : key);
    if (p.count == 1 || p.before + p.weight <= target) return Cut{l, 0xffffffffu};
    // among equal logits: the index, from the lowest up
    const int bits = 31 - __clz((uint32_t)V);
    const uint32_t all_ones = (2u << bits) - 1;
    const Place q = by_digits<MASS>(
        sh, near.own, weight, [&](int j) { return all_ones - near.idx[j]; },
        [&](int j) { return near.key[j] && near.key[j] >> LOW == key >> LOW; }, bits, 0, target - p.before, hist);
    return Cut{l, q.reached ? all_ones - q.value + 1 : 0xffffffffu};
}

// The cut at which the running count of tokens reaches `k`, or the running
// mass `target`, by a histogram of counts over bins of width 1/scale about the
// multiples of that below `mx`, and a list of the bin (of the bracket) that
// holds it; `width` is a bin's in units of log(e).  ALL: every token of
// logit `low` or more takes part, and the bins cover all of those; else those
// of which `in(l, idx)` holds, the last bin taking what lies below.  False:
// the list does not fit, or does not hold the cut.
template <bool MASS, bool ALL, bool CACHED, int LOW, typename RowT, typename In, typename Mass, typename Mass2,
          typename Prefetch>
__device__ __forceinline__ bool cut_by_list(const RowT &row, const Shared &sh, int rank, Cut &cut, uint32_t k,
                                            double target, float mx, float scale, float width, float low, int64_t V,
                                            In &&in, Mass &&mass, Mass2 &&mass2,
                                            Prefetch &&prefetch) {
    constexpr bool PIECES = ALL && CACHED;
    // 0 is the top bin: the distance from mx in bins, rounded by the sum with
    // 2^23, whose low bits it then is (above all bins for -inf)
    constexpr float kMagic = 0x1p23f;
    auto bin_of = [&](float l) { return __float_as_uint(fmaf(mx - l, scale, kMagic)) - 0x4b000000u; };
    auto clamped = [&](float l) { return min((uint32_t)kCountBins - 1, bin_of(l)); };
    auto in_bins = [&](float2 w) {
        return ffma2(__fadd2_rn(w, make_float2(-mx, -mx)), make_float2(-scale, -scale), make_float2(kMagic, kMagic));
    };
    __syncthreads();
    for (int i = threadIdx.x; i < kCountBins; i += kThreads) sh.put(kCount + i, 0);
    if (threadIdx.x == 0) {
        sh.put(kFoundBin, kCountBins - 1);
        sh.put(kFoundLast, kCountBins - 1);
        sh.put(kTightBin, kCountBins - 1);
        sh.put(kTightLast, kCountBins - 1);
        sh.put(kFoundCount, 0);
        sh.put(kListN, 0);
        sh.put(kNearN, 0);
    }
    __syncthreads();
    if constexpr (PIECES) {
        row.each_piece(low, [&](const auto &v, int) {
#pragma unroll
            for (const float2 &w : v) {
                const float2 m = in_bins(w);
                const uint32_t bx = __float_as_uint(m.x) - 0x4b000000u, by = __float_as_uint(m.y) - 0x4b000000u;
                if (bx < kCountBins) sh.add_only(kCount + bx, 1u);
                if (by < kCountBins) sh.add_only(kCount + by, 1u);
            }
        });
    } else {
        row.each(low, [&](float l, uint32_t idx) {
            if (in(l, idx)) sh.add_only(kCount + clamped(l), 1u);
        });
    }
    sh.sync();
    if (sh.cs > 1) {
        merge_bins(sh, kCount, kCountBins, rank);
        sh.sync();
    }
    // running sums over the bins: of tokens, or of an upper bound on their mass
    // (a token's e is at most that at its bin's upper edge, and at least that
    // times exp(-width): the true sum lies between the bound and that share)
    constexpr int PB = kCountBins / kThreads;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    float part[PB], sum = 0.f;
#pragma unroll
    for (int j = 0; j < PB; ++j) {
        const int bin = threadIdx.x * PB + j;
        part[j] = (float)sh.get(kCount + bin);
        if (MASS) part[j] *= ex2(-1.44269504088896341f * width * ((float)bin - 0.5f));
        sum += part[j];
    }
    float incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const float v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) sh.putf(kRed + warp, incl);
    __syncthreads();
    // (a thread's last bin ends at the very value from which the next thread
    // goes on, so that no value lies between two bins)
    float run = 0.f;
    for (int i = 0; i < warp; ++i) run += sh.getf(kRed + i);
    const float end = run + incl, before = __shfl_up_sync(0xffffffffu, incl, 1);
    if (lane > 0) run += before;
    // counts are exact in f32 up to 2^24; masses have room for the roundings
    const float first = MASS ? (float)target * 0.9999f : (float)k;
    const float last = MASS ? (float)target * 1.0001f * expf(width) : (float)k;
    // mid-bin masses are a good guess, within a sixth of a bin's width but for
    // rows whose mass lies in a few tokens: a bracket of about a third of a bin's
    // width of mass, instead of one of a whole, with the certain one behind it
    const float middle = MASS ? (float)target * expf(0.5f * width) : 0.f;
    const float first_tight = middle * (1.f - width / 6.f), last_tight = middle * (1.f + width / 6.f);
#pragma unroll
    for (int j = 0; j < PB; ++j) {
        const int bin = threadIdx.x * PB + j;
        const float next = j + 1 < PB ? run + part[j] : end;
        // (rounded masses may pass a value twice: the first bin counts)
        if (run < first && next >= first) {
            sh.min_only(kFoundBin, bin);
            if (!MASS) sh.put(kFoundCount, (uint32_t)run);
        }
        if (run < last && next >= last) sh.min_only(kFoundLast, bin);
        if (MASS && run < first_tight && next >= first_tight) sh.min_only(kTightBin, bin);
        if (MASS && run < last_tight && next >= last_tight) sh.min_only(kTightLast, bin);
        run = next;
    }
    __syncthreads();
    const uint32_t above_count = sh.get(kFoundCount);
    int total;
    for (bool tight = MASS;; tight = false) {
        const uint32_t b0 = sh.get(tight ? kTightBin : kFoundBin), b1 = sh.get(tight ? kTightLast : kFoundLast);
        float above = 0.f, inside = 0.f;  // masses
        if constexpr (PIECES) {
            const float f0 = kMagic + (float)b0, f1 = kMagic + (float)b1;
            float2 sum2 = make_float2(0.f, 0.f);
            row.each_piece(low, [&](const auto &v, int i0) {
                constexpr int VE = sizeof(v) / sizeof(float);
                uint32_t on = 0;      // bits of the tokens in the bracket
                bool ahead = false;   // one is above it
#pragma unroll
                for (int e = 0; e < VE; e += 2) {
                    const float2 m = in_bins(v[e / 2]);
                    if (MASS) {
                        const float2 x = mass2(v[e / 2]);
                        sum2 = __fadd2_rn(sum2, make_float2(m.x < f0 ? x.x : 0.f, m.y < f0 ? x.y : 0.f));
                    }
                    ahead = ahead || m.x < f0 || m.y < f0;
                    on |= (m.x >= f0 && m.x <= f1 ? 1u << e : 0) | (m.y >= f0 && m.y <= f1 ? 2u << e : 0);
                }
                if (ahead) prefetch(i0);
                while (on) {
                    const int e = __ffs(on) - 1;
                    on &= on - 1;
                    const float l = row.at(i0 + e);
                    enlist(sh, l, row.base + (uint32_t)(i0 + e));
                    if (MASS) inside += mass(l);
                }
            });
            above = sum2.x + sum2.y;
        } else {
            row.each(low, [&](float l, uint32_t idx) {
                const uint32_t bin = clamped(l);
                if (bin > b1 || !in(l, idx)) return;
                if (bin >= b0) enlist(sh, l, idx);
                if (MASS) (bin >= b0 ? inside : above) += mass(l);
            });
        }
        if (MASS) {
            above = block_sum(above, sh);
            inside = block_sum(inside, sh);
            if (threadIdx.x == 0) {
                sh.putf(kPartAbove, above);
                sh.putf(kPartIn, inside);
            }
        }
        send_list(sh);
        sh.sync();
        total = listed(sh);
        if (total < 0) return false;
        if (!MASS) break;
        const float all_above = sh.sum_ctas(kPartAbove);
        if (all_above < (float)target && all_above + sh.sum_ctas(kPartIn) >= (float)target) break;
        if (!tight) return false;  // (a target within roundings of the whole mass)
        sh.sync();
        if (threadIdx.x == 0) {
            sh.put(kListN, 0);
            sh.put(kNearN, 0);
        }
        sh.sync();
    }
    if (rank == 0) {
        Cut c = no_cut();
        if (total > 0) {
            Near near;
            near.load(sh, total);
            const double left = MASS ? target - (double)sh.sum_ctas(kPartAbove) : 0.0;
            c = cut_near<MASS, false, LOW>(
                sh, near, mass,
                [&](unsigned long long, double unit) -> unsigned long long {
                    if (!MASS) return k - above_count;
                    return left * unit > 1 ? __double2ull_ru(left * unit) : 1;
                },
                V);
        }
        if ((int)threadIdx.x < sh.cs) {
            sh.put(kCutL, (int)threadIdx.x, __float_as_uint(c.l));
            sh.put(kCutEnd, (int)threadIdx.x, c.end);
        }
    }
    sh.sync();
    cut.l = sh.getf(kCutL);
    cut.end = sh.get(kCutEnd);
    return true;
}

template <typename T, bool CACHED>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleArgs a, const int cs, const int64_t slice) {
    constexpr int VE = 16 / sizeof(T);
    constexpr int ROUNDS = sizeof(T) == 2 ? 2 : 3;
    constexpr int LOW = sizeof(T) == 2 ? 13 : 0;  // bits of a key that say nothing
    extern __shared__ __align__(16) unsigned char smem_raw[];
    const Shared sh{static_cast<uint32_t>(__cvta_generic_to_shared(smem_raw)), cs};
    pdl_trigger();
    pdl_wait();
    const int64_t r = blockIdx.x / cs;
    const int rank = blockIdx.x % cs;
    const int64_t base = rank * slice;
    const int n = (int)(a.V - base < slice ? (a.V > base ? a.V - base : 0) : slice);
    const T *src = static_cast<const T *>(a.logits) + r * a.logits_st + base;
    const float *noise = a.noise + r * a.noise_st;

    // the row's settings; a temperature below 2^-100 acts as that
    float temp = a.temperature ? a.temperature[r] : a.temperature_v;
    const float top_p = a.top_p ? a.top_p[r] : a.top_p_v;
    const float min_p = a.min_p ? a.min_p[r] : a.min_p_v;
    const int32_t top_k = a.top_k ? a.top_k[r] : a.top_k_v;
    const bool only_first = !(temp > 0.f) || top_p <= 0.f || min_p > 1.f || top_k == 1;
    temp = temp > 0.f ? fminf(fmaxf(temp, 0x1p-100f), FLT_MAX) : 1.f;
    const bool use_k = !only_first && top_k > 0 && top_k < a.V;
    const bool use_p = !only_first && top_p < 1.f;
    const bool use_m = !only_first && min_p > 0.f;
    const float to_log2 = 1.44269504088896341f / temp;
    auto e_below = [&](float l, float top) { return ex2((l - top) * to_log2); };

    if (!only_first && !use_k && !use_p && !use_m) {
        // all of the noise will be wanted: on its way to L2 with the logits
        const float *nb = noise + base;
        for (int i = (int)threadIdx.x * 32; i < n; i += kThreads * 32)
            asm volatile("prefetch.global.L2 [%0];\n" ::"l"(nb + i));
    }

    // the slice into shared memory, with each thread's maximum and mass
    Row<T, CACHED> row;
    row.n = n;
    row.base = (uint32_t)base;
    row.mis = CACHED ? (int)(reinterpret_cast<uintptr_t>(src) / sizeof(T) % VE) : 0;
    float my_max = -INFINITY, my_z = 0.f;
    auto take = [&](const uint4 &w) {
        const float top = piece_max<T>(w);
        if (top > my_max) {
            my_z *= e_below(my_max, top);
            my_max = top;
        }
        if (top == -INFINITY) return;
        RawPiece<T, VE> raw;
        raw.w = w;
        float v[VE];
        widen<T, VE>(v, raw);
        const float2 m2 = make_float2(-my_max, -my_max), c2 = make_float2(to_log2, to_log2);
#pragma unroll
        for (int e = 0; e < VE; e += 2) {
            const float2 d = fmul2(__fadd2_rn(make_float2(v[e], v[e + 1]), m2), c2);
            my_z += ex2(d.x) + ex2(d.y);
        }
    };
    row.src = src;
    row.pieces = sh.base + kSharedBytes;
    if constexpr (CACHED) {
        // the pieces that lie inside the slice, then those across its ends, with
        // -inf beside it
        const int first = row.mis > 0, end = (row.mis + n) / VE, all = row.count();
        const T *at = src - row.mis;
        constexpr int AHEAD = 4;  // pieces of a thread in flight
        for (int j = first + (int)threadIdx.x; j < end; j += AHEAD * kThreads) {
            RawPiece<T, VE> raw[AHEAD];
#pragma unroll
            for (int u = 0; u < AHEAD; ++u)
                if (j + u * kThreads < end) raw[u].w = row_piece(at + (int64_t)(j + u * kThreads) * VE);
#pragma unroll
            for (int u = 0; u < AHEAD; ++u)
                if (j + u * kThreads < end) {
                    const uint4 w = clean(raw[u]);
                    put_piece(row.pieces + 16 * (j + u * kThreads), w);
                    take(w);
                }
        }
        // (one thread per end; a slice within one piece has one)
        const bool head = threadIdx.x == 0 && first && all > 0, tail = threadIdx.x == 1 && end < all && end >= first;
        if (head || tail) {
            const int k = head ? 0 : end;
            float v[VE];
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                const int i = k * VE + e - row.mis;
                v[e] = i >= 0 && i < n ? Elem<T>::to_f32(src[i]) : -INFINITY;
            }
            const uint4 w = clean(narrow_piece<T, VE>(v));
            put_piece(row.pieces + 16 * k, w);
            take(w);
        }
        __syncthreads();
    } else {
        for (int i0 = (int)threadIdx.x * VE; i0 < n; i0 += kThreads * VE) {
            float top = -INFINITY;
#pragma unroll
            for (int e = 0; e < VE; ++e)
                if (i0 + e < n) top = fmaxf(top, logit(src[i0 + e]));
            if (top > my_max) {
                my_z *= e_below(my_max, top);
                my_max = top;
            }
            if (top > -INFINITY)
#pragma unroll
                for (int e = 0; e < VE; ++e)
                    if (i0 + e < n) my_z += e_below(logit(src[i0 + e]), my_max);
        }
    }
    // the row's maximum and mass: warps, then warps of the CTA, then CTAs, each
    // in a fixed order
    float mx = my_max, z = my_z;
    auto join = [&](float om, float oz) {
        const float top = fmaxf(mx, om);
        if (top > -INFINITY) z = z * e_below(mx, top) + oz * e_below(om, top);
        mx = top;
    };
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float om = __shfl_xor_sync(0xffffffffu, mx, o), oz = __shfl_xor_sync(0xffffffffu, z, o);
        join(om, oz);
    }
    if (threadIdx.x % 32 == 0) {
        sh.putf(kRed + threadIdx.x / 32, mx);
        sh.putf(kRed2 + threadIdx.x / 32, z);
    }
    if (threadIdx.x == 0) {
        sh.putf(kRace, 0.f);
        sh.put(kListN, 0);
        sh.put(kNearN, 0);
    }
    __syncthreads();
    mx = sh.getf(kRed + threadIdx.x % kWarps);
    z = sh.getf(kRed2 + threadIdx.x % kWarps);
#pragma unroll
    for (int o = kWarps / 2; o > 0; o >>= 1) {
        const float om = __shfl_xor_sync(0xffffffffu, mx, o), oz = __shfl_xor_sync(0xffffffffu, z, o);
        join(om, oz);
    }
    z = __shfl_sync(0xffffffffu, z, 0);  // (the lanes' sums may differ in their last bit)
    if (cs > 1) {
        if (threadIdx.x == 0) {
            sh.putf(kPartMax, mx);
            sh.putf(kPartZ, z);
        }
        sh.sync();
        const float om = __uint_as_float(sh.each_cta(kPartMax, __float_as_uint(-INFINITY)));
        const float oz = __uint_as_float(sh.each_cta(kPartZ, 0));
        mx = __shfl_sync(0xffffffffu, om, 0);
        z = __shfl_sync(0xffffffffu, oz, 0);
        for (int q = 1; q < cs; ++q) join(__shfl_sync(0xffffffffu, om, q), __shfl_sync(0xffffffffu, oz, q));
    }

    auto finish = [&](uint32_t token) {
        a.token[r] = (int32_t)token;
        if (a.logprob) {
            const float l = logit(static_cast<const T *>(a.logits)[r * a.logits_st + token]);
            a.logprob[r] = (l - mx) / temp - logf(z);
        }
    };
    if (mx == -INFINITY) {  // nothing is left in this row
        if (rank == 0 && threadIdx.x == 0) {
            a.token[r] = -1;
            if (a.logprob) a.logprob[r] = -INFINITY;
        }
        sh.sync();  // no CTA leaves while another reads its words
        return;
    }
    auto fast_e = [&](float l) { return e_below(l, mx); };
    auto fast_e2 = [&](float2 l) {
        const float2 d = fmul2(__fadd2_rn(l, make_float2(-mx, -mx)), make_float2(to_log2, to_log2));
        return make_float2(ex2(d.x), ex2(d.y));
    };
    auto exact_e = [&](float l) { return expf((l - mx) / temp); };
    auto over_min = [&](float l) {
        const float e = fast_e(l);
        if (fabsf(e - min_p) <= 1e-4f * min_p) return exact_e(l) >= min_p;
        return e >= min_p;
    };
    // The race.  A key is worked out in full only where the rough one, which is
    // within a ten-thousandth, may be the best.
    constexpr float kNearly = 0.9998f;
    float best = -1.f;
    uint32_t best_i = 0xffffffffu;
    auto rough = [&](float e, float nz) { return e * rcpf(fmaxf(nz, FLT_MIN)); };
    auto run = [&](float l, uint32_t idx, float nz) {
        const float key = exact_e(l) / fmaxf(nz, FLT_MIN);
        if (l > -INFINITY && (key > best || (key == best && idx < best_i))) {
            if (key > best) sh.max_only(kRace, __float_as_uint(key));
            best = key;
            best_i = idx;
        }
    };
    // a batch of tokens, all lanes of a warp together; those of rough key -1 do
    // not take part
    auto batch = [&](const auto &key, auto &&token) {
        constexpr int U = sizeof(key) / sizeof(float);
        float most = key[0];
#pragma unroll
        for (int u = 1; u < U; ++u) most = fmaxf(most, key[u]);
        const float ahead = kNearly * sh.getf(kRace);
        if (!__any_sync(0xffffffffu, most >= ahead)) return;
        const uint32_t of_warp = __reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(most, 0.f)));
        const float least = fmaxf(ahead, kNearly * __uint_as_float(of_warp));
        if (most >= least)
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (key[u] >= least) token(u);
    };
    // this CTA's winner, as (key, ~index), in every thread
    auto winner = [&]() {
        uint32_t k = best < 0.f ? 0 : __float_as_uint(best), i = best < 0.f ? 0xffffffffu : best_i;
        auto warp_best = [&]() {
            const uint32_t top = __reduce_max_sync(0xffffffffu, k);
            i = __reduce_min_sync(0xffffffffu, k == top ? i : 0xffffffffu);
            k = top;
        };
        warp_best();
        __syncthreads();
        if (threadIdx.x % 32 == 0) {
            sh.put(kRed + threadIdx.x / 32, k);
            sh.put(kRed2 + threadIdx.x / 32, i);
        }
        __syncthreads();
        k = sh.get(kRed + threadIdx.x % kWarps);
        i = sh.get(kRed2 + threadIdx.x % kWarps);
        warp_best();
        return join64(0xffffffffu - i, k);
    };

    Cut cut = no_cut();
    if (use_k && top_k <= kMaxK) {
        // at least k tokens of a slice reach the k-th largest of its threads'
        // maxima, so it lets all pass that can be among the first k
        const uint32_t mine = order_bits(my_max);
        uint32_t floor_ = 0;
#pragma unroll 1
        for (int bit = 31; bit >= (sizeof(T) == 2 ? 13 : 0); --bit) {
            const uint32_t t = floor_ | (1u << bit);
            if (__syncthreads_count(mine >= t) >= top_k) floor_ = t;
        }
        const float low = floor_ > order_bits(-FLT_MAX) ? from_order_bits(floor_) : -FLT_MAX;
        row.each(low, [&](float l, uint32_t idx) { enlist(sh, l, idx); });
        send_list(sh);
        sh.sync();
        const int total = listed(sh);
        if (total >= 0) {
            if (rank == 0) {
                Near near;
                near.load(sh, total);
                cut = cut_near<false, false, LOW>(
                    sh, near, fast_e, [&](unsigned long long, double) { return (unsigned long long)top_k; }, a.V);
                if (use_p) {
#pragma unroll
                    for (int j = 0; j < kOwn; ++j)
                        if (near.key[j] && !cut.keeps(from_order_bits(near.key[j]), near.idx[j])) near.key[j] = 0;
                    cut = cut_near<true, true, LOW>(
                        sh, near, fast_e,
                        [&](unsigned long long all, double) { return __double2ull_ru((double)top_p * (double)all); }, a.V);
                }
#pragma unroll
                for (int j = 0; j < kOwn; ++j) {
                    const float l = from_order_bits(near.key[j]);
                    if (near.key[j] && cut.keeps(l, near.idx[j]) && (!use_m || l == mx || over_min(l)))
                        run(l, near.idx[j], noise_at(noise + near.idx[j]));
                }
                const unsigned long long w = winner();
                if (threadIdx.x == 0) finish(0xffffffffu - (uint32_t)w);
            }
            sh.leave(rank);  // the first CTA stays while another reads its words
            return;
        }
        cut = narrow<false, ROUNDS>(row, sh, rank, cut, (uint32_t)top_k, 0.0, -FLT_MAX,
                              [](float, uint32_t) { return true; }, fast_e);
    } else if (use_k) {
        // bins from the largest logit to past the least of the threads' maxima
        float least = my_max;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) least = fminf(least, __shfl_xor_sync(0xffffffffu, least, o));
        __syncthreads();
        if (threadIdx.x % 32 == 0) sh.putf(kRed + threadIdx.x / 32, least);
        __syncthreads();
        for (int i = 0; i < kWarps; ++i) least = fminf(least, sh.getf(kRed + i));
        if (cs > 1) {
            if (threadIdx.x == 0) sh.putf(kPartLeast, least);
            sh.sync();
            least = __uint_as_float(sh.each_cta(kPartLeast, __float_as_uint(INFINITY)));
#pragma unroll
            for (int o = 4; o > 0; o >>= 1) least = fminf(least, __shfl_xor_sync(0xffffffffu, least, o));
            least = __shfl_sync(0xffffffffu, least, 0);
        }
        const float range = least > -INFINITY ? fmaxf(1.5f * (mx - least), 1e-20f) : 16.f * temp;
        if (!cut_by_list<false, false, CACHED, LOW>(row, sh, rank, cut, (uint32_t)top_k, 0.0, mx, fminf(kCountBins / range, 1e30f), 0.f,
                                -FLT_MAX, a.V, [](float, uint32_t) { return true; }, fast_e, fast_e2, [](int) {}))
            cut = narrow<false, ROUNDS>(row, sh, rank, cut, (uint32_t)top_k, 0.0, -FLT_MAX,
                                  [](float, uint32_t) { return true; }, fast_e);
    }
    if (use_p) {
        float zk = z;
        if (use_k) {
            zk = 0.f;
            row.each(cut.l, [&](float l, uint32_t idx) {
                if (cut.keeps(l, idx)) zk += fast_e(l);
            });
            zk = block_sum(zk, sh);
            if (cs > 1) {
                if (threadIdx.x == 0) sh.putf(kPartSum, zk);
                sh.sync();
                zk = sh.sum_ctas(kPartSum);
            }
        }
        // tokens of less than this e lie past the cut whatever their order: all
        // of them together hold less than 1 - top_p of the mass
        const float least = 0.5f * (1.f - top_p) * zk / (float)a.V;
        const float range = fmaxf(-logf(least), 1.f);
        const float low = fmaxf(mx - 1.0001f * range * temp, cut.l);
        const Cut k_cut = cut;
        auto in = [&](float l, uint32_t idx) { return k_cut.keeps(l, idx); };
        const float scale = kCountBins / (range * temp);
        bool done = false;
        if (scale < 1e30f) {
            const float width = range / kCountBins;
            const double target = (double)top_p * zk;
            // the noise of what is above the bracket will be wanted
            auto prefetch = [&](int i0) {
                asm volatile("prefetch.global.L2 [%0];\n" ::"l"(noise + base + max(i0, 0)));
            };
            done = use_k ? cut_by_list<true, false, CACHED, LOW>(row, sh, rank, cut, 0, target, mx, scale, width, low,
                                                                 a.V, in, fast_e, fast_e2, prefetch)
                         : cut_by_list<true, true, CACHED, LOW>(row, sh, rank, cut, 0, target, mx, scale, width, low,
                                                                a.V, in, fast_e, fast_e2, prefetch);
        }
        if (!done)
            cut = narrow<true, ROUNDS>(row, sh, rank, cut, 0, (double)top_p * zk * 0x1p40, low, in, fast_e);
        // the cuts above are exact among the tokens that top-k left, and may end
        // past the last of them: what top-k removed stays out
        if (cut.l < k_cut.l) cut = k_cut;
        else if (cut.l == k_cut.l) cut.end = min(cut.end, k_cut.end);
    }

    if (only_first) {
        row.each(mx, [&](float, uint32_t idx) {
            best = 1.f;
            if (idx < best_i) best_i = idx;
        });
    } else if (!use_k && !use_p && !use_m) {
        // neighbouring threads on neighbouring tokens, eight of each in flight
        constexpr int U = 8;
        const float *nb = noise + base;
        for (int i0 = threadIdx.x; i0 - (int)threadIdx.x < n; i0 += U * kThreads) {
            float nz[U], l[U], key[U];
            if (i0 + (U - 1) * kThreads < n) {
#pragma unroll
                for (int u = 0; u < U; ++u) nz[u] = noise_at(nb + i0 + u * kThreads);
#pragma unroll
                for (int u = 0; u < U; ++u) l[u] = row.at(i0 + u * kThreads);
            } else {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const bool in = i0 + u * kThreads < n;
                    nz[u] = in ? noise_at(nb + i0 + u * kThreads) : 1.f;
                    l[u] = in ? row.at(i0 + u * kThreads) : -INFINITY;
                }
            }
#pragma unroll
            for (int u = 0; u < U; u += 2) {
                const float2 e = fast_e2(make_float2(l[u], l[u + 1]));
                key[u] = l[u] > -INFINITY ? rough(e.x, nz[u]) : -1.f;
                key[u + 1] = l[u + 1] > -INFINITY ? rough(e.y, nz[u + 1]) : -1.f;
            }
            batch(key, [&](int u) { run(l[u], (uint32_t)(base + i0 + u * kThreads), nz[u]); });
        }
    } else {
        const float low = use_m ? fmaxf(cut.l, mx + 1.0001f * logf(0.999f * min_p) * temp) : cut.l;
        auto left = [&](float l, uint32_t idx) { return cut.keeps(l, idx) && (!use_m || l == mx || over_min(l)); };
        if constexpr (CACHED) {
            // (a masked token is never left, nor is a place outside the slice: no
            // noise is read for either)
            row.each_piece_warp(low, [&](const auto &v, int i0) {
                float nz[VE], key[VE];
                const float *np = noise + base + i0;
                const uint32_t idx = row.base + (uint32_t)i0;
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    const bool on = left(e % 2 ? v[e / 2].y : v[e / 2].x, idx + e);
                    nz[e] = on ? noise_at(np + e) : 1.f;
                    key[e] = on ? 0.f : -1.f;
                }
#pragma unroll
                for (int e = 0; e < VE; e += 2) {
                    const float2 x = fast_e2(v[e / 2]);
                    if (key[e] == 0.f) key[e] = rough(x.x, nz[e]);
                    if (key[e + 1] == 0.f) key[e + 1] = rough(x.y, nz[e + 1]);
                }
                batch(key, [&](int e) { run(e % 2 ? v[e / 2].y : v[e / 2].x, idx + e, nz[e]); });
            });
        } else {
            row.each(low, [&](float l, uint32_t idx) {
                if (left(l, idx)) run(l, idx, noise_at(noise + idx));
            });
        }
    }
    unsigned long long w = winner();
    if (cs > 1) {
        // each CTA's into the first one's memory
        if (threadIdx.x == 0) {
            sh.put(kNearKey + rank, 0, (uint32_t)(w >> 32));
            sh.put(kNearIdx + rank, 0, (uint32_t)w);
        }
        sh.sync();
        if (rank == 0 && threadIdx.x < 32) {
            const int q = threadIdx.x < cs ? threadIdx.x : 0;
            w = join64(sh.get(kNearIdx + q), sh.get(kNearKey + q));
#pragma unroll
            for (int o = 4; o > 0; o >>= 1) {
                const unsigned long long p = __shfl_xor_sync(0xffffffffu, w, o);
                if (p > w) w = p;
            }
        }
    }
    if (rank == 0 && threadIdx.x == 0) finish(0xffffffffu - (uint32_t)w);
}

constexpr size_t kMostShared = 200 * 1024;
constexpr size_t kTwoPerSm = 112 * 1024;

template <typename T, bool CACHED>
cudaError_t launch_cs(const SampleArgs &a, int cs, int64_t slice, size_t smem, cudaStream_t s) {
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(sample_kernel<T, CACHED>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   (int)kMostShared);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.R * cs));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)cs;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, sample_kernel<T, CACHED>, a, cs, slice);
}

template <typename T>
cudaError_t launch_t(const SampleArgs &a, int sm_count, cudaStream_t s) {
    constexpr int VE = 16 / sizeof(T);
    const int64_t sms = sm_count > 0 ? sm_count : 152;
    auto slice_of = [&](int cs) { return ((a.V + cs - 1) / cs + VE - 1) / VE * VE; };
    auto bytes_of = [&](int cs) { return kSharedBytes + (size_t)(slice_of(cs) + VE) * sizeof(T); };
    // A row over as few CTAs as leave room for two of them on an SM, so that
    // one loads while another computes; over more while SMs would stay idle.
    // 128 x 131072 bf16 with the three cuts over slices of up to 112 KB: 79 us;
    // 200 KB: 98 us, 60 KB: 94 us; 256 x 100003 uncut 58, 75 and 79 us.  One row
    // of 32000 f32 with top-p over slices down to 4096: 19.3 us, to 16384:
    // 25.3 us, to 2048: no change.
    int cs = 1;
    while (cs < kMaxCluster && bytes_of(cs) > kTwoPerSm) cs *= 2;
    while (cs < kMaxCluster && a.R * cs * 2 <= sms && slice_of(cs) > 4096) cs *= 2;
    if (a.R * cs > INT32_MAX) return cudaErrorInvalidConfiguration;
    if (bytes_of(cs) > kMostShared)
        return launch_cs<T, false>(a, cs, slice_of(cs), kSharedBytes, s);
    return launch_cs<T, true>(a, cs, slice_of(cs), bytes_of(cs), s);
}

}  // namespace

cudaError_t launch_sample(DType dt, const SampleArgs &a, int sm_count, cudaStream_t s) {
    switch (dt) {
    case DType::F32: return launch_t<float>(a, sm_count, s);
    case DType::BF16: return launch_t<__nv_bfloat16>(a, sm_count, s);
    case DType::F16: return launch_t<__half>(a, sm_count, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace gdn
