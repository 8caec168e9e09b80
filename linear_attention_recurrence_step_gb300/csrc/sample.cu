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
// So no sort is needed: a cut is a threshold on the logit's ordered bits plus
// an index limit among equal logits.  A first histogram has bins of equal
// width in the logit, which spreads the tokens evenly; the tokens of the bin
// that holds the cut then go into a short list (or, if they do not fit,
// stay where they are) and histograms over 11 bits of the ordered key at a
// time (two for 16-bit logits, three for f32) find the exact value.  Where
// top-k is at most the threads of a CTA, the k-th largest of the threads' own
// maxima bounds the cut from below and replaces the first histogram.  Masses
// are summed as integers (units of 2^-40 of the largest token's), so the
// order of the shared-memory atomics does not change any result.
//
// A row is read from memory once, with its maximum and its mass taken on the
// way: a cluster of CTAs holds its slices in shared memory and goes over them
// there; the noise is read only for tokens that are left.
#include <cfloat>
#include <cooperative_groups.h>

#include "layer.h"
#include "pieces.cuh"

namespace gdn {

namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kMaxCluster = 8;
constexpr int kList = 1024;     // tokens of a cut's bin that a CTA lists

struct SampleShared {
    uint32_t count[kBins], lo[kBins], hi[kBins];   // histogram: tokens, mass (64 bits in two words)
    uint2 list[kList];                             // (key, index) of tokens near a cut
    uint32_t list_n;
    float fslot[4];                                // this CTA's part of a cluster-wide value
    uint32_t ties;                                 // this CTA's tokens at the threshold
    unsigned long long best;                       // this CTA's (key, ~index)
    float redf[kWarps], redz[kWarps];
    unsigned long long redm[kWarps];
    uint32_t redc[kWarps];
    unsigned long long found_mass;                 // mass before the bin that holds the cut
    uint32_t found_bin, found_count, found_n;
    unsigned long long found_w;
    uint32_t limit;                                // index limit among equal logits
    float race;                                    // lower bound on the best key so far
};

// The logit as the rules see it: NaN is masked, +inf is the largest finite
// value of its type, -0 is 0.
template <typename T> __device__ __forceinline__ float canonical(float x);
template <> __device__ __forceinline__ float canonical<float>(float x) {
    return fminf(fmaxf(x, -INFINITY), FLT_MAX) + 0.f;
}
template <> __device__ __forceinline__ float canonical<__nv_bfloat16>(float x) {
    return fminf(fmaxf(x, -INFINITY), __uint_as_float(0x7f7f0000u)) + 0.f;
}
template <> __device__ __forceinline__ float canonical<__half>(float x) {
    return fminf(fmaxf(x, -INFINITY), 65504.f) + 0.f;
}
template <typename T> __device__ __forceinline__ float logit(T x) { return canonical<T>(Elem<T>::to_f32(x)); }
__device__ __forceinline__ uint32_t order_bits(float l) {
    const uint32_t u = __float_as_uint(l);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// What is left so far: the key's high bits above `prefix`, or equal to it
// with an index of at most `limit`.
struct Cut {
    uint32_t prefix = 0, limit = 0xffffffffu;
    int shift = 10;
    __device__ __forceinline__ bool keeps(uint32_t key, uint32_t idx) const {
        const uint32_t p = key >> shift;
        return p > prefix || (p == prefix && idx <= limit);
    }
};

template <typename T, bool CACHED> struct Row {
    const T *buf;        // shared memory (CACHED) or the row's slice in memory
    int mis;             // buf[mis] is the slice's first token when CACHED
    int64_t n;           // tokens in the slice
    uint32_t base;       // index of the first
    // f(logit, index) for every token of the slice, thread by thread; pieces
    // in shared memory hold logits as logit() gives them, and -inf around the
    // slice
    template <typename F> __device__ __forceinline__ void each(F &&f) const {
        if constexpr (CACHED) {
            constexpr int VE = 16 / sizeof(T);
            const int nvec = (int)((mis + n + VE - 1) / VE);
            for (int j = threadIdx.x; j < nvec; j += kThreads) {
                float v[VE];
                load_piece<T, VE>(v, buf + (int64_t)j * VE);
#pragma unroll
                for (int e = 0; e < VE; ++e) f(v[e], base + (uint32_t)(j * VE + e - mis));
            }
        } else {
            for (int64_t i = threadIdx.x; i < n; i += kThreads) f(logit(buf[i]), base + (uint32_t)i);
        }
    }
    __device__ __forceinline__ float at(int64_t i) const {
        return CACHED ? Elem<T>::to_f32(buf[mis + i]) : logit(buf[i]);
    }
};

__device__ __forceinline__ float block_sum(float v, SampleShared &sh) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if (threadIdx.x % 32 == 0) sh.redf[threadIdx.x / 32] = v;
    __syncthreads();
    v = 0.f;
    for (int i = 0; i < kWarps; ++i) v += sh.redf[i];
    return v;
}

__device__ __forceinline__ void cluster_sync(int cs) {
    if (cs > 1) cg::this_cluster().sync();
    else __syncthreads();
}
// A value in another CTA's shared memory of the cluster.
template <typename V> __device__ __forceinline__ V *remote(V *p, int rank, int cs) {
    return cs > 1 ? cg::this_cluster().map_shared_rank(p, rank) : p;
}

// The bin, counted from the top, of a histogram (over all CTAs of the cluster)
// in which the running count reaches `k` or the running mass reaches
// `target`; found_bin stays ~0 if none does.  Counts and masses of higher
// bins than any of the histogram are given.
template <bool MASS>
__device__ void find_bin(SampleShared &sh, int cs, int rank, uint32_t above_count, unsigned long long above_mass,
                         uint32_t k, double target) {
    if (cs > 1) {
        // each CTA adds up its share of the bins and hands the sums to all; it
        // alone reads and writes those bins
        cg::this_cluster().sync();
        const int share = kBins / cs;
        for (int i = threadIdx.x; i < share; i += kThreads) {
            const int bin = rank * share + i;
            uint32_t c = 0;
            unsigned long long m = 0;
            for (int q = 0; q < cs; ++q) {
                c += *remote(&sh.count[bin], q, cs);
                if (MASS)
                    m += (unsigned long long)*remote(&sh.lo[bin], q, cs) +
                         ((unsigned long long)*remote(&sh.hi[bin], q, cs) << 32);
            }
            for (int q = 0; q < cs; ++q) {
                *remote(&sh.count[bin], q, cs) = c;
                if (MASS) {
                    *remote(&sh.lo[bin], q, cs) = (uint32_t)m;
                    *remote(&sh.hi[bin], q, cs) = (uint32_t)(m >> 32);
                }
            }
        }
        cg::this_cluster().sync();
    } else {
        __syncthreads();
    }
    // running sums from the top bin: PB bins per thread
    constexpr int PB = kBins / kThreads;
    uint32_t c[PB], ctot = 0;
    unsigned long long m[PB], mtot = 0;
#pragma unroll
    for (int j = 0; j < PB; ++j) {
        const int bin = kBins - 1 - (threadIdx.x * PB + j);
        c[j] = sh.count[bin];
        m[j] = MASS ? (unsigned long long)sh.lo[bin] + ((unsigned long long)sh.hi[bin] << 32) : 0;
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
        sh.redc[warp] = cin;
        sh.redm[warp] = min_;
    }
    __syncthreads();
    uint32_t cbase = above_count + cin - ctot;
    unsigned long long mbase = above_mass + min_ - mtot;
    for (int i = 0; i < warp; ++i) {
        cbase += sh.redc[i];
        mbase += sh.redm[i];
    }
#pragma unroll
    for (int j = 0; j < PB; ++j) {
        const bool before = MASS ? (double)mbase < target : cbase < k;
        const bool reached = MASS ? (double)(mbase + m[j]) >= target : cbase + c[j] >= k;
        if (before && reached) {
            sh.found_bin = kBins - 1 - (threadIdx.x * PB + j);
            sh.found_count = cbase;
            sh.found_mass = mbase;
            sh.found_n = c[j];
            sh.found_w = m[j];
        }
        cbase += c[j];
        mbase += m[j];
    }
    __syncthreads();
}

// Clears the histogram; a barrier follows.
template <bool MASS> __device__ __forceinline__ void clear_bins(SampleShared &sh) {
    for (int i = threadIdx.x; i < kBins; i += kThreads) {
        sh.count[i] = 0;
        if (MASS) sh.lo[i] = sh.hi[i] = 0;
    }
    if (threadIdx.x == 0) sh.found_bin = 0xffffffffu;
    __syncthreads();
}

// e in units of 2^-40 added to a bin's mass.
__device__ __forceinline__ void add_mass(SampleShared &sh, uint32_t bin, float e) {
    uint32_t wh = 0;
    if (e >= 0x1p-8f) {
        wh = __float2uint_rz(e * 0x1p8f);
        e -= (float)wh * 0x1p-8f;
    }
    const uint32_t wl = __float2uint_rz(e * 0x1p40f);
    const uint32_t old = atomicAdd(&sh.lo[bin], wl);
    if (old + wl < old) ++wh;
    if (wh) atomicAdd(&sh.hi[bin], wh);
}

// Narrows `cut` to the tokens before the place where the running count reaches
// `k` (or the running mass reaches `target`), in the order (l descending,
// index ascending), among those of which `in(l, idx)` holds; `mass(l)` is a
// token's e.  scale > 0: a histogram of bins of width 1/scale below `mx` comes
// first.  Without it, the tokens that take part should be few.
template <bool MASS, int ROUNDS, typename RowT, typename In, typename Mass>
__device__ void narrow(const RowT &row, SampleShared &sh, int cs, int rank, Cut &cut, uint32_t k, double target,
                       float mx, float scale, In &&in, Mass &&mass) {
    uint32_t above_count = 0;
    unsigned long long above_mass = 0;
    auto linear = [&](float l) { return kBins - 1 - min(kBins - 1, __float2int_rz((mx - l) * scale)); };
    int lin_bin = -1;
    if (scale > 0.f) {
        clear_bins<MASS>(sh);
        row.each([&](float l, uint32_t idx) {
            if (!in(l, idx)) return;
            const int bin = linear(l);
            if (MASS) add_mass(sh, bin, mass(l));
            else atomicAdd(&sh.count[bin], 1u);
        });
        find_bin<MASS>(sh, cs, rank, 0, 0, k, target);
        if (sh.found_bin == 0xffffffffu) return;  // every token that takes part is left
        lin_bin = (int)sh.found_bin;
        above_count = sh.found_count;
        above_mass = sh.found_mass;
    }
    // the tokens of that bin, listed
    auto near = [&](float l, uint32_t idx) { return (lin_bin < 0 || linear(l) == lin_bin) && in(l, idx); };
    __syncthreads();
    if (threadIdx.x == 0) sh.list_n = 0;
    __syncthreads();
    row.each([&](float l, uint32_t idx) {
        if (!near(l, idx)) return;
        const uint32_t at = atomicAdd(&sh.list_n, 1u);
        if (at < kList) sh.list[at] = make_uint2(__float_as_uint(l), idx);
    });
    __syncthreads();
    const uint32_t listed = sh.list_n;
    const bool in_list = listed <= kList;
    auto visit = [&](auto &&f) {
        if (in_list)
            for (uint32_t i = threadIdx.x; i < listed; i += kThreads) f(__uint_as_float(sh.list[i].x), sh.list[i].y);
        else
            row.each([&](float l, uint32_t idx) {
                if (near(l, idx)) f(l, idx);
            });
    };
    uint32_t prefix = 0;
    int shift = 32;
#pragma unroll 1
    for (int round = 0; round < ROUNDS; ++round) {
        const int bits = round == 2 ? 10 : 11;
        const int next = shift - bits;
        clear_bins<MASS>(sh);
        visit([&](float l, uint32_t) {
            const uint32_t key = order_bits(l);
            if (round > 0 && (key >> shift) != prefix) return;
            const uint32_t bin = (key >> next) & ((1u << bits) - 1);
            atomicAdd(&sh.count[bin], 1u);
            if (MASS) add_mass(sh, bin, mass(l));
        });
        find_bin<MASS>(sh, cs, rank, above_count, above_mass, k, target);
        if (sh.found_bin == 0xffffffffu) return;  // every token that takes part is left
        prefix = (prefix << bits) | sh.found_bin;
        shift = next;
        above_count = sh.found_count;
        above_mass = sh.found_mass;
        __syncthreads();
    }
    // the tokens of the last bin are equal: the first `want` of them stay
    const uint32_t n_eq = sh.found_n;
    uint32_t want;
    if (MASS) {
        const double each = (double)sh.found_w / n_eq;
        const double q = each > 0 ? ceil((target - (double)above_mass) / each) : 1.0;
        want = q < 1 ? 1 : (q > (double)n_eq ? n_eq : (uint32_t)q);
    } else {
        want = k - above_count;
    }
    uint32_t limit = 0xffffffffu;
    if (want < n_eq) {
        // index of the want-th of them: the CTAs' slices are in index order
        const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
        const int64_t per = ((row.n + kWarps - 1) / kWarps + 31) / 32 * 32;
        const int64_t i0 = warp * per, i1 = i0 + per < row.n ? i0 + per : row.n;
        auto equal = [&](int64_t i) {
            if (i >= i1) return false;
            const float l = row.at(i);
            return (order_bits(l) >> shift) == prefix && near(l, row.base + (uint32_t)i);
        };
        uint32_t mine = 0;  // this warp's share: of the list, or of the slice (contiguous ranges)
        if (in_list) {
            for (uint32_t i = threadIdx.x; i < (listed + 31) / 32 * 32; i += kThreads)
                mine += __popc(__ballot_sync(0xffffffffu, i < listed && (order_bits(__uint_as_float(sh.list[i].x)) >> shift) == prefix));
        } else {
            for (int64_t i = i0; i < i1; i += 32) mine += __popc(__ballot_sync(0xffffffffu, equal(i + lane)));
        }
        if (lane == 0) sh.redc[warp] = mine;
        __syncthreads();
        if (threadIdx.x == 0) {
            uint32_t s = 0;
            for (int i = 0; i < kWarps; ++i) s += sh.redc[i];
            sh.ties = s;
        }
        cluster_sync(cs);
        uint32_t before = 0;
        for (int q = 0; q < rank; ++q) before += *remote(&sh.ties, q, cs);
        if (in_list) {
            if (before < want && want <= before + sh.ties)
                for (uint32_t i = threadIdx.x; i < listed; i += kThreads) {
                    if ((order_bits(__uint_as_float(sh.list[i].x)) >> shift) != prefix) continue;
                    const uint32_t idx = sh.list[i].y;
                    uint32_t at = before;  // equal ones of a lower index
                    for (uint32_t j = 0; j < listed; ++j)
                        at += (order_bits(__uint_as_float(sh.list[j].x)) >> shift) == prefix && sh.list[j].y < idx;
                    if (at == want - 1)
                        for (int q = 0; q < cs; ++q) *remote(&sh.limit, q, cs) = idx;
                }
        } else {
            for (int i = 0; i < warp; ++i) before += sh.redc[i];
            if (before < want && want <= before + mine) {
                uint32_t left = want - before;  // the left-th of this warp's
                for (int64_t i = i0; i < i1; i += 32) {
                    const uint32_t m = __ballot_sync(0xffffffffu, equal(i + lane));
                    const uint32_t c = __popc(m);
                    if (left <= c) {
                        const int pos = __fns(m, 0, (int)left);
                        if (lane == 0)
                            for (int q = 0; q < cs; ++q) *remote(&sh.limit, q, cs) = row.base + (uint32_t)(i + pos);
                        break;
                    }
                    left -= c;
                }
            }
        }
        cluster_sync(cs);
        limit = sh.limit;
    }
    cut.prefix = prefix;
    cut.shift = shift;
    cut.limit = limit;
}

template <typename T, bool CACHED>
__global__ void __launch_bounds__(kThreads) sample_kernel(const SampleArgs a, const int cs, const int64_t slice) {
    constexpr int VE = 16 / sizeof(T);
    constexpr int ROUNDS = sizeof(T) == 2 ? 2 : 3;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    SampleShared &sh = *reinterpret_cast<SampleShared *>(smem_raw);
    T *buf = reinterpret_cast<T *>(smem_raw + align16(sizeof(SampleShared)));
    pdl_trigger();
    pdl_wait();
    const int64_t r = blockIdx.x / cs;
    const int rank = blockIdx.x % cs;
    const int64_t base = rank * slice;
    const int64_t n = a.V - base < slice ? (a.V > base ? a.V - base : 0) : slice;
    const T *src = static_cast<const T *>(a.logits) + r * a.logits_st + base;
    const float *noise = a.noise + r * a.noise_st;

    // the row's settings
    float temp = a.temperature ? a.temperature[r] : a.temperature_v;
    const float top_p = a.top_p ? a.top_p[r] : a.top_p_v;
    const float min_p = a.min_p ? a.min_p[r] : a.min_p_v;
    const int32_t top_k = a.top_k ? a.top_k[r] : a.top_k_v;
    const bool only_first = !(temp > 0.f) || top_p <= 0.f || min_p > 1.f || top_k == 1;
    temp = temp > 0.f ? fminf(temp, FLT_MAX) : 1.f;
    const bool use_k = !only_first && top_k > 0 && top_k < a.V;
    const bool use_p = !only_first && top_p < 1.f;
    const bool use_m = !only_first && min_p > 0.f;
    const float to_log2 = 1.44269504088896341f / temp;
    const bool safe_scale = to_log2 < 1e30f;  // a temperature near zero: divide instead
    auto e_below = [&](float l, float top) {
        return safe_scale ? ex2((l - top) * to_log2) : ex2((l - top) / temp * 1.44269504088896341f);
    };

    // the slice into shared memory, with each thread's maximum and mass
    Row<T, CACHED> row;
    row.n = n;
    row.base = (uint32_t)base;
    row.mis = CACHED ? (int)(reinterpret_cast<uintptr_t>(src) / sizeof(T) % VE) : 0;
    float my_max = -INFINITY, my_z = 0.f;
    auto take = [&](const float (&v)[VE]) {
        float top = v[0];
#pragma unroll
        for (int e = 1; e < VE; ++e) top = fmaxf(top, v[e]);
        if (top > my_max) {
            my_z *= e_below(my_max, top);
            my_max = top;
        }
        if (my_max > -INFINITY)
#pragma unroll
            for (int e = 0; e < VE; ++e) my_z += e_below(v[e], my_max);
    };
    if constexpr (CACHED) {
        row.buf = buf;
        const int nvec = (int)((row.mis + n + VE - 1) / VE);
        constexpr int AHEAD = 4;  // pieces of a thread in flight
        for (int j0 = threadIdx.x; j0 < nvec; j0 += AHEAD * kThreads) {
            RawPiece<T, VE> raw[AHEAD];
#pragma unroll
            for (int u = 0; u < AHEAD; ++u) {
                const int64_t i = (int64_t)(j0 + u * kThreads) * VE - row.mis;
                if (i >= 0 && i + VE <= n) raw[u] = load_raw<T, VE>(src + i);
            }
#pragma unroll
            for (int u = 0; u < AHEAD; ++u) {
                const int j = j0 + u * kThreads;
                if (j >= nvec) break;
                const int64_t i = (int64_t)j * VE - row.mis;
                float v[VE];
                if (i >= 0 && i + VE <= n) {
                    widen<T, VE>(v, raw[u]);
                } else {
#pragma unroll
                    for (int e = 0; e < VE; ++e)
                        v[e] = i + e >= 0 && i + e < n ? Elem<T>::to_f32(src[i + e]) : -INFINITY;
                }
#pragma unroll
                for (int e = 0; e < VE; ++e) v[e] = canonical<T>(v[e]);
                store_piece<T, VE>(buf + (int64_t)j * VE, v);
                take(v);
            }
        }
    } else {
        row.buf = src;
        for (int64_t i0 = (int64_t)threadIdx.x * VE; i0 < n; i0 += (int64_t)kThreads * VE) {
            float v[VE];
#pragma unroll
            for (int e = 0; e < VE; ++e) v[e] = i0 + e < n ? logit(src[i0 + e]) : -INFINITY;
            take(v);
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
        sh.redf[threadIdx.x / 32] = mx;
        sh.redz[threadIdx.x / 32] = z;
    }
    if (threadIdx.x == 0) sh.race = 0.f;
    __syncthreads();
    mx = sh.redf[0];
    z = sh.redz[0];
    for (int i = 1; i < kWarps; ++i) join(sh.redf[i], sh.redz[i]);
    if (cs > 1) {
        if (threadIdx.x == 0) {
            sh.fslot[0] = mx;
            sh.fslot[1] = z;
        }
        cluster_sync(cs);
        mx = *remote(&sh.fslot[0], 0, cs);
        z = *remote(&sh.fslot[1], 0, cs);
        for (int q = 1; q < cs; ++q) join(*remote(&sh.fslot[0], q, cs), *remote(&sh.fslot[1], q, cs));
    }

    if (mx == -INFINITY) {  // nothing is left in this row
        if (rank == 0 && threadIdx.x == 0) {
            a.token[r] = -1;
            if (a.logprob) a.logprob[r] = -INFINITY;
        }
        cluster_sync(cs);
        return;
    }
    auto fast_e = [&](float l) { return e_below(l, mx); };
    auto exact_e = [&](float l) { return expf((l - mx) / temp); };
    auto over_min = [&](float l) {
        const float e = fast_e(l);
        if (fabsf(e - min_p) <= 1e-4f * min_p) return exact_e(l) >= min_p;
        return e >= min_p;
    };
    Cut cut;
    if (use_k) {
        if (top_k <= kThreads / 2) {
            // the k-th largest of the threads' maxima: at least k tokens of
            // this slice reach it, so it keeps all that can be among the first
            // k, and not many more
            const uint32_t mine = order_bits(my_max);
            uint32_t floor_ = 0;
#pragma unroll 1
            for (int bit = 31; bit >= (sizeof(T) == 2 ? 13 : 0); --bit) {
                const uint32_t t = floor_ | (1u << bit);
                if (__syncthreads_count(mine >= t) >= top_k) floor_ = t;
            }
            narrow<false, ROUNDS>(row, sh, cs, rank, cut, (uint32_t)top_k, 0.0, mx, 0.f,
                                  [&](float l, uint32_t) { return order_bits(l) >= floor_; }, fast_e);
        } else {
            // bins from the largest logit to past the least of the threads' maxima
            float least = my_max;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) least = fminf(least, __shfl_xor_sync(0xffffffffu, least, o));
            __syncthreads();
            if (threadIdx.x % 32 == 0) sh.redf[threadIdx.x / 32] = least;
            __syncthreads();
            for (int i = 0; i < kWarps; ++i) least = fminf(least, sh.redf[i]);
            if (cs > 1) {
                if (threadIdx.x == 0) sh.fslot[3] = least;
                cluster_sync(cs);
                for (int q = 0; q < cs; ++q) least = fminf(least, *remote(&sh.fslot[3], q, cs));
            }
            const float range = least > -INFINITY ? fmaxf(1.5f * (mx - least), 1e-20f) : 16.f * temp;
            narrow<false, ROUNDS>(row, sh, cs, rank, cut, (uint32_t)top_k, 0.0, mx, fminf(kBins / range, 1e30f),
                                  [&](float, uint32_t) { return true; }, fast_e);
        }
    }
    if (use_p) {
        float zk = z;
        if (use_k) {
            zk = 0.f;
            row.each([&](float l, uint32_t idx) {
                if (cut.keeps(order_bits(l), idx)) zk += fast_e(l);
            });
            zk = block_sum(zk, sh);
            if (cs > 1) {
                if (threadIdx.x == 0) sh.fslot[2] = zk;
                cluster_sync(cs);
                zk = 0.f;
                for (int q = 0; q < cs; ++q) zk += *remote(&sh.fslot[2], q, cs);
            }
        }
        // tokens of less than this e lie past the cut whatever their order: all
        // of them together hold less than 1 - top_p of the mass
        const float least = 0.5f * (1.f - top_p) * zk / (float)a.V;
        const float range = fmaxf(-logf(least), 1.f) * temp;   // of logits
        const float lowest = mx - 1.0001f * range;
        const Cut k_cut = cut;
        narrow<true, ROUNDS>(row, sh, cs, rank, cut, 0, (double)top_p * zk * 0x1p40, mx,
                             fminf(kBins / range, 1e30f),
                             [&](float l, uint32_t idx) { return l >= lowest && k_cut.keeps(order_bits(l), idx); },
                             fast_e);
    }

    // the race
    float best = -1.f;
    uint32_t best_i = 0xffffffffu;
    const bool all = !use_k && !use_p && !use_m && !only_first;
    auto run = [&](float l, uint32_t idx, float nz) {
        nz = fmaxf(nz, FLT_MIN);
        const float rough = __fdividef(fast_e(l), nz);
        const float floor_ = fmaxf(best, *(volatile float *)&sh.race);
        if (rough >= 0.9999f * floor_ || nz > 0x1p120f) {
            const float key = exact_e(l) / nz;
            if (key > best || (key == best && idx < best_i)) {
                best = key;
                best_i = idx;
                if (key > floor_) atomicMax(reinterpret_cast<int *>(&sh.race), __float_as_int(key));
            }
        }
    };
    if (only_first) {
        row.each([&](float l, uint32_t idx) {
            if (l == mx && idx < best_i) {
                best = 1.f;
                best_i = idx;
            }
        });
    } else if (all) {
        // four tokens per thread in flight, neighbouring threads on
        // neighbouring tokens
        int64_t i = threadIdx.x;
        for (; i + 3 * kThreads < n; i += 4 * kThreads) {
            float nz[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) nz[u] = noise[base + i + u * kThreads];
#pragma unroll
            for (int u = 0; u < 4; ++u) run(row.at(i + u * kThreads), (uint32_t)(base + i + u * kThreads), nz[u]);
        }
        for (; i < n; i += kThreads) run(row.at(i), (uint32_t)(base + i), noise[base + i]);
    } else {
        row.each([&](float l, uint32_t idx) {
            // (a masked token cannot win, and a piece's places around the slice
            // hold -inf: no noise is read for either)
            if (l == -INFINITY || !cut.keeps(order_bits(l), idx)) return;
            if (use_m && l != mx && !over_min(l)) return;
            run(l, idx, noise[idx]);
        });
    }
    unsigned long long pack =
        best < 0.f ? 0ull : ((unsigned long long)__float_as_uint(best) << 32) | (0xffffffffu - best_i);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const unsigned long long p = __shfl_xor_sync(0xffffffffu, pack, o);
        if (p > pack) pack = p;
    }
    __syncthreads();
    if (threadIdx.x % 32 == 0) sh.redm[threadIdx.x / 32] = pack;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 0; i < kWarps; ++i)
            if (sh.redm[i] > pack) pack = sh.redm[i];
        sh.best = pack;
    }
    cluster_sync(cs);
    if (rank == 0 && threadIdx.x == 0) {
        for (int q = 0; q < cs; ++q) {
            const unsigned long long p = *remote(&sh.best, q, cs);
            if (p > pack) pack = p;
        }
        const uint32_t token = 0xffffffffu - (uint32_t)pack;
        a.token[r] = (int32_t)token;
        if (a.logprob) {
            const float l = logit(static_cast<const T *>(a.logits)[r * a.logits_st + token]);
            a.logprob[r] = (l - mx) / temp - logf(z);
        }
    }
    cluster_sync(cs);  // no CTA leaves while another reads its shared memory
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
    auto bytes_of = [&](int cs) { return align16(sizeof(SampleShared)) + (size_t)(slice_of(cs) + VE) * sizeof(T); };
    // a row over as few CTAs as leave room for two of them on an SM, so that
    // one loads while another computes; over more while SMs would stay idle
    int cs = 1;
    while (cs < kMaxCluster && bytes_of(cs) > kTwoPerSm) cs *= 2;
    while (cs < kMaxCluster && a.R * cs * 2 <= sms && slice_of(cs) > 4096) cs *= 2;
    if (a.R * cs > INT32_MAX) return cudaErrorInvalidConfiguration;
    if (bytes_of(cs) > kMostShared)
        return launch_cs<T, false>(a, cs, slice_of(cs), align16(sizeof(SampleShared)), s);
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
