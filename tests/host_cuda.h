// host_cuda.h -- enough of CUDA C++ to run a kernel's source on the host.
//
// Every CUDA thread of a cluster is a fiber of one host thread; a fiber runs
// until it waits at a barrier (warp, block or cluster), and a set of fibers
// that all wait is reported as a deadlock.  Shared memory is filled with 0xcd
// before a block starts.  Accesses that a kernel makes by inline PTX (turned
// into calls of the `ptx` functions below by host_cuda.py) are checked for
// their alignment and their bounds: shared ones against the block's shared
// memory, global ones against the ranges that the caller has named.  A failed
// check ends the launch with an error message.
#pragma once

#include <sys/mman.h>
#include <ucontext.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <deque>
#include <functional>
#include <memory>
#include <vector>

using std::max;
using std::min;

#define __device__
#define __host__
#define __global__
#define __forceinline__ inline
#define __launch_bounds__(...)

struct uint3 { unsigned x, y, z; };
struct dim3 {
    unsigned x, y, z;
    dim3(unsigned a = 1, unsigned b = 1, unsigned c = 1) : x(a), y(b), z(c) {}
};
struct alignas(8) float2 { float x, y; };
struct alignas(16) float4 { float x, y, z, w; };
struct alignas(16) uint4 { uint32_t x, y, z, w; };
inline float2 make_float2(float a, float b) { return {a, b}; }
inline float4 make_float4(float a, float b, float c, float d) { return {a, b, c, d}; }
inline uint4 make_uint4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) { return {a, b, c, d}; }

extern uint3 threadIdx, blockIdx;
extern dim3 blockDim, gridDim;

// ------------------------------------------------------------------- fibers
namespace host {

constexpr size_t kStack = 128 * 1024;

struct Fiber;
struct Gate {  // a barrier of `need` fibers
    int need = 0, arrived = 0;
    uint64_t turn = 0;
    std::vector<Fiber *> waiting;
};
struct Warp {
    Gate gate;
    uint64_t slot[2][32];
};
struct Block {
    unsigned rank;
    uint3 idx;
    std::vector<unsigned char> memory;  // with room to align it
    unsigned char *shared;
    Gate gate;
    int count[2] = {0, 0};
    std::vector<Warp> warps;
};
struct Fiber {
    ucontext_t at;
    Block *block;
    unsigned thread;
};

struct Range { uintptr_t first, end; };

struct Machine {
    ucontext_t main;
    std::deque<Fiber *> ready;
    Fiber *now = nullptr;
    size_t running = 0, shared_bytes = 0;
    Gate cluster;
    std::vector<Block *> blocks;
    std::function<void()> kernel;
    std::vector<Range> ranges;
    char error[256] = "";
};
inline Machine m;

[[noreturn]] inline void fail(const char *fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    const int n = snprintf(m.error, sizeof m.error, "block %u thread %u: ", blockIdx.x, threadIdx.x);
    vsnprintf(m.error + n, sizeof m.error - n, fmt, ap);
    va_end(ap);
    setcontext(&m.main);
    abort();
}

inline void enter(Fiber *f) {
    m.now = f;
    threadIdx = {f->thread, 0, 0};
    blockIdx = f->block->idx;
}
// to the next fiber that can run
inline void next(ucontext_t *from) {
    if (m.ready.empty()) {
        if (m.running) fail("every thread waits");
        setcontext(&m.main);
    }
    Fiber *f = m.ready.front();
    m.ready.pop_front();
    enter(f);
    if (from) swapcontext(from, &f->at);
    else setcontext(&f->at);
}
inline uint64_t arrive(Gate &g) {
    const uint64_t turn = g.turn;
    if (++g.arrived == g.need) {
        g.arrived = 0;
        ++g.turn;
        for (Fiber *f : g.waiting) m.ready.push_back(f);
        g.waiting.clear();
    }
    return turn;
}
inline void wait(Gate &g, uint64_t turn) {
    while (g.turn == turn) {
        Fiber *self = m.now;
        g.waiting.push_back(self);
        next(&self->at);
    }
}
inline void pass(Gate &g) { wait(g, arrive(g)); }

inline void body() {
    m.kernel();
    --m.running;
    next(nullptr);
}

inline bool run(unsigned grid, unsigned block, unsigned cluster, size_t shared, const std::function<void()> &kernel) {
    const size_t n = (size_t)block * cluster;
    static std::vector<unsigned char *> stacks;
    while (stacks.size() < n) {
        void *p = mmap(nullptr, kStack, PROT_READ | PROT_WRITE, MAP_PRIVATE | MAP_ANONYMOUS | MAP_NORESERVE, -1, 0);
        if (p == MAP_FAILED) abort();
        stacks.push_back(static_cast<unsigned char *>(p));
    }
    blockDim = dim3(block);
    gridDim = dim3(grid);
    m.error[0] = 0;
    m.kernel = kernel;
    m.shared_bytes = shared;
    for (volatile unsigned c = 0; c < grid / cluster; c = c + 1) {
        std::vector<std::unique_ptr<Block>> blocks;
        std::vector<std::unique_ptr<Fiber>> fibers;
        m.blocks.clear();
        m.ready.clear();
        m.cluster = Gate();
        m.cluster.need = (int)n;
        m.running = n;
        for (unsigned q = 0; q < cluster; ++q) {
            auto b = std::make_unique<Block>();
            b->rank = q;
            b->idx = {c * cluster + q, 0, 0};
            b->memory.assign(shared + 1024, 0xcd);
            b->shared = b->memory.data() + (1024 - reinterpret_cast<uintptr_t>(b->memory.data()) % 1024) % 1024;
            b->gate.need = (int)block;
            b->warps.resize(block / 32);
            for (Warp &w : b->warps) w.gate.need = 32;
            for (unsigned t = 0; t < block; ++t) {
                auto f = std::make_unique<Fiber>();
                f->block = b.get();
                f->thread = t;
                getcontext(&f->at);
                f->at.uc_stack.ss_sp = stacks[q * block + t];
                f->at.uc_stack.ss_size = kStack;
                f->at.uc_link = nullptr;
                makecontext(&f->at, body, 0);
                m.ready.push_back(f.get());
                fibers.push_back(std::move(f));
            }
            m.blocks.push_back(b.get());
            blocks.push_back(std::move(b));
        }
        volatile bool started = false;
        getcontext(&m.main);  // fibers come back here
        if (!started) {
            started = true;
            next(nullptr);
        }
        if (m.error[0]) return false;
    }
    return true;
}

inline Warp &warp() { return m.now->block->warps[m.now->thread / 32]; }
// every lane's value of this turn (two turns are kept: a lane can be one ahead)
template <typename V> inline const uint64_t *exchange(V v) {
    Warp &w = warp();
    const int which = (int)(w.gate.turn & 1);
    uint64_t bits = 0;
    memcpy(&bits, &v, sizeof v);
    w.slot[which][m.now->thread % 32] = bits;
    pass(w.gate);
    return w.slot[which];
}
template <typename V> inline V value(uint64_t bits) {
    V v;
    memcpy(&v, &bits, sizeof v);
    return v;
}

// a shared::cluster address: the block's rank above an offset of 24 bits
inline unsigned char *shared(uint32_t a, size_t bytes) {
    const uint32_t rank = a >> 24, off = a & 0xffffff;
    if (rank >= m.blocks.size()) fail("shared address of block %u in a cluster of %zu", rank, m.blocks.size());
    if (off % bytes || off + bytes > m.shared_bytes)
        fail("%zu bytes of shared memory at %u of %zu", bytes, off, m.shared_bytes);
    return m.blocks[rank]->shared + off;
}
inline unsigned char *own(uint32_t a, size_t bytes) {
    if (a >> 24 != m.now->block->rank) fail("own shared memory by another block's address");
    return shared(a, bytes);
}
inline const unsigned char *global(uint64_t a, size_t bytes) {
    if (a % bytes) fail("%zu bytes of global memory at a multiple of %zu", bytes, (size_t)(a & -a));
    for (const Range &r : m.ranges)
        if (a >= r.first && a + bytes <= r.end) return reinterpret_cast<const unsigned char *>(a);
    fail("%zu bytes of global memory outside every tensor", bytes);
}
template <typename V> inline V at(const unsigned char *p) {
    V v;
    memcpy(&v, p, sizeof v);
    return v;
}
inline float ftz(float x) { return fabsf(x) < FLT_MIN ? copysignf(0.f, x) : x; }

}  // namespace host

// --------------------------------------------------- PTX (host_cuda.py's calls)
namespace ptx {
using namespace host;
inline void ld_shared_u32(uint32_t &v, uint32_t a) { v = at<uint32_t>(own(a, 4)); }
inline void ld_shared_f32(float &v, uint32_t a) { v = at<float>(own(a, 4)); }
inline void ld_shared_u16(uint16_t &v, uint32_t a) { v = at<uint16_t>(own(a, 2)); }
inline void st_shared_u32(uint32_t a, uint32_t v) { memcpy(own(a, 4), &v, 4); }
inline void ld_shared_v4_u32(uint32_t &x, uint32_t &y, uint32_t &z, uint32_t &w, uint32_t a) {
    const unsigned char *p = own(a, 16);
    x = at<uint32_t>(p), y = at<uint32_t>(p + 4), z = at<uint32_t>(p + 8), w = at<uint32_t>(p + 12);
}
inline void st_shared_v4_u32(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    const uint32_t v[4] = {x, y, z, w};
    memcpy(own(a, 16), v, 16);
}
inline void atom_add(unsigned char *p, uint32_t *old, uint32_t v) {
    const uint32_t was = at<uint32_t>(p), is = was + v;
    memcpy(p, &is, 4);
    if (old) *old = was;
}
inline void atom_shared_add_u32(uint32_t &old, uint32_t a, uint32_t v) { atom_add(own(a, 4), &old, v); }
inline void red_shared_add_u32(uint32_t a, uint32_t v) { atom_add(own(a, 4), nullptr, v); }
inline void red_shared_max_u32(uint32_t a, uint32_t v) {
    const uint32_t is = max(at<uint32_t>(own(a, 4)), v);
    memcpy(own(a, 4), &is, 4);
}
inline void red_shared_min_u32(uint32_t a, uint32_t v) {
    const uint32_t is = min(at<uint32_t>(own(a, 4)), v);
    memcpy(own(a, 4), &is, 4);
}
inline void mapa_shared_cluster_u32(uint32_t &to, uint32_t a, uint32_t rank) { to = (a & 0xffffff) | rank << 24; }
inline void ld_shared_cluster_u32(uint32_t &v, uint32_t a) { v = at<uint32_t>(shared(a, 4)); }
inline void st_shared_cluster_u32(uint32_t a, uint32_t v) { memcpy(shared(a, 4), &v, 4); }
inline void atom_shared_cluster_add_u32(uint32_t &old, uint32_t a, uint32_t v) { atom_add(shared(a, 4), &old, v); }
inline uint64_t cluster_turn;
inline void barrier_cluster_arrive_release_aligned() { cluster_turn = arrive(m.cluster); }
// (a fiber goes from its arrive to its wait without another in between)
inline void barrier_cluster_wait_acquire_aligned() { host::wait(m.cluster, cluster_turn); }
inline void ld_global_nc_f32(float &v, const void *p) { v = at<float>(global(reinterpret_cast<uint64_t>(p), 4)); }
inline void ld_global_nc_v4_u32(uint32_t &x, uint32_t &y, uint32_t &z, uint32_t &w, uint64_t a) {
    const unsigned char *p = global(a, 16);
    x = at<uint32_t>(p), y = at<uint32_t>(p + 4), z = at<uint32_t>(p + 8), w = at<uint32_t>(p + 12);
}
inline void prefetch_global_L2(const void *p) { global(reinterpret_cast<uint64_t>(p) & ~(uint64_t)3, 4); }
inline void ex2_approx_ftz_f32(float &y, float x) { y = ftz(exp2f(ftz(x))); }
inline void rcp_approx_ftz_f32(float &y, float x) { y = ftz(1.f / ftz(x)); }
}  // namespace ptx

// ---------------------------------------------------------------- intrinsics
inline size_t __cvta_generic_to_shared(const void *) { return (size_t)host::m.now->block->rank << 24; }
inline void __syncthreads() { host::pass(host::m.now->block->gate); }
inline int __syncthreads_count(bool p) {
    host::Block &b = *host::m.now->block;
    const int which = (int)(b.gate.turn & 1);
    b.count[which] += p;
    if (b.gate.arrived + 1 == b.gate.need) b.count[which ^ 1] = 0;  // the next turn's
    host::pass(b.gate);
    return b.count[which];
}
template <typename V> inline V __shfl_sync(unsigned, V v, int lane) { return host::value<V>(host::exchange(v)[lane & 31]); }
template <typename V> inline V __shfl_xor_sync(unsigned, V v, int o) {
    return host::value<V>(host::exchange(v)[(threadIdx.x % 32) ^ (unsigned)o]);
}
template <typename V> inline V __shfl_up_sync(unsigned, V v, int o) {
    const int lane = (int)(threadIdx.x % 32);
    return host::value<V>(host::exchange(v)[lane >= o ? lane - o : lane]);
}
inline uint32_t __ballot_sync(unsigned, bool p) {
    const uint64_t *all = host::exchange(p);
    uint32_t bits = 0;
    for (int i = 0; i < 32; ++i) bits |= (uint32_t)(all[i] != 0) << i;
    return bits;
}
inline bool __any_sync(unsigned mask, bool p) { return __ballot_sync(mask, p) != 0; }
template <typename Join> inline uint32_t reduce_lanes(uint32_t v, Join join) {
    const uint64_t *all = host::exchange(v);
    uint32_t r = (uint32_t)all[0];
    for (int i = 1; i < 32; ++i) r = join(r, (uint32_t)all[i]);
    return r;
}
inline uint32_t __reduce_add_sync(unsigned, uint32_t v) { return reduce_lanes(v, [](uint32_t a, uint32_t b) { return a + b; }); }
inline uint32_t __reduce_max_sync(unsigned, uint32_t v) { return reduce_lanes(v, [](uint32_t a, uint32_t b) { return max(a, b); }); }
inline uint32_t __reduce_min_sync(unsigned, uint32_t v) { return reduce_lanes(v, [](uint32_t a, uint32_t b) { return min(a, b); }); }

inline uint32_t __float_as_uint(float f) {
    uint32_t u;
    memcpy(&u, &f, 4);
    return u;
}
inline float __uint_as_float(uint32_t u) {
    float f;
    memcpy(&f, &u, 4);
    return f;
}
inline int __popc(uint32_t x) { return __builtin_popcount(x); }
inline int __ffs(uint32_t x) { return x ? __builtin_ctz(x) + 1 : 0; }
inline int __clz(uint32_t x) { return x ? __builtin_clz(x) : 32; }
inline int __fns(uint32_t mask, unsigned, int n) {  // place of the n-th set bit
    for (int i = 0; i < 32; ++i)
        if (mask >> i & 1 && --n == 0) return i;
    return -1;
}
inline uint32_t to_uint(double d) { return !(d > 0) ? 0 : d >= 4294967295.0 ? 0xffffffffu : (uint32_t)d; }
inline uint32_t __float2uint_rz(float f) { return to_uint(std::trunc((double)f)); }
inline uint32_t __float2uint_rn(float f) { return to_uint(std::nearbyint((double)f)); }
inline unsigned long long __double2ull_ru(double d) { return d > 0 ? (unsigned long long)std::ceil(d) : 0; }
inline float2 __fadd2_rn(float2 a, float2 b) { return {a.x + b.x, a.y + b.y}; }
inline float2 __fmul2_rn(float2 a, float2 b) { return {a.x * b.x, a.y * b.y}; }
inline float2 __ffma2_rn(float2 a, float2 b, float2 c) { return {fmaf(a.x, b.x, c.x), fmaf(a.y, b.y, c.y)}; }

// ------------------------------------------------------------- 16-bit types
struct __nv_bfloat16 { uint16_t bits; };
struct __half { _Float16 v; };
struct alignas(4) __nv_bfloat162 { __nv_bfloat16 x, y; };
struct alignas(4) __half2 { __half x, y; };
inline float __bfloat162float(__nv_bfloat16 x) { return __uint_as_float((uint32_t)x.bits << 16); }
inline __nv_bfloat16 __float2bfloat16_rn(float f) {
    if (f != f) return {0x7fff};
    uint32_t u = __float_as_uint(f);
    u += 0x7fff + (u >> 16 & 1);
    return {(uint16_t)(u >> 16)};
}
inline float __half2float(__half x) { return (float)x.v; }
inline __half __float2half_rn(float f) { return {(_Float16)f}; }
inline float2 __half22float2(__half2 x) { return {__half2float(x.x), __half2float(x.y)}; }
inline __half2 __floats2half2_rn(float a, float b) { return {__float2half_rn(a), __float2half_rn(b)}; }
inline __nv_bfloat162 __floats2bfloat162_rn(float a, float b) { return {__float2bfloat16_rn(a), __float2bfloat16_rn(b)}; }
inline float __low2float(__nv_bfloat162 x) { return __bfloat162float(x.x); }
inline float __high2float(__nv_bfloat162 x) { return __bfloat162float(x.y); }
inline float __low2float(__half2 x) { return __half2float(x.x); }
inline float __high2float(__half2 x) { return __half2float(x.y); }
// (fmaxf and fminf take the number beside a NaN, as these do)
inline __nv_bfloat162 __hmax2(__nv_bfloat162 a, __nv_bfloat162 b) {
    return __floats2bfloat162_rn(fmaxf(__low2float(a), __low2float(b)), fmaxf(__high2float(a), __high2float(b)));
}
inline __nv_bfloat162 __hmin2(__nv_bfloat162 a, __nv_bfloat162 b) {
    return __floats2bfloat162_rn(fminf(__low2float(a), __low2float(b)), fminf(__high2float(a), __high2float(b)));
}
inline __half2 __hmax2(__half2 a, __half2 b) {
    return __floats2half2_rn(fmaxf(__low2float(a), __low2float(b)), fmaxf(__high2float(a), __high2float(b)));
}
inline __half2 __hmin2(__half2 a, __half2 b) {
    return __floats2half2_rn(fminf(__low2float(a), __low2float(b)), fminf(__high2float(a), __high2float(b)));
}

namespace cooperative_groups {
struct Cluster {
    void sync() const { host::pass(host::m.cluster); }
};
inline Cluster this_cluster() { return {}; }
}  // namespace cooperative_groups

// ----------------------------------------------------------------- launching
enum cudaError_t { cudaSuccess, cudaErrorInvalidValue, cudaErrorInvalidConfiguration, cudaErrorLaunchFailure };
typedef struct Stream *cudaStream_t;
enum { cudaFuncAttributeMaxDynamicSharedMemorySize };
enum { cudaLaunchAttributeProgrammaticStreamSerialization, cudaLaunchAttributeClusterDimension };
struct cudaLaunchAttribute {
    int id;
    struct { int programmaticStreamSerializationAllowed; struct { unsigned x, y, z; } clusterDim; } val;
};
struct cudaLaunchConfig_t {
    dim3 gridDim, blockDim;
    size_t dynamicSmemBytes;
    cudaStream_t stream;
    cudaLaunchAttribute *attrs;
    unsigned numAttrs;
};
constexpr size_t kSharedLimit = 227 * 1024;
template <typename F> cudaError_t cudaFuncSetAttribute(F *, int, int bytes) {
    return (size_t)bytes <= kSharedLimit ? cudaSuccess : cudaErrorInvalidValue;
}
template <typename... K, typename... A>
cudaError_t cudaLaunchKernelEx(const cudaLaunchConfig_t *cfg, void (*kernel)(K...), A &&...args) {
    unsigned cluster = 1;
    for (unsigned i = 0; i < cfg->numAttrs; ++i)
        if (cfg->attrs[i].id == cudaLaunchAttributeClusterDimension) cluster = cfg->attrs[i].val.clusterDim.x;
    if (cfg->gridDim.x % cluster || cfg->dynamicSmemBytes > kSharedLimit) return cudaErrorInvalidConfiguration;
    return host::run(cfg->gridDim.x, cfg->blockDim.x, cluster, cfg->dynamicSmemBytes, [&] { kernel(args...); })
               ? cudaSuccess
               : cudaErrorLaunchFailure;
}

// what common.cuh gives the kernels
namespace gdn {
template <typename... K, typename... A>
cudaError_t launch_dependent(void (*kernel)(K...), unsigned grid, unsigned block, size_t smem, cudaStream_t st, A &&...args) {
    cudaLaunchConfig_t cfg{dim3(grid), dim3(block), smem, st, nullptr, 0};
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}
inline void pdl_wait() {}
inline void pdl_trigger() {}
template <typename T> struct Elem;
template <> struct Elem<float> {
    static float to_f32(float x) { return x; }
    static float from_f32(float x) { return x; }
};
template <> struct Elem<__nv_bfloat16> {
    static float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
    static __nv_bfloat16 from_f32(float x) { return __float2bfloat16_rn(x); }
};
template <> struct Elem<__half> {
    static float to_f32(__half x) { return __half2float(x); }
    static __half from_f32(float x) { return __float2half_rn(x); }
};
template <typename T> inline float ld_f32(const T *p) { return Elem<T>::to_f32(*p); }
template <typename T> inline void st_from_f32(T *p, float x) { *p = Elem<T>::from_f32(x); }
inline float2 ffma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
inline float2 fmul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
}  // namespace gdn
