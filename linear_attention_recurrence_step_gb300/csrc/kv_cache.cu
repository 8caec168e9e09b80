// kv_cache.cu -- writing tokens to the 4-bit paged cache and reading them.
//
// A group of 16 elements u = x / head scale is held as s * e2m1(u / s) with
// s = e4m3(max|u| / 6).  Both roundings are to the nearest of the exact
// quotient: a float32 quotient can fall on a border between two codes only
// where its remainder says on which side of it the exact one lies.
//
// Bound by issue: 70 % of the slots of a write, 56 % of a read go to index arithmetic
// and conversions (write and read of 4 prompts of up to 4096 tokens of 8 heads of 128, 86
// MB in the mean: 28 us, 31 with cold caches, of 13 by the bytes).  One thread per group,
// neighbouring threads on neighbouring groups, whose scales go out four to a word.
#include "attend.h"
#include "fp4.cuh"
#include "pieces.cuh"

namespace gdn {

namespace {

constexpr int kKvThreads = 256;

// A quotient a/b >= 0 from its float32 rounding q, moved off q if a/b is not q
// itself: on the same side of every border that q is not on.
__device__ __forceinline__ float beside(float q, float a, float b) {
    const float r = fmaf(-q, b, a);
    return r > 0.f ? __uint_as_float(__float_as_uint(q) + 1u)
                   : r < 0.f ? __uint_as_float(__float_as_uint(q) - 1u) : q;
}

// The larger one, a NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float m;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
    return m;
}

// Where a (token, kv, head, group) of the flat index lies.
struct Place {
    int64_t token;
    int head, group;
    bool value;
};
__device__ __forceinline__ Place place_of(int64_t i, int H, int groups) {
    Place p;
    const unsigned half = (unsigned)(H * groups), per = 2 * half;
    unsigned r;
    if (i <= UINT32_MAX) {  // (a quarter of the cost of the other division)
        p.token = (unsigned)i / per;
        r = (unsigned)i - (unsigned)p.token * per;
    } else {
        p.token = i / per;
        r = (unsigned)(i - p.token * per);
    }
    p.value = r >= half;
    if (p.value) r -= half;
    p.head = (int)(r / (unsigned)groups);
    p.group = (int)(r - (unsigned)p.head * (unsigned)groups);
    return p;
}
// The group's codes and scale in the cache (the slot is valid).
__device__ __forceinline__ unsigned char *codes_of(const KvArgs &a, int slot, const Place &p, unsigned char **scale) {
    const int page = 1 << a.page_shift, half = page * a.D / 2;
    const int64_t block = ((int64_t)(slot >> a.page_shift) * a.H + p.head) * kv_block_bytes(page, a.D);
    unsigned char *base = a.cache + block + (p.value ? half + page * (a.D / 16) : 0);
    const int row = slot & (page - 1);
    *scale = base + half + row * (a.D / 16) + p.group;
    return base + row * (a.D / 2) + p.group * 8;
}

template <typename T, bool VECTOR>
__global__ void __launch_bounds__(kKvThreads) kv_append_kernel(const KvArgs a, int64_t total) {
    pdl_trigger();
    pdl_wait();
    const int64_t i = (int64_t)blockIdx.x * kKvThreads + threadIdx.x;
    Place p{};
    int slot = -1;
    if (i < total) {
        p = place_of(i, a.H, a.D / 16);
        slot = a.slots[p.token];
        if ((slot >> a.page_shift) >= a.pages) slot = -1;
    }
    uint32_t sb = 0u;
    unsigned char *scale = nullptr;
    if (slot >= 0) {
        int64_t b = 0, t = p.token;
        if (a.B > 1) {
            b = p.token <= INT32_MAX && a.T <= INT32_MAX ? (unsigned)p.token / (unsigned)a.T : p.token / a.T;
            t -= b * a.T;
        }
        const T *src = static_cast<const T *>(p.value ? a.v_in : a.k_in) + b * (p.value ? a.v_sb : a.k_sb) +
                       t * (p.value ? a.v_st : a.k_st) + (int64_t)p.head * a.D + p.group * 16;
        constexpr int VEC = VECTOR ? 16 / (int)sizeof(T) : 1;
        float u[16];
#pragma unroll
        for (int e = 0; e < 16; e += VEC) {
            float v[VEC];
            load_piece<T, VEC>(v, src + e);
#pragma unroll
            for (int f = 0; f < VEC; ++f) u[e + f] = v[f];
        }
        const float *hs = p.value ? a.v_scale : a.k_scale;
        bool any = sizeof(T) == 4;  // u may be any float
        if (hs) {
            // a power of two divides exactly by its reciprocal, any other number by division
            const float g = hs[p.head], r = 1.f / g;
            if ((__float_as_uint(g) & 0x007fffffu) == 0 && r >= 0x1p-126f && r <= 0x1p126f) {
#pragma unroll
                for (int e = 0; e < 16; ++e) u[e] *= r;
            } else {
                any = true;
#pragma unroll
                for (int e = 0; e < 16; ++e) u[e] /= g;
            }
        }
        float top = 0.f;
#pragma unroll
        for (int e = 0; e < 16; ++e) top = max_nan(top, fabsf(u[e]));
        if (!(top < INFINITY)) {  // a NaN is written as zero, an infinity as the largest value
            top = 0.f;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                u[e] = u[e] == u[e] ? fminf(fmaxf(u[e], -3.4e38f), 3.4e38f) : 0.f;
                top = fmaxf(top, fabsf(u[e]));
            }
        }
        sb = f32_to_e4m3(beside(top / 6.f, top, 6.f));
        const float s = f16_lo(e4m3x2_to_f16(sb));
        const float inv = s > 0.f ? 1.f / s : 0.f;
        uint32_t word[2] = {0u, 0u};
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
            float q[2];
#pragma unroll
            for (int f = 0; f < 2; ++f) {
                // the quotient's nearest float; of 16-bit values' none but a border itself
                // is one
                float x = u[e + f] * inv;
                x = fmaf(fmaf(-x, s, u[e + f]), inv, x);
                if (any && s > 0.f) x = copysignf(beside(fabsf(x), fabsf(u[e + f]), s), u[e + f]);
                q[f] = x;
            }
            word[e / 8] |= f32_to_e2m1x2(q[0], q[1]) << (4 * (e % 8));
        }
        *reinterpret_cast<uint2 *>(codes_of(a, slot, p, &scale)) = make_uint2(word[0], word[1]);
    }
    // (groups of four are of one token and head: D/16 is a multiple of four)
    sb |= __shfl_down_sync(0xffffffffu, sb, 1) << 8;
    sb |= __shfl_down_sync(0xffffffffu, sb, 2) << 16;
    if (slot >= 0 && p.group % 4 == 0) *reinterpret_cast<uint32_t *>(scale) = sb;
}

template <typename T, bool VECTOR>
__global__ void __launch_bounds__(kKvThreads) kv_read_kernel(const KvArgs a, int64_t total) {
    pdl_trigger();
    pdl_wait();
    const int64_t i = (int64_t)blockIdx.x * kKvThreads + threadIdx.x;
    if (i >= total) return;
    const Place p = place_of(i, a.H, a.D / 16);
    const int slot = a.slots[p.token];
    if (slot < 0 || (slot >> a.page_shift) >= a.pages) return;
    unsigned char *scale;
    const uint2 w = *reinterpret_cast<const uint2 *>(codes_of(a, slot, p, &scale));
    const float *hs = p.value ? a.v_scale : a.k_scale;
    const float s = f16_lo(e4m3x2_to_f16(*scale)), g = hs ? hs[p.head] : 1.f;
    float u[16];
    const uint32_t word[2] = {w.x, w.y};
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        uint32_t h[4];
        e2m1x8_to_f16(word[j], h);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            u[8 * j + 2 * e] = f16_lo(h[e]) * s * g;
            u[8 * j + 2 * e + 1] = f16_hi(h[e]) * s * g;
        }
    }
    T *dst = static_cast<T *>(p.value ? a.v_out : a.k_out) + (p.token * a.H + p.head) * a.D + p.group * 16;
    constexpr int VEC = VECTOR ? 16 / (int)sizeof(T) : 1;
#pragma unroll
    for (int e = 0; e < 16; e += VEC) {
        float v[VEC];
#pragma unroll
        for (int f = 0; f < VEC; ++f) v[f] = u[e + f];
        store_piece<T, VEC>(dst + e, v);
    }
}

template <typename T>
cudaError_t launch_append_t(const KvArgs &a, cudaStream_t s) {
    const int64_t total = a.B * a.T * 2 * a.H * (a.D / 16), blocks = (total + kKvThreads - 1) / kKvThreads;
    if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
    return a.vec ? launch_dependent(kv_append_kernel<T, true>, (unsigned)blocks, kKvThreads, 0, s, a, total)
                 : launch_dependent(kv_append_kernel<T, false>, (unsigned)blocks, kKvThreads, 0, s, a, total);
}
template <typename T>
cudaError_t launch_read_t(const KvArgs &a, cudaStream_t s) {
    const int64_t total = a.B * a.T * 2 * a.H * (a.D / 16), blocks = (total + kKvThreads - 1) / kKvThreads;
    if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
    return a.vec ? launch_dependent(kv_read_kernel<T, true>, (unsigned)blocks, kKvThreads, 0, s, a, total)
                 : launch_dependent(kv_read_kernel<T, false>, (unsigned)blocks, kKvThreads, 0, s, a, total);
}

}  // namespace

cudaError_t launch_kv_append(DType dt, const KvArgs &a, cudaStream_t s) {
    switch (dt) {
    case DType::F32: return launch_append_t<float>(a, s);
    case DType::BF16: return launch_append_t<__nv_bfloat16>(a, s);
    case DType::F16: return launch_append_t<__half>(a, s);
    }
    return cudaErrorInvalidValue;
}
cudaError_t launch_kv_read(DType dt, const KvArgs &a, cudaStream_t s) {
    switch (dt) {
    case DType::F32: return launch_read_t<float>(a, s);
    case DType::BF16: return launch_read_t<__nv_bfloat16>(a, s);
    case DType::F16: return launch_read_t<__half>(a, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace gdn
