// rotary.cu -- rotary positions of queries and keys.
//
// Pair i of a head is turned by the angle position * inv_freq[i].  Far
// positions leave nothing of such an angle's fraction in float32, so it is
// counted in turns with 64 fixed-point bits: F = frac(inv_freq / 2 pi) 2^64
// once per frequency (one double product), position * F modulo 2^64 drops the
// whole turns by itself, and the upper 32 bits are the fraction, off by 2^-32
// of a turn and 2^-53 of inv_freq per step at most.
//
// Bound by memory: every element is read once and written once.  A block
// makes the sines of its tokens once, in shared memory, and uses them for all
// heads of q and k.
#include "attend.h"
#include "pieces.cuh"

namespace gdn {

namespace {

constexpr int kRotThreads = 256;

// Sine and cosine of 2 pi f, where f is a fraction of a turn (2^-32 units).
__device__ __forceinline__ float2 turn(int32_t f, float scale, bool inverse) {
    float s, c;
    sincospif((float)f * 0x1p-31f, &s, &c);
    return make_float2(c * scale, (inverse ? -s : s) * scale);
}

template <typename T, int VEC, bool HALF>
__global__ void __launch_bounds__(kRotThreads) rotary_kernel(const RotaryArgs a, int tokens_block) {
    extern __shared__ float2 cs[];  // [tokens_block][R/2]
    pdl_trigger();
    pdl_wait();
    const int n = a.R / 2;
    const int64_t tok0 = (int64_t)blockIdx.x * tokens_block, all = a.B * a.T;
    for (int i = threadIdx.x; i < tokens_block * n; i += kRotThreads) {
        const int tk = i / n, f = i - tk * n;
        const int pos = tok0 + tk < all ? a.positions[tok0 + tk] : -1;
        if (pos < 0) continue;
        double per = (double)a.inv_freq[f] * 0.15915494309189533577;
        per -= floor(per);
        const unsigned long long F = __double2ull_rn(per * 18446744073709551616.0);
        cs[i] = turn((int32_t)(((unsigned long long)(unsigned)pos * F) >> 32), a.scale, a.inverse);
    }
    __syncthreads();
    // units of a head: pieces of pairs (VEC elements of each half, or VEC
    // neighbouring elements), then pieces that stay as they are
    constexpr int kPairs1 = HALF ? VEC : VEC / 2 + (VEC == 1);
    const int turned = n / kPairs1, rest = (a.D - a.R) / VEC, units = turned + rest;
    const int heads = a.Hq + (a.k ? a.Hk : 0), per_token = heads * units;
    for (int i = threadIdx.x; i < tokens_block * per_token; i += kRotThreads) {
        const int tk = i / per_token, r = i - tk * per_token, h = r / units, u = r - h * units;
        const int64_t tok = tok0 + tk;
        if (tok >= all || a.positions[tok] < 0) continue;
        const int64_t b = tok / a.T, t = tok - b * a.T;
        const bool key = h >= a.Hq;
        const int hh = key ? h - a.Hq : h;
        const T *src = static_cast<const T *>(key ? a.k : a.q) + b * (key ? a.k_sb : a.q_sb) +
                       t * (key ? a.k_st : a.q_st) + (int64_t)hh * a.D;
        T *dst = static_cast<T *>(key ? a.k_out : a.q_out) + b * (key ? a.ko_sb : a.qo_sb) +
                 t * (key ? a.ko_st : a.qo_st) + (int64_t)hh * a.D;
        if (u >= turned) {
            const int d = a.R + (u - turned) * VEC;
            if (dst != src) store_raw<T, VEC>(dst + d, load_raw<T, VEC>(src + d));
            continue;
        }
        const float2 *w = cs + tk * n + u * kPairs1;
        if constexpr (HALF) {
            float x[VEC], y[VEC];
            load_piece<T, VEC>(x, src + u * VEC);
            load_piece<T, VEC>(y, src + n + u * VEC);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float2 c = w[e];
                const float p = x[e] * c.x - y[e] * c.y;
                y[e] = x[e] * c.y + y[e] * c.x;
                x[e] = p;
            }
            store_piece<T, VEC>(dst + u * VEC, x);
            store_piece<T, VEC>(dst + n + u * VEC, y);
        } else if constexpr (VEC == 1) {
            const float x = ld_f32(src + 2 * u), y = ld_f32(src + 2 * u + 1);
            const float2 c = w[0];
            st_from_f32(dst + 2 * u, x * c.x - y * c.y);
            st_from_f32(dst + 2 * u + 1, x * c.y + y * c.x);
        } else {
            float x[VEC];
            load_piece<T, VEC>(x, src + u * VEC);
#pragma unroll
            for (int e = 0; e < VEC; e += 2) {
                const float2 c = w[e / 2];
                const float p = x[e] * c.x - x[e + 1] * c.y;
                x[e + 1] = x[e] * c.y + x[e + 1] * c.x;
                x[e] = p;
            }
            store_piece<T, VEC>(dst + u * VEC, x);
        }
    }
}

template <typename T, int VEC>
cudaError_t launch_t(const RotaryArgs &a, int sm_count, cudaStream_t s) {
    const int64_t all = a.B * a.T;
    const int tb = all > (int64_t)(sm_count > 0 ? sm_count : 152) * 8 && a.R <= 2048 ? 4 : 1;
    const int64_t blocks = (all + tb - 1) / tb;
    if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
    const size_t smem = (size_t)tb * (a.R / 2) * sizeof(float2);
    return a.half ? launch_dependent(rotary_kernel<T, VEC, true>, (unsigned)blocks, kRotThreads, smem, s, a, tb)
                  : launch_dependent(rotary_kernel<T, VEC, false>, (unsigned)blocks, kRotThreads, smem, s, a, tb);
}

}  // namespace

cudaError_t launch_rotary(DType dt, const RotaryArgs &a, int sm_count, cudaStream_t s) {
    switch (dt) {
    case DType::F32: return a.vec ? launch_t<float, 4>(a, sm_count, s) : launch_t<float, 1>(a, sm_count, s);
    case DType::BF16:
        return a.vec ? launch_t<__nv_bfloat16, 8>(a, sm_count, s) : launch_t<__nv_bfloat16, 1>(a, sm_count, s);
    case DType::F16: return a.vec ? launch_t<__half, 8>(a, sm_count, s) : launch_t<__half, 1>(a, sm_count, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace gdn
