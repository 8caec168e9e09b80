// rotary.cu -- rotary positions of queries and keys.
//
// Pair i of a head is turned by the angle position * inv_freq[i].  Far
// positions leave nothing of such an angle's fraction in float32, so it is
// counted in turns with 64 fixed-point bits: F = frac(inv_freq / 2 pi) 2^64
// once per frequency (one double product), position * F modulo 2^64 drops the
// whole turns by itself, and the upper 32 bits are the fraction, off by 2^-32
// of a turn and 2^-53 of inv_freq per step at most.
//
// Every element is read once and written once: 84 MB of 4096 tokens of 40 heads of 128
// in 15.6 us from and to L2, 20.8 with cold caches (4.0 TB/s; 12.4 by the bytes), bound by
// waits for a token's position and sines in front of its loads.  A block makes the sines
// of its tokens once, in shared memory, and uses them for all heads of q and k; a thread
// takes the same piece of all of the block's tokens, so that where it lies in a token is
// worked out once and their loads are in flight together.
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

// TB tokens per block.
template <typename T, int VEC, bool HALF, int TB>
__global__ void __launch_bounds__(kRotThreads) rotary_kernel(const RotaryArgs a) {
    extern __shared__ float2 cs[];  // [TB][R/2]
    __shared__ int pos[TB];
    __shared__ int64_t off[TB][4];  // a token's offsets in q, k, q_out and k_out
    pdl_trigger();
    pdl_wait();
    const int n = a.R / 2;
    const int64_t tok0 = (int64_t)blockIdx.x * TB, all = a.B * a.T;
    if (threadIdx.x < TB) {
        const int64_t tok = tok0 + threadIdx.x, b = tok / a.T, t = tok - b * a.T;
        pos[threadIdx.x] = tok < all ? a.positions[tok] : -1;
        off[threadIdx.x][0] = b * a.q_sb + t * a.q_st;
        off[threadIdx.x][1] = b * a.k_sb + t * a.k_st;
        off[threadIdx.x][2] = b * a.qo_sb + t * a.qo_st;
        off[threadIdx.x][3] = b * a.ko_sb + t * a.ko_st;
    }
    __syncthreads();
    for (int f = threadIdx.x; f < n; f += kRotThreads) {
        double per = (double)a.inv_freq[f] * 0.15915494309189533577;
        per -= floor(per);
        const unsigned long long F = __double2ull_rn(per * 18446744073709551616.0);
#pragma unroll
        for (int k = 0; k < TB; ++k)
            cs[k * n + f] = turn((int32_t)(((unsigned long long)(unsigned)max(pos[k], 0) * F) >> 32), a.scale, a.inverse);
    }
    __syncthreads();
    // units of a head: pieces of pairs (VEC elements of each half, or VEC
    // neighbouring elements), then pieces that stay as they are
    constexpr int PAIRS = HALF ? VEC : VEC / 2 + (VEC == 1);
    constexpr int SECOND = HALF || VEC == 1;  // a unit has two pieces
    const int turned = n / PAIRS, rest = (a.D - a.R) / VEC, units = turned + rest;
    const int heads = a.Hq + (a.k ? a.Hk : 0);
    for (int i = threadIdx.x; i < heads * units; i += kRotThreads) {
        const int h = i / units, u = i - h * units;
        const bool key = h >= a.Hq, turns = u < turned;
        const int64_t head = (int64_t)(key ? h - a.Hq : h) * a.D;
        const T *src = static_cast<const T *>(key ? a.k : a.q) + head;
        T *dst = static_cast<T *>(key ? a.k_out : a.q_out) + head;
        const int d0 = !turns ? a.R + (u - turned) * VEC : HALF ? u * VEC : VEC == 1 ? 2 * u : u * VEC;
        const int d1 = HALF ? d0 + n : d0 + 1;
        RawPiece<T, VEC> x0[TB], x1[TB];
#pragma unroll
        for (int k = 0; k < TB; ++k)
            if (pos[k] >= 0) {
                const T *p = src + off[k][key];
                x0[k] = load_raw<T, VEC>(p + d0);
                if (SECOND && turns) x1[k] = load_raw<T, VEC>(p + d1);
            }
#pragma unroll
        for (int k = 0; k < TB; ++k) {
            if (pos[k] < 0) continue;
            T *q = dst + off[k][2 + key];
            if (!turns) {
                if (q != src + off[k][key]) store_raw<T, VEC>(q + d0, x0[k]);
                continue;
            }
            const float2 *w = cs + k * n + u * PAIRS;
            float x[VEC];
            widen<T, VEC>(x, x0[k]);
            if constexpr (SECOND) {
                float y[VEC];
                widen<T, VEC>(y, x1[k]);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float2 c = w[e];
                    const float p = x[e] * c.x - y[e] * c.y;
                    y[e] = x[e] * c.y + y[e] * c.x;
                    x[e] = p;
                }
                store_piece<T, VEC>(q + d1, y);
            } else {
#pragma unroll
                for (int e = 0; e < VEC; e += 2) {
                    const float2 c = w[e / 2];
                    const float p = x[e] * c.x - x[e + 1] * c.y;
                    x[e + 1] = x[e] * c.y + x[e + 1] * c.x;
                    x[e] = p;
                }
            }
            store_piece<T, VEC>(q + d0, x);
        }
    }
}

template <typename T, int VEC, int TB>
cudaError_t launch_tb(const RotaryArgs &a, cudaStream_t s) {
    const int64_t blocks = (a.B * a.T + TB - 1) / TB;
    if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
    const size_t smem = (size_t)TB * (a.R / 2) * sizeof(float2);
    return a.half ? launch_dependent(rotary_kernel<T, VEC, true, TB>, (unsigned)blocks, kRotThreads, smem, s, a)
                  : launch_dependent(rotary_kernel<T, VEC, false, TB>, (unsigned)blocks, kRotThreads, smem, s, a);
}

// Four tokens per block once blocks of one fill the SMs some four times over (and
// their sines fit the shared memory that needs no asking).  40 heads of 128: 2048
// tokens 8.8 us with one per block, 10.2 with four; 4096 15.3 and 16.7; 8192 34.6 and
// 30.2; 16384 64.2 and 55.7.  Measured on such wide tokens: of 5 heads, which leave most
// of a block idle, 4864 tokens take 12.1 us with one per block and 4865 7.6 with four.
template <typename T, int VEC>
cudaError_t launch_t(const RotaryArgs &a, int sm_count, cudaStream_t s) {
    const bool many = a.B * a.T > (int64_t)(sm_count > 0 ? sm_count : 152) * 32 && a.R <= 2048;
    return many ? launch_tb<T, VEC, 4>(a, s) : launch_tb<T, VEC, 1>(a, s);
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
