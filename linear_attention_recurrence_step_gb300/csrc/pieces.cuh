// pieces.cuh -- loads and stores of VEC neighbouring elements as f32, and the
// gate function, shared by the operators around the recurrence.  A piece of
// 16 bytes is one vector access (its address is 16-byte aligned); others go
// element by element.
#pragma once

#include "common.cuh"

namespace gdn {

// Two neighbouring elements from one 32-bit word, and back.
template <typename T> __device__ __forceinline__ float2 unpack2(uint32_t w);
template <> __device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t w) {
    // bf16 -> f32 is exact: the bf16 bits are the top half of the f32 bits
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <> __device__ __forceinline__ float2 unpack2<__half>(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}
template <typename T> __device__ __forceinline__ uint32_t pack2(float a, float b);
template <> __device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
template <> __device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// The raw bits of a piece, so that loads can be issued ahead of their use.
template <typename T, int VEC> struct RawPiece;
template <> struct RawPiece<float, 4> { uint4 w; };
template <> struct RawPiece<__nv_bfloat16, 8> { uint4 w; };
template <> struct RawPiece<__half, 8> { uint4 w; };
template <> struct RawPiece<float, 1> { float w; };
template <> struct RawPiece<__nv_bfloat16, 1> { __nv_bfloat16 w; };
template <> struct RawPiece<__half, 1> { __half w; };

template <typename T, int VEC>
__device__ __forceinline__ RawPiece<T, VEC> load_raw(const T *p) {
    RawPiece<T, VEC> r;
    if constexpr (VEC == 1) r.w = *p;
    else r.w = *reinterpret_cast<const uint4 *>(p);
    return r;
}

template <typename T, int VEC>
__device__ __forceinline__ void store_raw(T *p, const RawPiece<T, VEC> &r) {
    if constexpr (VEC == 1) *p = r.w;
    else *reinterpret_cast<uint4 *>(p) = r.w;
}

template <typename T, int VEC>
__device__ __forceinline__ void widen(float (&v)[VEC], const RawPiece<T, VEC> &r) {
    if constexpr (VEC == 1) {
        v[0] = Elem<T>::to_f32(r.w);
    } else if constexpr (sizeof(T) == 4) {
        v[0] = __uint_as_float(r.w.x);
        v[1] = __uint_as_float(r.w.y);
        v[2] = __uint_as_float(r.w.z);
        v[3] = __uint_as_float(r.w.w);
    } else {
        const uint32_t w[4] = {r.w.x, r.w.y, r.w.z, r.w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = unpack2<T>(w[i]);
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    }
}

template <typename T, int VEC>
__device__ __forceinline__ void load_piece(float (&v)[VEC], const T *p) {
    widen<T, VEC>(v, load_raw<T, VEC>(p));
}

// f32 values rounded to the type.
template <typename T, int VEC>
__device__ __forceinline__ RawPiece<T, VEC> narrow_piece(const float (&v)[VEC]) {
    RawPiece<T, VEC> r;
    if constexpr (VEC == 1) {
        r.w = Elem<T>::from_f32(v[0]);
    } else if constexpr (sizeof(T) == 4) {
        r.w = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    } else {
        r.w = make_uint4(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]), pack2<T>(v[4], v[5]), pack2<T>(v[6], v[7]));
    }
    return r;
}

template <typename T, int VEC>
__device__ __forceinline__ void store_piece(T *p, const float (&v)[VEC]) {
    store_raw<T, VEC>(p, narrow_piece<T, VEC>(v));
}

__device__ __forceinline__ float ex2f(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcpf(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// x * sigmoid(x), within a few units in the last place (the exponential's
// argument costs |x| of them).  exp overflowing to infinity gives the limit,
// -0.  The two-lane form takes one packed instruction for both where there is
// one.
__device__ __forceinline__ float silu(float x) { return x * rcpf(1.f + ex2f(-1.44269504088896341f * x)); }
__device__ __forceinline__ float2 silu2(float2 x) {
    const float2 t = fmul2(x, make_float2(-1.44269504088896341f, -1.44269504088896341f));
    const float2 d = __fadd2_rn(make_float2(ex2f(t.x), ex2f(t.y)), make_float2(1.f, 1.f));
    return fmul2(x, make_float2(rcpf(d.x), rcpf(d.y)));
}

// A piece as pairs (a single element: the first of a pair, beside a zero).
template <int VEC> constexpr int kPairs = (VEC + 1) / 2;
template <typename T, int VEC>
__device__ __forceinline__ void widen2(float2 (&v)[kPairs<VEC>], const RawPiece<T, VEC> &r) {
    float f[VEC];
    widen<T, VEC>(f, r);
#pragma unroll
    for (int i = 0; i < kPairs<VEC>; ++i) v[i] = make_float2(f[2 * i], 2 * i + 1 < VEC ? f[(2 * i + 1) % VEC] : 0.f);
}
template <typename T, int VEC>
__device__ __forceinline__ void store_piece2(T *p, const float2 (&v)[kPairs<VEC>]) {
    float f[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) f[i] = i % 2 ? v[i / 2].y : v[i / 2].x;
    store_piece<T, VEC>(p, f);
}

}  // namespace gdn
