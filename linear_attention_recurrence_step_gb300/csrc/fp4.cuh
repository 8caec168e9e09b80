// fp4.cuh -- the cache's values: groups of 16 elements with one e4m3 scale and
// e2m1 codes (0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign).  A code has two
// significant bits and a scale four, so their product (2^-10 to 2688) is exact
// in f16: the matrix products over the cache take exact operands.
//
// A page of one head is one block: the keys' codes [page, D/2 bytes] (element
// 2i in the low half of byte i), the keys' scales [page, D/16], then the
// values' codes and scales.
#pragma once

#include "common.cuh"

namespace gdn {

// Four bytes, the i-th with codes (lo, hi), as four f16 pairs.
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&h)[4]) {
    asm("{\n.reg .b8 b0, b1, b2, b3;\n"
        "mov.b32 {b0, b1, b2, b3}, %4;\n"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\ncvt.rn.f16x2.e2m1x2 %1, b1;\n"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\ncvt.rn.f16x2.e2m1x2 %3, b3;\n}\n"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}
// Two e4m3 bytes (bits 0-7, 8-15) as an f16 pair.
__device__ __forceinline__ uint32_t e4m3x2_to_f16(uint32_t w) {
    uint32_t h;
    asm("{\n.reg .b16 s;\ncvt.u16.u32 s, %1;\ncvt.rn.f16x2.e4m3x2 %0, s;\n}\n" : "=r"(h) : "r"(w));
    return h;
}
__device__ __forceinline__ float f16_lo(uint32_t h) {
    return __low2float(*reinterpret_cast<const __half2 *>(&h));
}
__device__ __forceinline__ float f16_hi(uint32_t h) {
    return __high2float(*reinterpret_cast<const __half2 *>(&h));
}
// The nearest e4m3 of x >= 0 (ties to even, at most 448).
__device__ __forceinline__ uint32_t f32_to_e4m3(float x) {
    uint32_t r;
    asm("{\n.reg .b16 s;\ncvt.rn.satfinite.e4m3x2.f32 s, %1, %1;\ncvt.u32.u16 %0, s;\n}\n" : "=r"(r) : "f"(x));
    return r & 0xffu;
}
// The nearest e2m1 codes (ties to even, at most 6) of two values: bits 0-3
// and 4-7.
__device__ __forceinline__ uint32_t f32_to_e2m1x2(float lo, float hi) {
    uint32_t r;
    asm("{\n.reg .b8 b, z;\nmov.b32 {z, z, z, z}, 0;\ncvt.rn.satfinite.e2m1x2.f32 b, %1, %2;\n"
        "mov.b32 %0, {b, z, z, z};\n}\n"
        : "=r"(r)
        : "f"(hi), "f"(lo));
    return r;
}

}  // namespace gdn
