// abi_util.h -- argument checks and error reporting shared by the C entry
// points (abi.cu, layer_abi.cu).  Everything here runs on the host before
// anything is enqueued.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <initializer_list>

#include "gdn.h"

namespace gdn {
namespace abi {

// Record a message for gdn_last_error() and return `st` (defined in abi.cu,
// as is the per-thread message itself).
gdn_status fail(gdn_status st, const char *fmt, ...);
gdn_status ok();
gdn_status cuda_fail(const char *fn, const char *what, cudaError_t e);

// Testing hook gdn_force_launch_failures: consume one forced failure.
bool take_forced_failure();
gdn_status forced_failure(const char *fn);

// SM count of the current device (0 if it cannot be read).
int current_sm_count(cudaError_t *err);

inline bool mul_ok(int64_t a, int64_t b, int64_t *out) { return !__builtin_mul_overflow(a, b, out); }

// Product of dims (all > 0) times elem_bytes, or -1 on overflow.
inline int64_t nbytes(std::initializer_list<int64_t> dims, int64_t elem_bytes) {
    int64_t acc = elem_bytes;
    for (int64_t d : dims)
        if (!mul_ok(acc, d, &acc)) return -1;
    return acc;
}

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline bool overlap(const void *a, int64_t na, const void *b, int64_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + (uintptr_t)nb && y < x + (uintptr_t)na;
}

inline int elem_bytes(gdn_dtype dt) {
    switch (dt) {
    case GDN_DTYPE_F32: return 4;
    case GDN_DTYPE_BF16: return 2;
    case GDN_DTYPE_F16: return 2;
    }
    return 0;
}

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Elements from the first to the last of a [n0,n1,inner] tensor whose first
// two strides are given (inner dense; either of them may be the outer one), or
// -1: strides that do not keep its rows apart, or an overflow.
inline int64_t extent(int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t inner) {
    if (s1 < 0 || s0 < 0) return -1;
    int64_t e0, e1, e;
    if (!mul_ok(n0 - 1, s0, &e0) || !mul_ok(n1 - 1, s1, &e1)) return -1;
    if (__builtin_add_overflow(e0, e1, &e) || __builtin_add_overflow(e, inner, &e)) return -1;
    const bool first_outer = (n0 == 1 || s0 >= e1 + inner) && (n1 == 1 || s1 >= inner);
    const bool second_outer = (n0 == 1 || s0 >= inner) && (n1 == 1 || s1 >= e0 + inner);
    return first_outer || second_outer ? e : -1;
}

inline bool over(const void *a, int64_t na, const void *b, int64_t nb) { return a && b && overlap(a, na, b, nb); }

inline int64_t scaled(int64_t elems, int eb) {
    int64_t out;
    return elems >= 0 && mul_ok(elems, eb, &out) ? out : -1;
}

}  // namespace abi
}  // namespace gdn
