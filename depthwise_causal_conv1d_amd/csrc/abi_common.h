// What the files of the C-ABI front end share (internal): the calling thread's
// error and kernel name, and the checks of operands' extents and overlaps.
#pragma once

#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>

#include "dcconv.h"

namespace dcconv {
namespace abi {

inline thread_local char g_error[512];
inline thread_local const char *g_kernel = "";

inline int fail(int code, const char *fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_error, sizeof g_error, fmt, ap);
    va_end(ap);
    g_kernel = "";
    return code;
}

inline int succeed(const char *kernel) {
    g_error[0] = '\0';
    g_kernel = kernel;
    return DCCONV_OK;
}

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// A byte range [lo, hi) of one operand, for the overlap checks.
struct Span {
    const char *name;
    uintptr_t lo, hi;
};

inline Span span(const char *name, const void *p, int64_t bytes) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return Span{name, lo, p ? lo + (uintptr_t)(bytes > 0 ? bytes : 0) : lo};
}

inline bool overlaps(const Span &a, const Span &b) {
    return a.hi > a.lo && b.hi > b.lo && a.lo < b.hi && b.lo < a.hi;
}

constexpr int64_t kI32Max = 2147483647;

// Bytes spanned by an [e0, e1, e2] BF16 array at element strides st (strides
// >= 0): 2 * (sum (e_i - 1) * st_i + 1), or 0 for an empty array.  False when
// the span overflows or exceeds 2^47 bytes, more than any device address space.
inline bool span_bytes(const int64_t e[3], const int64_t st[3], int64_t *bytes) {
    const int64_t kMaxElems = (int64_t)1 << 46;
    int64_t last = 0;
    for (int i = 0; i < 3; ++i)
        if (e[i] <= 0) {
            *bytes = 0;
            return true;
        }
    for (int i = 0; i < 3; ++i) {
        int64_t term;
        if (__builtin_mul_overflow(e[i] - 1, st[i], &term) || term > kMaxElems) return false;
        last += term;
        if (last > kMaxElems) return false;
    }
    *bytes = 2 * (last + 1);
    return true;
}

// True when no two elements of an [e0, e1, e2] array at strides s0, s1, s2 share
// an address: sorted by stride, each dimension must step over the whole extent of
// the ones below it.
inline bool strides_distinct(const int64_t e[3], const int64_t st[3]) {
    int64_t ext[3], str[3];
    int k = 0;
    for (int i = 0; i < 3; ++i)
        if (e[i] > 1) {
            ext[k] = e[i];
            str[k] = st[i];
            ++k;
        }
    for (int i = 1; i < k; ++i)
        for (int j = i; j > 0 && str[j] < str[j - 1]; --j) {
            const int64_t te = ext[j], ts = str[j];
            ext[j] = ext[j - 1];
            str[j] = str[j - 1];
            ext[j - 1] = te;
            str[j - 1] = ts;
        }
    int64_t span_below = 1;
    for (int i = 0; i < k; ++i) {
        if (str[i] < span_below) return false;
        span_below = str[i] * (ext[i] - 1) + span_below;
    }
    return true;
}

}  // namespace abi
}  // namespace dcconv
