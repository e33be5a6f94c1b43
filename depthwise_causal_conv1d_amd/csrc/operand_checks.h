// Checks of operands that the state-space, delta-rule and norm entry points share
// (internal): spans, addresses, alignment and overlaps, element types.
#pragma once

#include "abi_common.h"

namespace dcconv {
namespace abi {

// Bytes from an array's first element to its last: extents e at element strides
// st, `inner` dense elements behind them.  False when that passes 2^47 bytes.
inline bool extent(const int64_t (&e)[3], const int64_t (&st)[3], int64_t inner, int64_t elem, int64_t *bytes) {
    *bytes = 0;
    int64_t last = 0;
    const int64_t most = ((int64_t)1 << 47) / elem;
    if (inner <= 0) return true;
    if (inner > most) return false;
    for (int i = 0; i < 3; ++i)
        if (e[i] <= 0) return true;
    for (int i = 0; i < 3; ++i) {
        int64_t term;
        if (__builtin_mul_overflow(e[i] - 1, st[i], &term) || term > most) return false;
        last += term;
        if (last > most) return false;
    }
    if (last + inner > most) return false;
    *bytes = elem * (last + inner);
    return true;
}

// Whether rows of `inner` dense elements at extents e and strides st are disjoint.
inline bool rows_distinct(const int64_t (&e)[3], const int64_t (&st)[3], int64_t inner) {
    int order[3] = {0, 1, 2};
    for (int i = 1; i < 3; ++i)
        for (int j = i; j > 0 && st[order[j]] < st[order[j - 1]]; --j) {
            const int t = order[j];
            order[j] = order[j - 1];
            order[j - 1] = t;
        }
    int64_t below = inner;
    for (int i = 0; i < 3; ++i) {
        const int q = order[i];
        if (e[q] <= 1) continue;
        if (st[q] < below) return false;
        below += st[q] * (e[q] - 1);
    }
    return true;
}

struct Operand {
    const char *name;
    const void *ptr;
    int64_t bytes, align;
    bool written;
};

// Alignment of every operand, and none written that overlaps another.
template <int N>
inline int check_operands(const Operand (&ops)[N]) {
    for (const Operand &o : ops)
        if (o.ptr != nullptr && !aligned(o.ptr, (uintptr_t)o.align))
            return fail(DCCONV_EINVAL, "%s must be %lld-byte aligned", o.name, (long long)o.align);
    for (int i = 0; i < N; ++i)
        for (int j = 0; j < N; ++j)
            if (i != j && ops[i].written &&
                overlaps(span(ops[i].name, ops[i].ptr, ops[i].bytes), span(ops[j].name, ops[j].ptr, ops[j].bytes)))
                return fail(DCCONV_EINVAL, "%s overlaps %s", ops[i].name, ops[j].name);
    return DCCONV_OK;
}

inline bool known_dtype(int dtype) { return dtype == DCCONV_DTYPE_BF16 || dtype == DCCONV_DTYPE_F32; }
inline int64_t dtype_bytes(int dtype) { return dtype == DCCONV_DTYPE_F32 ? 4 : 2; }

template <int N>
inline bool any_negative(const int64_t (&v)[N]) {
    for (int64_t x : v)
        if (x < 0) return true;
    return false;
}

// A slot stride, h*p*k elements behind it; false past 2^47 bytes.
inline bool state_extent(int64_t s, int64_t ss_s, int64_t inner, int dtype, int64_t *bytes) {
    return extent({s, 1, 1}, {ss_s, 0, 0}, inner, dtype_bytes(dtype), bytes);
}

}  // namespace abi
}  // namespace dcconv
