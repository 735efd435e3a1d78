// la_views.h -- host checks of strided operands shared by the entry points whose operands differ in their
// extents (grouped heads, packed sequences, channel blocks): layout rules and overlaps.
#pragma once

#include <stdint.h>

#include "../../include/la.h"

namespace la {

// An operand: rows of `width` contiguous elements, stepped by three dimensions of the given extents and
// element strides (a dimension of extent 1 is never stepped).
struct View {
    const void *p;
    long long ext[3], st[3];
    long long width;
    int elem;  // bytes
};

// Sets v's strides from the caller's (nullptr: `dense`, the contiguous ones) and checks them: each a multiple of
// 16 bytes, and the rows not overlapping one another (ordered by stride, the dimensions of extent > 1 nest).
inline int set_view(View &v, const long long *given, const long long *dense) {
    for (int k = 0; k < 3; ++k) {
        v.st[k] = given ? given[k] : dense[k];
        if (v.ext[k] == 1) v.st[k] = v.width;
        if (v.st[k] < 1 || v.st[k] >= (1LL << 40) / v.elem) return LA_ERR_INVALID_ARG;
        if (v.ext[k] > 1 && (v.st[k] * v.elem) % 16 != 0) return LA_ERR_INVALID_ARG;
    }
    int idx[3] = {0, 1, 2};
    for (int a = 0; a < 3; ++a)
        for (int b = a + 1; b < 3; ++b)
            if (v.st[idx[b]] < v.st[idx[a]]) { const int t = idx[a]; idx[a] = idx[b]; idx[b] = t; }
    long long need = v.width;
    for (int k = 0; k < 3; ++k) {
        const int d = idx[k];
        if (v.ext[d] == 1) continue;
        if (v.st[d] < need) return LA_ERR_INVALID_ARG;
        need = v.st[d] * v.ext[d];
    }
    return LA_OK;
}

// Bytes from a view's base to one past its last element (0 when it has no rows).
inline size_t view_bytes(const View &v) {
    long long n = v.width;
    for (int k = 0; k < 3; ++k) {
        if (v.ext[k] < 1) return 0;
        n += (v.ext[k] - 1) * v.st[k];
    }
    return (size_t)n * v.elem;
}

inline bool ranges_meet(const void *a, size_t an, const void *b, size_t bn) {
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return an && bn && x < y + bn && y < x + an;
}

// Whether delta = sum_k i_k st_k + d for some i_k in [lo_k, hi_k] and |d| < width; st in decreasing order and
// nested, so at each level only the quotients next to delta / st can work.
__attribute__((noinline)) static bool steps_meet(long long delta, const long long *st, const long long *lo, const long long *hi, int n,
                       long long width) {
    if (n == 0) return delta > -width && delta < width;
    const long long q = delta / st[0];
    for (long long c = q - 2; c <= q + 2; ++c)
        if (c >= lo[0] && c <= hi[0] && steps_meet(delta - c * st[0], st + 1, lo + 1, hi + 1, n - 1, width)) return true;
    return false;
}

// Whether two views share an element.  Exact for views of equal strides (slices of one tensor, whatever their
// extents); views of other strides whose address ranges meet count as sharing.
inline bool views_meet(const View &a, const View &b) {
    if (!ranges_meet(a.p, view_bytes(a), b.p, view_bytes(b))) return false;
    if (a.elem != b.elem || a.width != b.width) return true;
    // the stride of a dimension that only one of them steps is that one's; of one that neither does, 0
    long long st[3] = {}, lo[3] = {}, hi[3] = {};
    int n = 0;
    for (int k = 0; k < 3; ++k) {
        if (a.ext[k] == 1 && b.ext[k] == 1) continue;
        if (a.ext[k] > 1 && b.ext[k] > 1 && a.st[k] != b.st[k]) return true;
        st[k] = a.ext[k] > 1 ? a.st[k] : b.st[k];
        lo[k] = -(b.ext[k] - 1);
        hi[k] = a.ext[k] - 1;
        ++n;
    }
    auto order = [&](int x, int y) {
        if (st[y] <= st[x]) return;
        long long t;
        t = st[x], st[x] = st[y], st[y] = t;
        t = lo[x], lo[x] = lo[y], lo[y] = t;
        t = hi[x], hi[x] = hi[y], hi[y] = t;
    };
    order(0, 1), order(1, 2), order(0, 1);  // by decreasing stride
    for (int x = 0; x < n; ++x) {  // the two together have to nest for the search below; else refuse
        long long inner = a.width;
        if (x + 1 < n) inner = st[x + 1] * ((hi[x + 1] > -lo[x + 1] ? hi[x + 1] : -lo[x + 1]) + 1);
        if (st[x] < inner) return true;
    }
    const long long diff = (long long)((uintptr_t)b.p - (uintptr_t)a.p);
    if (diff % a.elem != 0) return true;
    return steps_meet(diff / a.elem, st, lo, hi, n, a.width);
}

inline bool same_view(const View &a, const View &b) {
    return a.p == b.p && a.st[0] == b.st[0] && a.st[1] == b.st[1] && a.st[2] == b.st[2];
}

}  // namespace la
