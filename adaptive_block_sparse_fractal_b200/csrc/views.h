// Host arithmetic of strided views: what a view spans, and whether two views, or
// two rows of one, share memory.  Plain C++, no CUDA.
#pragma once

#include <algorithm>
#include <cstdint>

#include "../../include/nabla.h"

namespace nabla {
namespace views {

constexpr int64_t kMaxExtent = 1ll << 46;  // bytes a view may span: keeps the arithmetic in 64 bits

// Rows of `row` bytes at lo + sum of index * step over [batch, head, token].
struct Box {
    int64_t n[3], stride[3], step[3];  // extents, distances in elements and bytes (0 where the extent is 1)
    int64_t row, size;                 // bytes of a row and of an element
    uintptr_t lo, hi;                  // bytes it spans: [lo, hi), empty if equal
};

// Extents and span of [B, heads, tokens, D] elements of `size` bytes; false for
// negative distances or a span beyond kMaxExtent.  Without elements it is empty.
inline bool make_box(const nabla_view *v, int64_t B, int64_t heads, int64_t tokens, int64_t D, int size,
                     Box *b) {
    const int64_t n[3] = {B, heads, tokens}, s[3] = {v->batch, v->head, v->token};
    const bool none = B == 0 || heads == 0 || tokens == 0;
    int64_t last = D;
    for (int i = 0; i < 3; ++i) {
        b->n[i] = none ? 1 : n[i];
        b->stride[i] = b->n[i] > 1 ? s[i] : 0;
        if (b->stride[i] < 0 || b->stride[i] > kMaxExtent) return false;
        if (b->n[i] > 1 && b->stride[i] > kMaxExtent / b->n[i]) return false;
        b->step[i] = b->stride[i] * size;
        last += (b->n[i] - 1) * b->stride[i];
    }
    if (last > kMaxExtent / size) return false;
    b->row = D * size;
    b->size = size;
    b->lo = reinterpret_cast<uintptr_t>(v->data);
    b->hi = b->lo + (none ? 0 : static_cast<uintptr_t>(last) * size);
    return true;
}

// `bytes` bytes in a row
inline Box flat(const void *p, int64_t bytes) {
    Box b = {};
    for (int i = 0; i < 3; ++i) b.n[i] = 1;
    b.row = p == nullptr ? 0 : bytes;
    b.size = 1;
    b.lo = reinterpret_cast<uintptr_t>(p);
    b.hi = b.lo + static_cast<uintptr_t>(b.row);
    return b;
}

inline bool multiple_of_16(const Box &b) {
    return (b.lo & 15u) == 0 && b.step[0] % 16 == 0 && b.step[1] % 16 == 0 && b.step[2] % 16 == 0;
}

// step * x for x in [lo, hi]
struct Term {
    int64_t step, lo, hi;
};

// Whether some choice of every term's x puts their sum into [from, to].  Terms come by
// falling step.  Where each step clears what lies inside it, as in any slice of a
// tensor, a term has two or three candidates; `work` bounds the search for others, and
// running out of it counts as yes.
inline bool reaches(const Term *t, int n, int64_t from, int64_t to, int *work) {
    if (n == 0) return from <= 0 && 0 <= to;
    if (--*work < 0) return true;
    int64_t least = 0, most = 0;  // of the terms behind this one
    for (int i = 1; i < n; ++i) {
        least += t[i].step * t[i].lo;
        most += t[i].step * t[i].hi;
    }
    auto floor_div = [](int64_t a, int64_t b) { return a / b - (a % b < 0); };
    const int64_t x0 = std::max(t->lo, -floor_div(most - from, t->step)), x1 = std::min(t->hi, floor_div(to - least, t->step));
    if (n == 1) return x0 <= x1;
    for (int64_t x = x0; x <= x1; ++x)
        if (reaches(t + 1, n - 1, from - t->step * x, to - t->step * x, work)) return true;
    return false;
}

constexpr int kSearch = 4096;

// Terms of a box's dimensions, merged into those that are there already with the same
// step; `sign` is that of the indices.
inline int add_terms(const Box &b, int sign, Term *t, int n) {
    for (int i = 0; i < 3; ++i) {
        if (b.n[i] == 1 || b.step[i] == 0) continue;
        int at = 0;
        while (at < n && t[at].step != b.step[i]) ++at;
        if (at == n) t[n++] = {b.step[i], 0, 0};
        (sign > 0 ? t[at].hi : t[at].lo) += sign * (b.n[i] - 1);
    }
    return n;
}

inline bool by_step(const Term &a, const Term &b) { return a.step > b.step; }

// Whether two views share no byte, where the bytes that they span do.
inline bool rows_apart(const Box &a, const Box &b) {
    Term t[6];
    const int n = add_terms(b, -1, t, add_terms(a, 1, t, 0));
    std::sort(t, t + n, by_step);
    // a row of a begins `d` bytes behind one of b: they meet for -a.row < d < b.row
    const int64_t first = a.lo >= b.lo ? static_cast<int64_t>(a.lo - b.lo) : -static_cast<int64_t>(b.lo - a.lo);
    int work = kSearch;
    return !reaches(t, n, 1 - a.row - first, b.row - 1 - first, &work);
}
// Whether two views share no byte.
inline bool disjoint(const Box &a, const Box &b) {
    return a.lo == a.hi || b.lo == b.hi || a.hi <= b.lo || b.hi <= a.lo || rows_apart(a, b);
}

// Whether no two rows of a view share a byte (one that is written must not).
inline bool self_disjoint(const Box &b) {
    Term t[3];
    int n = 0;
    for (int i = 0; i < 3; ++i) {
        if (b.n[i] == 1) continue;
        if (b.step[i] == 0) return false;
        t[n++] = {b.step[i], 1 - b.n[i], b.n[i] - 1};
    }
    std::sort(t, t + n, by_step);
    // commonly each step clears what lies inside it
    int64_t inner = b.row;
    int i = n - 1;
    for (; i >= 0 && t[i].step >= inner; --i) inner += t[i].hi * t[i].step;
    if (i < 0) return true;
    // two rows differ first in dimension i, there by a positive number of steps
    int work = kSearch;
    for (i = 0; i < n; ++i) {
        Term d[3];
        std::copy(t + i, t + n, d);
        d[0].lo = 1;
        if (reaches(d, n - i, 1 - b.row, b.row - 1, &work)) return false;
    }
    return true;
}

inline bool same_view(const Box &a, const Box &b) {
    return a.lo == b.lo && a.stride[0] == b.stride[0] && a.stride[1] == b.stride[1] &&
           a.stride[2] == b.stride[2];
}

}  // namespace views
}  // namespace nabla
