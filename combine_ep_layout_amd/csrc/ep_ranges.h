// Host checks of pointers: alignment, and whether arrays share memory.  Not
// installed; callers use include/ep_layout.h.
#pragma once

#include <stdint.h>
#include <algorithm>
#include <vector>

namespace epk {
namespace {

inline bool aligned(const void* p, int n) { return ((uintptr_t)p & (uintptr_t)(n - 1)) == 0; }

// n rows of `width` bytes, `ld` bytes apart.
struct Rows {
    uintptr_t at;
    __int128 ld, width, n;
    Rows(const void* p, int64_t ld_, int64_t width_, int64_t n_, int size)
        : at((uintptr_t)p), ld((__int128)ld_ * size), width((__int128)width_ * size), n(n_) {
        if (n == 1 || ld == width) {            // one piece
            width *= n;
            ld = width;
            n = 1;
        }
    }
    __int128 row(__int128 i) const { return (__int128)at + i * ld; }
    // whether a row shares a byte with [p, q)
    bool meets(__int128 p, __int128 q) const {
        const __int128 i = p < row(0) + width ? 0 : (p - row(0) - width) / ld + 1;      // the first row that ends behind p
        return i < n && row(i) < q;
    }
    bool meets_row(const Rows& o, __int128 i) const { return meets(o.row(i), o.row(i) + o.width); }
};

// Whether two arrays share a byte: column slices of one buffer lie between each
// other's rows and share none.
inline bool share(const Rows& a, const Rows& b) {
    if (a.row(a.n - 1) + a.width <= b.at || b.row(b.n - 1) + b.width <= a.at) return false;
    // equal strides: where rows i and j meet, rows i - m and j - m do, and with m the smaller one is row 0
    if (a.ld == b.ld) return a.meets_row(b, 0) || b.meets_row(a, 0);
    const Rows& few = a.n < b.n ? a : b;
    const Rows& many = a.n < b.n ? b : a;
    for (__int128 i = 0; i < few.n; ++i)
        if (many.meets_row(few, i)) return true;
    return false;
}

// Bytes [at, end) of one buffer of many.
struct Range {
    uintptr_t at, end;
    bool wrote;
    bool operator<(const Range& o) const { return at < o.at; }
};

// Merges the ranges from `from` on, one kind of buffer of every tensor, into
// those before.  A kind mostly lies in memory in the list's order, and is only
// merged then: the checks of 300 tensors take 11.3 us on the host, 12.2 with one
// sort of them all; out of order 15.8 and 15.2.
inline void merge_in(std::vector<Range>& r, size_t from) {
    const auto mid = r.begin() + (std::ptrdiff_t)from;
    if (!std::is_sorted(mid, r.end())) std::sort(mid, r.end());
    std::inplace_merge(r.begin(), mid, r.end());
}

// Whether a buffer that is written shares memory with another buffer (r in order).
inline bool shared(const std::vector<Range>& r) {
    uintptr_t any = 0, written = 0;         // furthest end so far, of all and of those written
    for (const Range& x : r) {
        if (x.at < written || (x.wrote && x.at < any)) return true;
        any = std::max(any, x.end);
        if (x.wrote) written = std::max(written, x.end);
    }
    return false;
}

}  // namespace
}  // namespace epk
