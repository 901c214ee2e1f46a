// gdn_checks.cuh -- argument checks of the entry points for linear-attention sequences and rotary positions.
#pragma once

#include "gdn_seq.cuh"

namespace gdn {
namespace check {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool given(const void* p) { return p != nullptr && aligned16(p); }
// gates, indices and positions are read one by one: any row of a larger tensor will do
inline bool words(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
inline bool given_words(const void* p) { return p != nullptr && words(p); }
inline bool type_ok(int dtype) { return dtype == GDN_DTYPE_BF16 || dtype == GDN_DTYPE_F32; }
inline bool dim_ok(int d) { return d >= 16 && d <= kMaxDim && d % 16 == 0; }

struct Span {
    const void* p;
    size_t n;
};
inline bool overlap(const Span& a, const Span& b) {
    if (a.p == nullptr || b.p == nullptr || a.n == 0 || b.n == 0) return false;
    const char *x = static_cast<const char*>(a.p), *y = static_cast<const char*>(b.p);
    return x < y + b.n && y < x + a.n;
}
// No written span may meet a read one or another written one.
inline bool disjoint(const Span* w, int nw, const Span* r, int nr) {
    for (int i = 0; i < nw; ++i) {
        for (int j = i + 1; j < nw; ++j)
            if (overlap(w[i], w[j])) return false;
        for (int j = 0; j < nr; ++j)
            if (overlap(w[i], r[j])) return false;
    }
    return true;
}
// Bytes from the first to the last element of `total` rows of `row` elements, `ld` apart.
inline size_t strided_bytes(long long total, long long ld, long long row, int e) {
    return total == 0 ? 0 : (size_t)((total - 1) * ld + row) * e;
}

}  // namespace check
}  // namespace gdn
