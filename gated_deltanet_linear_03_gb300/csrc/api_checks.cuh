// Argument checks that the C entry points share (host only).
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace gdn {
namespace api {

inline bool aligned(const void *p, uintptr_t n = 16) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

struct Range {
    const void *p;
    size_t n;
};

inline bool overlaps(const Range &a, const Range &b) {
    if (!a.p || !b.p || a.n == 0 || b.n == 0) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return x < y + b.n && y < x + a.n;
}

// No output may overlap an input or another output.
template <size_t N, size_t M>
bool disjoint(const Range (&outs)[N], const Range (&ins)[M]) {
    for (size_t i = 0; i < N; ++i) {
        for (const Range &in : ins)
            if (overlaps(outs[i], in)) return false;
        for (size_t j = i + 1; j < N; ++j)
            if (overlaps(outs[i], outs[j])) return false;
    }
    return true;
}

// bytes of `tokens` rows of `row` bf16 elements, `stride` elements apart
inline size_t rows_bytes(int tokens, long long stride, long long row) {
    return tokens > 0 ? ((size_t)(tokens - 1) * stride + row) * 2 : 0;
}

}  // namespace api
}  // namespace gdn
