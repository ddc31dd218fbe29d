// Host-side checks of strided tensors, shared by the attention and the rotation.  Not part of the
// ABI.
#pragma once

#include <stdint.h>

#include <algorithm>

namespace da {

typedef __int128 wide_t;

// Bytes from a strided tensor's first number to its last; dimensions n (batch entries, tokens, heads)
// and D consecutive numbers of e bytes.
inline wide_t extent_bytes(const int64_t (&stride)[3], int64_t batch, int64_t tokens, int64_t heads,
                           int64_t D, int e) {
    if (batch == 0 || tokens == 0) return 0;
    return ((wide_t)(batch - 1) * stride[0] + (wide_t)(tokens - 1) * stride[1] +
            (wide_t)(heads - 1) * stride[2] + D) * e;
}

// [a, a + na) and [b, b + nb) share a byte
inline bool ranges_clash(const void* a, wide_t na, const void* b, wide_t nb) {
    const wide_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return a && b && na > 0 && nb > 0 && x < y + nb && y < x + na;
}

// Two places of a strided tensor are one: some stride, in the order of their size, does not pass what
// the smaller ones span.
inline bool overlaps_itself(const int64_t (&stride)[3], int64_t batch, int64_t tokens, int64_t heads,
                            int64_t D) {
    struct Dim {
        int64_t n, s;
    } d[3] = {{batch, stride[0]}, {tokens, stride[1]}, {heads, stride[2]}};
    std::sort(d, d + 3, [](const Dim& a, const Dim& b) { return a.s < b.s; });
    wide_t span = D;
    for (const Dim& x : d) {
        if (x.n <= 1) continue;
        if ((wide_t)x.s < span) return true;
        span += (wide_t)(x.n - 1) * x.s;
    }
    return false;
}

}  // namespace da
