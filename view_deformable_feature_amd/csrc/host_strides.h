// Host-side checks of strided tensors, shared by the attention and the rotation.  Not part of the
// ABI.
#pragma once

#include <stdint.h>

#include <algorithm>
#include <utility>

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

// A tensor of [batch, tokens, heads, D] numbers of e bytes as its checks see it.
struct Heads {
    const void* at;
    int64_t n[3];          // batch entries, tokens, heads
    const int64_t* stride;
    int64_t D;
    int e;

    wide_t bytes() const {
        const int64_t s[3] = {stride[0], stride[1], stride[2]};
        return extent_bytes(s, n[0], n[1], n[2], D, e);
    }
};

// a and b lie between each other, as parts of one packed tensor do: some dimension of the same stride
// in both, the period, holds what is within it side by side, a's and b's apart, and dimensions beyond
// it have equal strides, too, that each pass what the smaller ones span.
inline bool lie_between(const Heads& a, const Heads& b) {
    // of dimensions that have more than one place in either
    const auto counts = [&](int i) { return a.n[i] > 1 || b.n[i] > 1; };
    const auto stride = [&](int i) { return a.n[i] > 1 ? a.stride[i] : b.stride[i]; };
    const auto common = [&](int i) { return a.n[i] <= 1 || b.n[i] <= 1 || a.stride[i] == b.stride[i]; };
    for (int period = 0; period < 3; ++period) {
        if (!counts(period) || !common(period) || stride(period) == 0) continue;
        const wide_t P = stride(period);
        wide_t span_a = a.D, span_b = b.D;
        int beyond[2], more = 0;
        bool fits = true;
        for (int i = 0; i < 3; ++i) {
            if (i == period || !counts(i)) continue;
            const bool in_a = a.n[i] <= 1 || a.stride[i] < P, in_b = b.n[i] <= 1 || b.stride[i] < P;
            if (in_a && in_b) {
                span_a += a.n[i] > 1 ? (wide_t)(a.n[i] - 1) * a.stride[i] : 0;
                span_b += b.n[i] > 1 ? (wide_t)(b.n[i] - 1) * b.stride[i] : 0;
            } else if (common(i)) {
                beyond[more++] = i;
            } else {
                fits = false;
            }
        }
        if (more == 2 && stride(beyond[0]) > stride(beyond[1])) std::swap(beyond[0], beyond[1]);
        wide_t reach = P * std::max(a.n[period], b.n[period]);
        for (int k = 0; k < more; ++k) {
            const wide_t s = stride(beyond[k]);
            fits = fits && s >= reach;
            reach = s * std::max(a.n[beyond[k]], b.n[beyond[k]]);
        }
        const wide_t d = (wide_t)reinterpret_cast<uintptr_t>(b.at) - (wide_t)reinterpret_cast<uintptr_t>(a.at);
        if (fits && (d >= 0 ? d >= span_a * a.e && d + span_b * a.e <= P * a.e
                            : -d >= span_b * a.e && -d + span_a * a.e <= P * a.e))
            return true;
    }
    return false;
}

// Some place of a may be one of b (of the same type).
inline bool may_meet(const Heads& a, const Heads& b) {
    return ranges_clash(a.at, a.bytes(), b.at, b.bytes()) && !lie_between(a, b);
}

}  // namespace da
