// Rotation of heads by the angles of their positions, with the head norm, and the gradients.
// Contract and formulas: include/rotary.h.
//
// A head's numbers go by units of two vectors, a and b, that lie so that a pair never leaves
// its lane: in the half layout the vectors j and j + R / 2 V of the rotated part, in the
// interleaved one neighbours.  A power of two of lanes has a head.  A workgroup has some tokens and
// forms their turns first, once each, in LDS: one costs some 30 instructions, a third of them in
// binary64, as much as two numbers' way through the rest.  Then groups of lanes walk over the
// tokens' heads, several abreast; other waves' loads cover a head's wait (numbers held ahead cost
// more waves than they won).  Bound by memory: every number is read once and written once
// (2 x 4096 tokens of 40 heads of 128 with the norm, bfloat16: 34 us for 168 MB; 134 MB of the
// rotation alone, read and written, 52 us, as a copy of them takes).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "act_device.h"
#include "rope_internal.h"

namespace da {
namespace {

// Cosine and sine of an angle given in binary64.  The nearest multiple of pi / 2 goes off in two
// multiply-adds: the first is exact, the second's result to 2^-53 of itself.  Which multiple is the
// nearest is known to 2^-52.5 of the angle, so that the rest is at most pi / 4 and as much.  It goes
// by the two series, whose first terms left out are 2^-28.5 and 2^-32.5 of the result at pi / 4 and
// still 2^-27.7 and 2^-31.5 for angles of 2^48: with the roundings to binary32 on the way it is off
// by at most 3.2 times 2^-24 of the result.  Towards 2^52, where neighbouring angles are half a radian
// apart, the rest reaches 1.5 and the series are off by up to 2^-18.
__device__ __forceinline__ void turn_of(double angle, float& c, float& s) {
    const double q = rint(angle * 0.63661977236758134);   // 2 / pi
    double rest = fma(-q, 6.123233995736766e-17, fma(-q, 1.5707963267948966, angle));
    if (!(fabs(angle) < 0x1p52)) rest = __builtin_nan("");   // no place within a turn
    const int quadrant = (int)(q - 4.0 * rint(q * 0.25));
    const float y = (float)rest, z = y * y;
    float sp = fmaf(z, 2.7557319e-6f, -1.9841270e-4f);
    sp = fmaf(z, sp, 8.3333333e-3f);
    sp = fmaf(z, sp, -1.6666667e-1f);
    const float sn = fmaf(y * z, sp, y);
    float cp = fmaf(z, -2.7557319e-7f, 2.4801587e-5f);
    cp = fmaf(z, cp, -1.3888889e-3f);
    cp = fmaf(z, cp, 4.1666667e-2f);
    cp = fmaf(z, cp, -0.5f);
    const float cs = fmaf(z, cp, 1.0f);
    const float a = quadrant & 1 ? sn : cs, b = quadrant & 1 ? cs : sn;
    c = (quadrant + 1) & 2 ? -a : a;
    s = quadrant & 2 ? -b : b;
}

// Of all tokens' `token`-th.
__device__ __forceinline__ double position_of(const RopeSide& t, uint32_t token) {
    const uint32_t b = token / (uint32_t)t.N, n = token - b * (uint32_t)t.N;
    const int64_t at = b * t.pos_batch + n;
    switch (t.pos_type) {
        case ROPE_POS_I32: return (double)static_cast<const int32_t*>(t.positions)[at];
        case ROPE_POS_I64: return (double)static_cast<const int64_t*>(t.positions)[at];
        case ROPE_POS_F32: return (double)static_cast<const float*>(t.positions)[at];
        default: return (double)n;
    }
}

// A vector of V numbers as it is in memory.
template <typename T, int V>
struct Piece {
    T v[V];
    __device__ __forceinline__ void load(const T* p) { __builtin_memcpy(v, __builtin_assume_aligned(p, sizeof(v)), sizeof(v)); }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] = (T)0.0f;
    }
};
template <typename T, int V>
__device__ __forceinline__ void store_piece(T* p, const float* v) {
    T t[V];
#pragma unroll
    for (int e = 0; e < V; ++e) t[e] = (T)v[e];
    __builtin_memcpy(__builtin_assume_aligned(p, sizeof(t)), t, sizeof(t));
}

// Where a lane's units lie, and their turns.
template <int V, int U>
struct Units {
    int a[U], b[U];                  // first numbers of the two vectors, or -1
    int left[U];                     // turned pairs from the unit's first on
    float c[U][V], s[U][V];          // of pairs (a[e], b[e]); interleaved: of a's pairs, then b's
    __device__ __forceinline__ Units(const RopeArgs& r, int lane) {
        const int half = r.layout == ROPE_LAYOUT_HALF ? r.R / (2 * V) : 0;   // rotated units
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int n = lane + u * r.lanes;
            if (n < half) {
                a[u] = n * V;
                b[u] = a[u] + r.R / 2;
            } else {
                a[u] = half * 2 * V + (n - half) * 2 * V;
                b[u] = a[u] + V;
            }
            left[u] = n < r.units ? r.R / 2 - n * V : 0;   // interleaved pairs run through both vectors
            if (n >= r.units || a[u] >= r.D) a[u] = -1;
            if (n >= r.units || b[u] >= r.D) b[u] = -1;
        }
    }
    // from the token's turns
    __device__ __forceinline__ void load(const RopeArgs& r, int lane, const float2* turns) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float2 t = e < left[u] ? turns[(lane + u * r.lanes) * V + e] : make_float2(1.0f, 0.0f);
                c[u][e] = t.x;
                s[u][e] = t.y;
            }
    }
    // x = [a's V, b's V] turned; SIGN -1 the other way.  Numbers past R stay what they are, whatever
    // their neighbours hold.
    template <int SIGN>
    __device__ __forceinline__ void rotate(const RopeArgs& r, int u, float (&x)[2 * V]) const {
        if (r.R == r.D)
            rotate_some<SIGN, true>(r.layout == ROPE_LAYOUT_INTERLEAVED, u, x);
        else
            rotate_some<SIGN, false>(r.layout == ROPE_LAYOUT_INTERLEAVED, u, x);
    }
    template <int SIGN, bool ALL>
    __device__ __forceinline__ void rotate_some(bool interleaved, int u, float (&x)[2 * V]) const {
        if (V > 1 && interleaved) {
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float p = x[2 * e], q = x[2 * e + 1], t = SIGN * s[u][e];
                x[2 * e] = ALL || e < left[u] ? p * c[u][e] - q * t : p;
                x[2 * e + 1] = ALL || e < left[u] ? q * c[u][e] + p * t : q;
            }
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float p = x[e], q = x[e + V], t = SIGN * s[u][e];
                x[e] = ALL || e < left[u] ? p * c[u][e] - q * t : p;
                x[e + V] = ALL || e < left[u] ? q * c[u][e] + p * t : q;
            }
        }
    }
};

// The sum over the lanes of a head, a power of two: pairs, fours, eights (which then read their
// mirror image) and sixteens by data-parallel primitives, then halves of the wave exchanged.  Every
// lane has the same sum, bit for bit.
template <int CTRL>
__device__ __forceinline__ float moved(float v) {
    return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float head_sum(float v, int lanes) {
    if (lanes > 1) v += moved<0xb1>(v);    // quad_perm 1 0 3 2
    if (lanes > 2) v += moved<0x4e>(v);    // quad_perm 2 3 0 1
    if (lanes > 4) v += moved<0x141>(v);   // row_half_mirror
    if (lanes > 8) v += moved<0x140>(v);   // row_mirror
    if (lanes > 16) {
        const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
    if (lanes > 32) {
        const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
    return v;
}

// The turns of a workgroup's tokens from `first` on, R / 2 to each.
__device__ __forceinline__ void form_turns(const RopeArgs& r, const RopeSide& t, uint32_t first, int count,
                                           float2* turns) {
    const uint32_t pairs = r.R / 2, all = count * pairs;
    for (uint32_t i = threadIdx.x; i < all; i += kRopeThreads) {
        const uint32_t token = first + i / pairs;
        if (token >= (uint32_t)t.tokens) break;
        float c, s;
        turn_of(position_of(t, token) * r.freqs[i % pairs], c, s);
        turns[i] = make_float2(c * r.magnitude, s * r.magnitude * r.sign);
    }
}

// A workgroup's share: its groups of lanes have `abreast` heads of `count` tokens.
struct Share {
    int lane, head, token, count;
    __device__ __forceinline__ Share(const RopeArgs& r, const RopeSide& t) {
        const int group = threadIdx.x / r.lanes;
        lane = threadIdx.x % r.lanes;
        head = group % t.abreast;
        token = group / t.abreast;
        count = kRopeThreads / r.lanes / t.abreast;
    }
};

template <typename T, int V, int U>
struct Vectors {
    Piece<T, V> v[U][2];
    __device__ __forceinline__ void load(const Units<V, U>& units, const T* p) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            v[u][0].zero();
            v[u][1].zero();
            if (units.a[u] >= 0) v[u][0].load(p + units.a[u]);
            if (units.b[u] >= 0) v[u][1].load(p + units.b[u]);
        }
    }
    __device__ __forceinline__ void unpack(int u, float (&x)[2 * V]) const {
#pragma unroll
        for (int e = 0; e < V; ++e) {
            x[e] = (float)v[u][0].v[e];
            x[e + V] = (float)v[u][1].v[e];
        }
    }
};
template <int V, int U>
__device__ __forceinline__ void load_weights(const Units<V, U>& units, const float* weight,
                                             float (&w)[U][2 * V]) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int e = 0; e < 2 * V; ++e) w[u][e] = 1.0f;
        if (weight && units.a[u] >= 0) __builtin_memcpy(w[u], weight + units.a[u], 4 * V);
        if (weight && units.b[u] >= 0) __builtin_memcpy(w[u] + V, weight + units.b[u], 4 * V);
    }
}

template <typename T, int V, int U, bool NORM>
__global__ __launch_bounds__(kRopeThreads) void rope_kernel(RopeArgs r) {
    __shared__ float2 turns[kRopeThreads * V * U];   // lanes * V * U >= R / 2 to a token
    const int which = blockIdx.x >= (uint32_t)r.side[0].blocks;
    const RopeSide& t = r.side[which];
    const Share at(r, t);
    const uint32_t first = (blockIdx.x - (which ? r.side[0].blocks : 0)) * at.count;
    const uint32_t token = first + at.token;
    const bool there = token < (uint32_t)t.tokens && at.head < t.H;   // for whole heads alike
    Units<V, U> units(r, at.lane);
    const uint32_t b = there ? token / (uint32_t)t.N : 0, n = there ? token - b * (uint32_t)t.N : 0;
    const T* x = static_cast<const T*>(t.x) + b * t.x_batch + n * t.x_token;
    T* y = static_cast<T*>(t.y) + b * t.y_batch + n * t.y_token;
    Vectors<T, V, U> in;
    if (there) in.load(units, x + at.head * t.x_head);
    float w[U][2 * V];
    if constexpr (NORM) load_weights(units, t.weight, w);
    form_turns(r, t, first, at.count, turns);
    __syncthreads();
    if (!there) return;
    units.load(r, at.lane, turns + at.token * (r.R / 2));
    for (int head = at.head; head < t.H; head += t.abreast) {
        const bool more = head + t.abreast < t.H;
        float v[U][2 * V], sum = 0.0f;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            in.unpack(u, v[u]);
            if constexpr (NORM) {
#pragma unroll
                for (int e = 0; e < 2 * V; ++e) sum = fmaf(v[u][e], v[u][e], sum);
            }
        }
        if constexpr (NORM) {
            const float f = rsqrtf(head_sum(sum, r.lanes) / (float)r.D + r.eps);
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int e = 0; e < 2 * V; ++e) v[u][e] *= f * w[u][e];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            units.template rotate<1>(r, u, v[u]);
            T* to = y + head * t.y_head;
            if (units.a[u] >= 0) store_piece<T, V>(to + units.a[u], v[u]);
            if (units.b[u] >= 0) store_piece<T, V>(to + units.b[u], v[u] + V);
        }
        if (more) in.load(units, x + (head + t.abreast) * t.x_head);
    }
}

// The gradients.  Workgroups walk over the tokens, so that a lane's sums for the weights' gradient
// stay in registers; they meet in the workgroup through LDS, in an order of their own, and the
// workgroups' sums in rope_weight_kernel.  Bound by memory (2 x 4096 tokens of 20 heads of 128,
// bfloat16, 126 MB: 33 us; 512 workgroups, since more cost their sums' way).
template <typename T, int V, int U>
__global__ __launch_bounds__(kRopeThreads) void rope_backward_kernel(RopeArgs r) {
    __shared__ float meet[kRopeThreads * U * 2 * V];   // turns, then the sums
    float2* turns = reinterpret_cast<float2*>(meet);
    const int which = blockIdx.x >= (uint32_t)r.side[0].blocks;
    const RopeSide& t = r.side[which];
    const int block = blockIdx.x - (which ? r.side[0].blocks : 0);
    const Share at(r, t);
    Units<V, U> units(r, at.lane);
    float w[U][2 * V], gw[U][2 * V];
    load_weights(units, t.weight, w);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int e = 0; e < 2 * V; ++e) gw[u][e] = 0.0f;
    for (uint32_t first = block * at.count; first < (uint32_t)t.tokens; first += t.blocks * at.count) {
        const uint32_t token = first + at.token;
        const bool there = token < (uint32_t)t.tokens && at.head < t.H;
        const uint32_t b = there ? token / (uint32_t)t.N : 0, n = there ? token - b * (uint32_t)t.N : 0;
        const T* x = static_cast<const T*>(t.x) + b * t.x_batch + n * t.x_token;
        const T* g = static_cast<const T*>(t.y) + b * t.y_batch + n * t.y_token;
        T* dx = static_cast<T*>(t.dx) + (int64_t)(there ? token : 0) * t.H * r.D;
        Vectors<T, V, U> px, pg;
        if (there) {
            px.load(units, x + at.head * t.x_head);
            pg.load(units, g + at.head * t.y_head);
        }
        __syncthreads();
        form_turns(r, t, first, at.count, turns);
        __syncthreads();
        if (!there) continue;
        units.load(r, at.lane, turns + at.token * (r.R / 2));
        for (int head = at.head; head < t.H; head += t.abreast) {
            const bool more = head + t.abreast < t.H;
            float v[U][2 * V], d[U][2 * V], squares = 0.0f, dot = 0.0f;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                px.unpack(u, v[u]);
                pg.unpack(u, d[u]);
                units.template rotate<-1>(r, u, d[u]);
#pragma unroll
                for (int e = 0; e < 2 * V; ++e) {
                    squares = fmaf(v[u][e], v[u][e], squares);
                    dot = fmaf(d[u][e] * w[u][e], v[u][e], dot);
                }
            }
            squares = head_sum(squares, r.lanes);
            dot = head_sum(dot, r.lanes);
            const float f = rsqrtf(squares / (float)r.D + r.eps);
            const float mean = dot * f / (float)r.D;   // of dn weight xhat
#pragma unroll
            for (int u = 0; u < U; ++u) {
#pragma unroll
                for (int e = 0; e < 2 * V; ++e) {
                    const float hat = v[u][e] * f;
                    gw[u][e] = fmaf(d[u][e], hat, gw[u][e]);
                    d[u][e] = f * (d[u][e] * w[u][e] - hat * mean);
                }
                if (t.dx) {
                    T* to = dx + (int64_t)head * r.D;
                    if (units.a[u] >= 0) store_piece<T, V>(to + units.a[u], d[u]);
                    if (units.b[u] >= 0) store_piece<T, V>(to + units.b[u], d[u] + V);
                }
            }
            if (more) {
                px.load(units, x + (head + t.abreast) * t.x_head);
                pg.load(units, g + (head + t.abreast) * t.y_head);
            }
        }
    }
    if (!t.grad_weight) return;
    __syncthreads();
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int e = 0; e < 2 * V; ++e)
            meet[(u * 2 * V + e) * kRopeThreads + threadIdx.x] = gw[u][e];
    __syncthreads();
    // thread k adds up number (u, e) of lane l over the workgroup's heads
    const int per = kRopeThreads / r.lanes;
    for (int k = threadIdx.x; k < U * 2 * V * r.lanes; k += kRopeThreads) {
        const int l = k % r.lanes, ue = k / r.lanes;
        const Units<V, U> of(r, l);
        int place = -1;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                if (ue == u * 2 * V + e && of.a[u] >= 0) place = of.a[u] + e;
                if (ue == u * 2 * V + e + V && of.b[u] >= 0) place = of.b[u] + e;
            }
        if (place < 0) continue;
        double sum = 0.0;
        for (int p = 0; p < per; ++p) sum += (double)meet[ue * kRopeThreads + p * r.lanes + l];
        t.part[(int64_t)block * r.D + place] = (float)sum;
    }
}

// The workgroups' sums joined in binary64: 8 numbers of a head to a workgroup, 32 threads to each.
constexpr int kJoinNumbers = 8;
__global__ __launch_bounds__(kRopeThreads) void rope_weight_kernel(RopeArgs r) {
    constexpr int kRows = kRopeThreads / kJoinNumbers;
    __shared__ double meet[kRopeThreads];
    const int tiles = (r.D + kJoinNumbers - 1) / kJoinNumbers;
    const RopeSide& t = r.side[blockIdx.x / tiles];
    if (!t.grad_weight) return;
    const int at = blockIdx.x % tiles * kJoinNumbers + threadIdx.x % kJoinNumbers;
    double sum = 0.0;
    if (at < r.D) {
#pragma unroll 16
        for (int k = threadIdx.x / kJoinNumbers; k < t.blocks; k += kRows)
            sum += (double)t.part[(int64_t)k * r.D + at];
    }
    meet[threadIdx.x] = sum;
    __syncthreads();
    if (threadIdx.x >= kJoinNumbers || at >= r.D) return;
#pragma unroll
    for (int k = 1; k < kRows; ++k) sum += meet[k * kJoinNumbers + threadIdx.x];
    t.grad_weight[at] = (float)sum;
}

template <typename T, int V, int U>
void launch(const RopeArgs& a, int kind, hipStream_t stream) {
    const uint32_t blocks = (uint32_t)a.side[0].blocks + (a.sides > 1 ? (uint32_t)a.side[1].blocks : 0u);
    if (blocks == 0) return;   // weights' gradients of no tokens
    if (kind == 0)
        rope_kernel<T, V, U, false><<<blocks, kRopeThreads, 0, stream>>>(a);
    else if (kind == 1)
        rope_kernel<T, V, U, true><<<blocks, kRopeThreads, 0, stream>>>(a);
    else
        rope_backward_kernel<T, V, U><<<blocks, kRopeThreads, 0, stream>>>(a);
}

template <typename T, int V>
void launch_units(const RopeArgs& a, int kind, int per_lane, hipStream_t stream) {
    // 512 numbers are 64 lanes' worth of units of 16 bytes or two numbers, of shorter ones more
    if (per_lane <= 1)
        launch<T, V, 1>(a, kind, stream);
    else if constexpr (V <= 2) {
        if (per_lane <= 2)
            launch<T, V, 2>(a, kind, stream);
        else if constexpr (V == 1)
            launch<T, V, 4>(a, kind, stream);
    }
}

template <typename T>
void launch_type(const RopeArgs& a, int kind, int vec, int per_lane, hipStream_t stream) {
    if (vec == 1)
        launch_units<T, 1>(a, kind, per_lane, stream);
    else if (vec == 2)
        launch_units<T, 2>(a, kind, per_lane, stream);
    else if (vec == 4)
        launch_units<T, 4>(a, kind, per_lane, stream);
    else if constexpr (sizeof(T) == 2)
        launch_units<T, 8>(a, kind, per_lane, stream);
}

hipError_t launch_kind(const RopeArgs& a, int kind, int vec, int per_lane, hipStream_t stream) {
    if (a.dtype == DA_BF16)
        launch_type<__bf16>(a, kind, vec, per_lane, stream);
    else if (a.dtype == DA_F16)
        launch_type<_Float16>(a, kind, vec, per_lane, stream);
    else
        launch_type<float>(a, kind, vec, per_lane, stream);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_rope(const RopeArgs& a, bool norm, int vec, int per_lane, hipStream_t stream) {
    return launch_kind(a, norm ? 1 : 0, vec, per_lane, stream);
}

hipError_t launch_rope_norm_backward(const RopeArgs& a, int vec, int per_lane, hipStream_t stream) {
    const hipError_t e = launch_kind(a, 2, vec, per_lane, stream);
    bool weights = false;
    for (int i = 0; i < a.sides; ++i) weights = weights || a.side[i].grad_weight;
    if (e != hipSuccess || !weights) return e;
    rope_weight_kernel<<<(uint32_t)(a.sides * ((a.D + kJoinNumbers - 1) / kJoinNumbers)), kRopeThreads, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace da
