// Rotation of heads by the angles of their positions, with the head norm, and the gradients.
// Contract and formulas: include/rotary.h.
//
// A head's numbers go by units of two vectors, a and b, that lie so that a pair never leaves
// its lane: in the half layout the vectors j and j + R / 2 V of the rotated part, in the
// interleaved one neighbours.  A power of two of lanes has a head, a lane keeps its units
// while it walks over a token's heads, and so forms their angles once for all of them: an angle
// costs some 40 instructions, eight heads' worth of the rest.
// Bound by memory: every number is read once and written once.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "act_device.h"
#include "rope_internal.h"

namespace da {
namespace {

// Cosine and sine of an angle given in binary64.  The nearest multiple of pi / 2 goes off in two
// multiply-adds, whose results are exact to 2^-53 of a turn for angles of billions; the rest, at most
// pi / 4, goes by the two series, whose first terms left out are below 2^-29 and 2^-33 of the
// result.  Off by about a unit in the last place of binary32.
__device__ __forceinline__ void turn_of(double angle, float& c, float& s) {
    const double q = rint(angle * 0.63661977236758134);   // 2 / pi
    const double rest = fma(-q, 6.123233995736766e-17, fma(-q, 1.5707963267948966, angle));
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

__device__ __forceinline__ double position_of(const RopeSide& t, int64_t b, int64_t n) {
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
    __device__ __forceinline__ void turns(const RopeArgs& r, int lane, double position) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                c[u][e] = s[u][e] = 0.0f;
                if (e < left[u]) {
                    turn_of(position * r.freqs[(lane + u * r.lanes) * V + e], c[u][e], s[u][e]);
                    c[u][e] *= r.magnitude;
                    s[u][e] *= r.magnitude * r.sign;
                }
            }
    }
    // x = [a's V, b's V] turned; SIGN -1 the other way.  Numbers past R stay what they are, whatever
    // their neighbours hold.
    template <int SIGN>
    __device__ __forceinline__ void rotate(bool interleaved, int u, float (&x)[2 * V]) const {
        if (V > 1 && interleaved) {
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float p = x[2 * e], q = x[2 * e + 1], t = SIGN * s[u][e];
                x[2 * e] = e < left[u] ? p * c[u][e] - q * t : p;
                x[2 * e + 1] = e < left[u] ? q * c[u][e] + p * t : q;
            }
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float p = x[e], q = x[e + V], t = SIGN * s[u][e];
                x[e] = e < left[u] ? p * c[u][e] - q * t : p;
                x[e + V] = e < left[u] ? q * c[u][e] + p * t : q;
            }
        }
    }
};

// The sum over the lanes of a head.
__device__ __forceinline__ float head_sum(float v, int lanes) {
    for (int m = 1; m < lanes; m *= 2) v += __shfl_xor(v, m);
    return v;
}

// What a thread has to do: `lanes` lanes have an item, a token and a slice of its heads.
struct Item {
    int64_t b, n;
    int head;
    __device__ __forceinline__ Item(const RopeSide& t, int64_t item) {
        const int64_t token = item / t.slices;
        head = (int)(item % t.slices);
        b = token / t.N;
        n = token % t.N;
    }
};

template <typename T, int V, int U, bool NORM>
__global__ __launch_bounds__(kRopeThreads) void rope_kernel(RopeArgs r) {
    const int which = blockIdx.x >= (uint32_t)r.side[0].blocks;
    const RopeSide& t = r.side[which];
    const int64_t thread =
        (int64_t)(blockIdx.x - (which ? r.side[0].blocks : 0)) * kRopeThreads + threadIdx.x;
    const int lane = (int)(thread % r.lanes);
    const int64_t item = thread / r.lanes;
    if (item >= t.items) return;   // whole heads
    const Item it(t, item);
    Units<V, U> units(r, lane);
    const bool interleaved = r.layout == ROPE_LAYOUT_INTERLEAVED;
    const T* x = static_cast<const T*>(t.x) + it.b * t.x_batch + it.n * t.x_token;
    T* y = static_cast<T*>(t.y) + it.b * t.y_batch + it.n * t.y_token;
    Piece<T, V> in[U][2], next[U][2];
    const auto fetch = [&](int head, Piece<T, V> (&to)[U][2]) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            to[u][0].zero();
            to[u][1].zero();
            if (units.a[u] >= 0) to[u][0].load(x + head * t.x_head + units.a[u]);
            if (units.b[u] >= 0) to[u][1].load(x + head * t.x_head + units.b[u]);
        }
    };
    fetch(it.head, in);
    float w[U][2 * V];
    if constexpr (NORM) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                w[u][e] = t.weight && units.a[u] >= 0 ? t.weight[units.a[u] + e] : 1.0f;
                w[u][e + V] = t.weight && units.b[u] >= 0 ? t.weight[units.b[u] + e] : 1.0f;
            }
    }
    units.turns(r, lane, position_of(t, it.b, it.n));
    for (int head = it.head; head < t.H; head += t.slices) {
        const bool more = head + t.slices < t.H;
        if (more) fetch(head + t.slices, next);
        float v[U][2 * V], sum = 0.0f;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                v[u][e] = (float)in[u][0].v[e];
                v[u][e + V] = (float)in[u][1].v[e];
                if constexpr (NORM) sum = fmaf(v[u][e], v[u][e], fmaf(v[u][e + V], v[u][e + V], sum));
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
            units.template rotate<1>(interleaved, u, v[u]);
            T* to = y + head * t.y_head;
            if (units.a[u] >= 0) store_piece<T, V>(to + units.a[u], v[u]);
            if (units.b[u] >= 0) store_piece<T, V>(to + units.b[u], v[u] + V);
        }
        if (more) {
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < 2; ++i) in[u][i] = next[u][i];
        }
    }
}

// The gradients.  Workgroups walk over the items, so that a lane's sums for the weights' gradient
// stay in registers; they meet in the workgroup through LDS, in an order of their own, and the
// workgroups' sums in rope_weight_kernel.
template <typename T, int V, int U>
__global__ __launch_bounds__(kRopeThreads) void rope_backward_kernel(RopeArgs r) {
    __shared__ float meet[kRopeThreads * U * 2 * V];
    const int which = blockIdx.x >= (uint32_t)r.side[0].blocks;
    const RopeSide& t = r.side[which];
    const int block = blockIdx.x - (which ? r.side[0].blocks : 0);
    const int lane = threadIdx.x % r.lanes, per = kRopeThreads / r.lanes;
    Units<V, U> units(r, lane);
    const bool interleaved = r.layout == ROPE_LAYOUT_INTERLEAVED;
    float w[U][2 * V], gw[U][2 * V];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int e = 0; e < V; ++e) {
            w[u][e] = t.weight && units.a[u] >= 0 ? t.weight[units.a[u] + e] : 1.0f;
            w[u][e + V] = t.weight && units.b[u] >= 0 ? t.weight[units.b[u] + e] : 1.0f;
            gw[u][e] = gw[u][e + V] = 0.0f;
        }
    for (int64_t item = (int64_t)block * per + threadIdx.x / r.lanes; item < t.items;
         item += (int64_t)t.blocks * per) {
        const Item it(t, item);
        const T* x = static_cast<const T*>(t.x) + it.b * t.x_batch + it.n * t.x_token;
        const T* g = static_cast<const T*>(t.y) + it.b * t.y_batch + it.n * t.y_token;
        T* dx = static_cast<T*>(t.dx) + (it.b * t.N + it.n) * t.H * r.D;
        units.turns(r, lane, position_of(t, it.b, it.n));
        for (int head = it.head; head < t.H; head += t.slices) {
            Piece<T, V> px[U][2], pg[U][2];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                px[u][0].zero(), px[u][1].zero(), pg[u][0].zero(), pg[u][1].zero();
                if (units.a[u] >= 0) {
                    px[u][0].load(x + head * t.x_head + units.a[u]);
                    pg[u][0].load(g + head * t.y_head + units.a[u]);
                }
                if (units.b[u] >= 0) {
                    px[u][1].load(x + head * t.x_head + units.b[u]);
                    pg[u][1].load(g + head * t.y_head + units.b[u]);
                }
            }
            float v[U][2 * V], d[U][2 * V], squares = 0.0f, dot = 0.0f;
#pragma unroll
            for (int u = 0; u < U; ++u) {
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    v[u][e] = (float)px[u][0].v[e];
                    v[u][e + V] = (float)px[u][1].v[e];
                    d[u][e] = (float)pg[u][0].v[e];
                    d[u][e + V] = (float)pg[u][1].v[e];
                }
                units.template rotate<-1>(interleaved, u, d[u]);
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
        }
    }
    if (!t.grad_weight) return;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int e = 0; e < 2 * V; ++e)
            meet[(u * 2 * V + e) * kRopeThreads + threadIdx.x] = gw[u][e];
    __syncthreads();
    // thread k adds up number (u, e) of lane l over the workgroup's heads
    for (int k = threadIdx.x; k < U * 2 * V * r.lanes; k += kRopeThreads) {
        const int l = k % r.lanes, ue = k / r.lanes;
        const Units<V, U> of(r, l);
        int at = -1;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                if (ue == u * 2 * V + e && of.a[u] >= 0) at = of.a[u] + e;
                if (ue == u * 2 * V + e + V && of.b[u] >= 0) at = of.b[u] + e;
            }
        if (at < 0) continue;
        double sum = 0.0;
        for (int p = 0; p < per; ++p) sum += (double)meet[ue * kRopeThreads + p * r.lanes + l];
        t.part[(int64_t)block * r.D + at] = (float)sum;
    }
}

// The workgroups' sums joined in binary64: 16 numbers of a head to a workgroup, 16 threads to each.
__global__ __launch_bounds__(kRopeThreads) void rope_weight_kernel(RopeArgs r) {
    __shared__ double meet[kRopeThreads];
    const int tiles = (r.D + 15) / 16;
    const RopeSide& t = r.side[blockIdx.x / tiles];
    if (!t.grad_weight) return;
    const int at = blockIdx.x % tiles * 16 + threadIdx.x % 16;
    double sum = 0.0;
    if (at < r.D)
        for (int k = threadIdx.x / 16; k < t.blocks; k += 16) sum += (double)t.part[(int64_t)k * r.D + at];
    meet[threadIdx.x] = sum;
    __syncthreads();
    if (threadIdx.x >= 16 || at >= r.D) return;
    for (int k = 1; k < 16; ++k) sum += meet[k * 16 + threadIdx.x];
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
    rope_weight_kernel<<<(uint32_t)(a.sides * ((a.D + 15) / 16)), kRopeThreads, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace da
