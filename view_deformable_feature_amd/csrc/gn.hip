// Group norm with an activation on channels-last maps, forward and backward.
// Contract and formulas: include/group_norm.h.
//
// Lanes lie along the channels of a row, so every access is a run of whole 16-byte
// vectors, and a thread stays with one vector of channels: its weights, its groups'
// statistics and the backward's per-channel sums sit in registers.
//
// The operator has a handful of operations to a value, so memory bounds it: its floor is a copy
// of as many bytes, which reaches 4.9 to 5.3 TB/s from 100 MB on and 6.4 at 77 MB.  Times here
// are of one MI355X, inputs and outputs in rotation so that no call finds its own in cache.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "act_device.h"
#include "gn_internal.h"

namespace da {
namespace {

// Where a workgroup works: its slab of channels, and its threads' places in it.
struct Slab {
    int ch0, width;        // channels
    int unit0, nunits;     // statistics units
    int g0;                // first group
    int cols, R;           // vectors per row, rows at a time
    int r, v;              // this thread's row and vector; r >= R: none
};

template <int V>
__device__ __forceinline__ Slab slab_of(const GnArgs& a, int s, int threads) {
    Slab b;
    if (a.upg == 1) {
        b.ch0 = s * a.slab_ch;
        b.width = min(a.slab_ch, a.C - b.ch0);
        b.g0 = b.unit0 = b.ch0 / a.cpg;
        b.nunits = b.width / a.cpg;
    } else {
        const int g = s / a.upg, u = s - g * a.upg;
        b.ch0 = g * a.cpg + u * a.cpu;
        b.width = min(a.cpu, a.cpg - u * a.cpu);
        b.g0 = g;
        b.unit0 = s;
        b.nunits = 1;
    }
    b.cols = b.width / V;
    b.R = threads / b.cols;
    b.r = threadIdx.x / b.cols;
    b.v = threadIdx.x - b.r * b.cols;
    return b;
}

// out[u] = factor * the sum of red[r * cols + j] over r < R and the `per` columns of unit u,
// added up in M, by a run of 8 to 64 lanes per unit: as many as have something to add and leave
// all units to one pass, since a pass waits for its exchanges one after the other.  Every thread
// of the workgroup calls it; red is complete on entry, out on return.
template <typename M>
__device__ __forceinline__ void unit_sums(const float* red, int R, int cols, int per, int nunits,
                                          double factor, M* out) {
    int run = kWave;
    while (run > 8 && (nunits * run > (int)blockDim.x || run / 2 >= R * per)) run /= 2;
    const int lane = threadIdx.x & (run - 1), skip_r = run / per, skip_j = run - skip_r * per;
    const int r0 = lane / per, j0 = lane - r0 * per;
    for (int u = threadIdx.x / run; u - (int)threadIdx.x / run < nunits; u += blockDim.x / run) {
        M t = 0;
        if (u < nunits)
            for (int r = r0, j = j0; r < R; r += skip_r) {
                t += red[r * cols + u * per + j];
                j += skip_j;
                if (j >= per) {
                    j -= per;
                    ++r;
                }
            }
        t = group_sum(t, run);
        if (lane == run - 1 && u < nunits) out[u] = (M)(t * factor);
    }
    __syncthreads();
}

// Units of a thread's channels: channel e of vector v lies in unit u[e] of the slab.
template <int V>
__device__ __forceinline__ void units_of(const Slab& b, int per_ch, int (&u)[V]) {
    int unit = b.v * V / per_ch, left = per_ch - (b.v * V - unit * per_ch);
#pragma unroll
    for (int e = 0; e < V; ++e) {
        u[e] = unit;
        if (--left == 0) {
            ++unit;
            left = per_ch;
        }
    }
}

// The group's first value in image n: all of the group's means are formed and kept as
// differences from it, so that a large common offset cancels before anything is rounded.
__device__ __forceinline__ float origin_of(const GnArgs& a, int n, int g) {
    return load_elem(a.x, (int64_t)n * a.S * a.C + (int64_t)g * a.cpg, a.x_dtype);
}

// 1 / sqrt(var + eps), rounded once; squares past binary32 leave no number.
__device__ __forceinline__ float rstd_of(double var, float eps) {
    return var < 0x1p127 ? (float)(1.0 / sqrt(var + (double)eps)) : __uint_as_float(0x7fc00000u);
}

// A workgroup's statistics from its threads' (share: 1 over the number of a unit's values):
// each of cnt rows of V channels, with the sums of their differences from `first` and of those
// differences' squares, taken about that value so that a large common offset cancels before
// anything is rounded.  Leaves in um the units' means less the group's origin, in uq their sums
// of squared deviations from that mean, both in binary64: a difference from an origin far from
// the mean, rounded to binary32, would be the mean's error.  red holds one value per thread
// where a vector lies in one unit, else V.
template <int V>
__device__ __forceinline__ void join_threads(const GnArgs& a, const Slab& b, int n, double share,
                                             int cnt, const float (&first)[V],
                                             const float (&sum)[V], const float (&sq)[V],
                                             float* red, double* um, double* uq) {
    const int per_ch = a.upg == 1 ? a.cpg : b.width;
    const bool whole = per_ch % V == 0;
    const int cols = whole ? b.cols : b.width, per = whole ? per_ch / V : per_ch;
    const float rc = cnt ? 1.0f / cnt : 0.0f;
    float m[V], dev[V];   // this thread's channel means, less the origin; squares about them
    int u[V];
    units_of(b, per_ch, u);
    float origin = origin_of(a, n, b.g0 + u[0]);
#pragma unroll
    for (int e = 0; e < V; ++e) {
        if (!whole) origin = origin_of(a, n, b.g0 + u[e]);
        m[e] = (first[e] - origin) + sum[e] * rc;
        // sum of squares about m is sq - sum^2 / cnt, below zero by rounding alone; a NaN stays
        dev[e] = sq[e] - sum[e] * sum[e] * rc;
    }
    if (b.r < b.R) {
        if (whole) {
            float t = 0.0f;
#pragma unroll
            for (int e = 0; e < V; ++e) t += m[e];
            red[b.r * cols + b.v] = t * cnt;
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e) red[b.r * cols + b.v * V + e] = m[e] * cnt;
        }
    }
    __syncthreads();
    unit_sums(red, b.R, cols, per, b.nunits, share, um);
    float mean = (float)um[u[0]];
#pragma unroll
    for (int e = 0; e < V; ++e) {
        if (!whole) mean = (float)um[u[e]];
        const float d = m[e] - mean;
        dev[e] = cnt ? (dev[e] < 0.0f ? 0.0f : dev[e]) + cnt * d * d : 0.0f;
    }
    if (b.r < b.R) {
        if (whole) {
            float t = 0.0f;
#pragma unroll
            for (int e = 0; e < V; ++e) t += dev[e];
            red[b.r * cols + b.v] = t;
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e) red[b.r * cols + b.v * V + e] = dev[e];
        }
    }
    __syncthreads();
    unit_sums(red, b.R, cols, per, b.nunits, 1.0, uq);
}

// One chunk: (mean less the group's origin, M2) of each unit, where M2 is the sum of
// squared deviations from that mean.  Each thread takes its squares about its first row,
// then moves them to the unit's mean.
//
// By chunks x is read twice: 6 x 11264 x 256 binary32 (69 MB) takes 23 us here and 26 us in
// gn_apply_kernel, 48 us a call (floor 28 us).  The second read comes in part from cache; this one
// runs at 3 TB/s, two batches of loads to a thread, the second asked for when the first is added up.
// Rows of 256 bytes to a slab and 16 rows to a thread; with a slab per group (32 bytes of a
// row) held in LDS and read once it took 62 us, since an image has too few workgroups.
template <typename T, int V>
__global__ __launch_bounds__(kGnThreads) void gn_stats_kernel(GnArgs a) {
    __shared__ float red[kGnThreads * V];
    __shared__ double um[kGnUnits], uq[kGnUnits];
    const int s = blockIdx.x % a.slabs;
    const int chunk = (blockIdx.x / a.slabs) % a.chunks;
    const int n = blockIdx.x / a.slabs / a.chunks;
    const Slab b = slab_of<V>(a, s, kGnThreads);
    const int64_t r0 = chunk * a.rows_per_chunk, r1 = min(r0 + a.rows_per_chunk, a.S);
    const T* p = static_cast<const T*>(a.x) + ((int64_t)n * a.S) * a.C + b.ch0 + b.v * V;

    float first[V], sum[V], sq[V];
    int cnt = 0;
#pragma unroll
    for (int e = 0; e < V; ++e) first[e] = sum[e] = sq[e] = 0.0f;
    if (b.r < b.R) {
        int64_t row = r0 + b.r;
        if (row < r1) Raw<T, V>::load(p + row * a.C).unpack(first);
        constexpr int U = 8;
        for (; row < r1; row += U * b.R) {
            Raw<T, V> q[U];
#pragma unroll
            for (int i = 0; i < U; ++i)
                if (row + i * b.R < r1) q[i] = Raw<T, V>::load(p + (row + i * b.R) * a.C);
#pragma unroll
            for (int i = 0; i < U; ++i)
                if (row + i * b.R < r1) {
                    float x[V];
                    q[i].unpack(x);
                    ++cnt;
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        const float d = x[e] - first[e];
                        sum[e] += d;
                        sq[e] = fmaf(d, d, sq[e]);
                    }
                }
        }
    }
    const double share = 1.0 / ((double)(r1 - r0) * (a.upg == 1 ? a.cpg : b.width));
    join_threads(a, b, n, share, cnt, first, sum, sq, red, um, uq);
    double2* part = a.stat_part + ((int64_t)n * a.chunks + chunk) * a.units + b.unit0;
    for (int u = threadIdx.x; u < b.nunits; u += kGnThreads) {
        part[u] = make_double2(um[u], uq[u]);
        // kept: x may be overwritten in place by the time the chunks are joined
        if (chunk == 0 && (a.upg == 1 || s % a.upg == 0))
            a.origins[(int64_t)n * a.G + b.g0 + u] = origin_of(a, n, b.g0 + u);
    }
}

// The chunks' statistics of groups g0 .. g0 + ngroups - 1 joined in binary64, a run of 8 to
// 64 lanes to a group: mean and rstd into LDS.  Every thread of the workgroup calls it.
__device__ __forceinline__ void join_stats(const GnArgs& a, int n, int g0, int ngroups, float* gm,
                                           float* gr) {
    const int run = ngroups <= 4 ? 64 : ngroups <= 8 ? 32 : ngroups <= 16 ? 16 : 8;
    const int lane = threadIdx.x & (run - 1), entries = a.chunks * a.upg;
    const double total = (double)a.S * a.cpg;
    constexpr int kHold = 4;
    for (int j0 = 0; j0 < ngroups; j0 += kGnThreads / run) {
        const int j = j0 + (int)threadIdx.x / run, g = g0 + min(j, ngroups - 1);
        const double2* part = a.stat_part + (int64_t)n * a.chunks * a.units + (int64_t)g * a.upg;
        // entry e: unit e % upg of chunk e / upg, and how many values it stands for
        const auto entry = [&](int e, double2& q, double& cnt) {
            const int c = a.upg == 1 ? e : e / a.upg, u = e - c * a.upg;
            const int64_t r0 = c * a.rows_per_chunk;
            q = part[(int64_t)c * a.units + u];
            cnt = (double)(min(r0 + a.rows_per_chunk, a.S) - r0) * min(a.cpu, a.cpg - u * a.cpu);
        };
        double2 q[kHold];
        double cnt[kHold], sum = 0.0, m2 = 0.0;
#pragma unroll
        for (int i = 0; i < kHold; ++i) {
            q[i] = make_double2(0.0, 0.0);
            cnt[i] = 0.0;
            if (lane + i * run < entries) entry(lane + i * run, q[i], cnt[i]);
        }
#pragma unroll
        for (int i = 0; i < kHold; ++i) sum += cnt[i] * q[i].x;
        for (int e = lane + kHold * run; e < entries; e += run) {
            entry(e, q[0], cnt[0]);
            sum += cnt[0] * q[0].x;
        }
        for (int m = run / 2; m; m >>= 1) sum += __shfl_xor(sum, m);
        const double mean = sum / total;
        if (entries > kHold * run) {   // the first entry was read over
            q[0] = make_double2(0.0, 0.0);
            cnt[0] = 0.0;
            entry(lane, q[0], cnt[0]);
        }
#pragma unroll
        for (int i = 0; i < kHold; ++i) m2 += q[i].y + cnt[i] * (q[i].x - mean) * (q[i].x - mean);
        for (int e = lane + kHold * run; e < entries; e += run) {
            entry(e, q[0], cnt[0]);
            m2 += q[0].y + cnt[0] * (q[0].x - mean) * (q[0].x - mean);
        }
        for (int m = run / 2; m; m >>= 1) m2 += __shfl_xor(m2, m);
        if (lane == 0 && j < ngroups) {
            gm[j] = (float)(mean + (double)a.origins[(int64_t)n * a.G + g]);
            gr[j] = rstd_of(m2 / total, a.eps);
        }
    }
    __syncthreads();
}

// mean and rstd alone: 4 groups to a workgroup.
constexpr int kGnJoin = kGnThreads / kWave;
__global__ __launch_bounds__(kGnThreads) void gn_join_kernel(GnArgs a) {
    __shared__ float gm[kGnJoin], gr[kGnJoin];
    const int blocks = (a.G + kGnJoin - 1) / kGnJoin;
    const int n = blockIdx.x / blocks, g0 = (blockIdx.x - n * blocks) * kGnJoin;
    const int ngroups = min(kGnJoin, a.G - g0);
    join_stats(a, n, g0, ngroups, gm, gr);
    if ((int)threadIdx.x < ngroups) {
        a.mean[(int64_t)n * a.G + g0 + threadIdx.x] = gm[threadIdx.x];
        a.rstd[(int64_t)n * a.G + g0 + threadIdx.x] = gr[threadIdx.x];
    }
}

template <typename T, int V>
__global__ __launch_bounds__(kGnThreads) void gn_apply_kernel(GnArgs a) {
    __shared__ float gm[kGnUnits], gr[kGnUnits];
    const int s = blockIdx.x % a.slabs;
    const int chunk = (blockIdx.x / a.slabs) % a.chunks;
    const int n = blockIdx.x / a.slabs / a.chunks;
    const Slab b = slab_of<V>(a, s, kGnThreads);
    // every workgroup joins the chunks of its groups itself: a launch less, and with others to
    // run meanwhile the wait for them is hidden (by one wave to a group, one after the other,
    // it took longer than the normalisation; by runs of lanes it is not seen)
    const int ngroups = a.upg == 1 ? b.nunits : 1;
    join_stats(a, n, b.g0, ngroups, gm, gr);
    if (chunk == 0 && (a.upg == 1 || s % a.upg == 0)) {
        for (int j = threadIdx.x; j < ngroups; j += kGnThreads) {
            if (a.mean) a.mean[(int64_t)n * a.G + b.g0 + j] = gm[j];
            if (a.rstd) a.rstd[(int64_t)n * a.G + b.g0 + j] = gr[j];
        }
    }
    if (b.r >= b.R) return;
    float mu[V], sc[V], bi[V];
    int u[V];
    units_of(b, a.upg == 1 ? a.cpg : b.width, u);
#pragma unroll
    for (int e = 0; e < V; ++e) {
        const int c = b.v * V + e, j = u[e];
        mu[e] = gm[j];
        sc[e] = gr[j] * (a.weight ? a.weight[b.ch0 + c] : 1.0f);
        bi[e] = a.bias ? a.bias[b.ch0 + c] : 0.0f;
    }
    const int64_t r0 = chunk * a.rows_per_chunk, r1 = min(r0 + a.rows_per_chunk, a.S);
    const int64_t base = ((int64_t)n * a.S) * a.C + b.ch0 + b.v * V;
    const T* p = static_cast<const T*>(a.x) + base;
    constexpr int U = 4;
    for (int64_t row = r0 + b.r; row < r1; row += U * b.R) {
        Raw<T, V> q[U];
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (row + i * b.R < r1) q[i] = Raw<T, V>::load(p + (row + i * b.R) * a.C);
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (row + i * b.R < r1) {
                float z[V];
                q[i].unpack(z);
#pragma unroll
                for (int e = 0; e < V; ++e) z[e] = fmaf(z[e] - mu[e], sc[e], bi[e]);
                activate(z, a.act);
                store_vec(a.out, base + (row + i * b.R) * a.C, z, a.out_dtype);
            }
    }
}

// The threads' sums A and B of each channel added up over their rows: ra[c], rb[c] for c <
// width.  Rows fold in halves: R -> ceil(R / 2) -> ... -> 1.
template <int V>
__device__ __forceinline__ void fold_rows(const Slab& b, const float (&A)[V], const float (&B)[V],
                                          float* ra, float* rb) {
    if (b.r < b.R) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
            ra[b.r * b.width + b.v * V + e] = A[e];
            rb[b.r * b.width + b.v * V + e] = B[e];
        }
    }
    __syncthreads();
    for (int R = b.R; R > 1;) {
        const int half = (R + 1) / 2, n2 = (R - half) * b.width;
        for (int e = threadIdx.x; e < n2; e += blockDim.x) {
            ra[e] += ra[e + half * b.width];
            rb[e] += rb[e + half * b.width];
        }
        R = half;
        __syncthreads();
    }
}

// Sums of dz and dz * xhat: per channel (for grad_weight and grad_bias) and, weighted,
// per unit (for grad_x), of one chunk.
template <typename T, int V>
__global__ __launch_bounds__(kGnThreads) void gn_bwd_stats_kernel(GnArgs a) {
    __shared__ float ra[kGnThreads * V], rb[kGnThreads * V];
    __shared__ float ua[kGnUnits], ub[kGnUnits];
    const int s = blockIdx.x % a.slabs;
    const int chunk = (blockIdx.x / a.slabs) % a.chunks;
    const int n = blockIdx.x / a.slabs / a.chunks;
    const Slab b = slab_of<V>(a, s, kGnThreads);
    const int64_t r0 = chunk * a.rows_per_chunk, r1 = min(r0 + a.rows_per_chunk, a.S);
    const int64_t base = ((int64_t)n * a.S) * a.C + b.ch0 + b.v * V;
    const T* p = static_cast<const T*>(a.x) + base;

    float A[V], B[V];
#pragma unroll
    for (int e = 0; e < V; ++e) A[e] = B[e] = 0.0f;
    if (b.r < b.R) {
        float mu[V], rs[V], w[V], bi[V];
        int u[V];
        units_of(b, a.upg == 1 ? a.cpg : b.width, u);
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const int c = b.v * V + e, j = u[e];
            mu[e] = a.mean[(int64_t)n * a.G + b.g0 + j];
            rs[e] = a.rstd[(int64_t)n * a.G + b.g0 + j];
            w[e] = a.weight ? a.weight[b.ch0 + c] : 1.0f;
            bi[e] = a.bias ? a.bias[b.ch0 + c] : 0.0f;
        }
        constexpr int U = 2;
        for (int64_t row = r0 + b.r; row < r1; row += U * b.R) {
            Raw<T, V> q[U];
            float d[U][V];
#pragma unroll
            for (int i = 0; i < U; ++i)
                if (row + i * b.R < r1) {
                    q[i] = Raw<T, V>::load(p + (row + i * b.R) * a.C);
                    load_vec(a.grad_out, base + (row + i * b.R) * a.C, d[i], a.out_dtype);
                }
#pragma unroll
            for (int i = 0; i < U; ++i)
                if (row + i * b.R < r1) {
                    float x[V], z[V];
                    q[i].unpack(x);
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        x[e] = (x[e] - mu[e]) * rs[e];
                        z[e] = fmaf(x[e], w[e], bi[e]);
                    }
                    activate_grad(d[i], z, a.act);
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        A[e] += d[i][e];
                        B[e] = fmaf(d[i][e], x[e], B[e]);
                    }
                }
        }
    }
    fold_rows(b, A, B, ra, rb);
    float2* cp = a.chan_part + ((int64_t)n * a.chunks + chunk) * a.C + b.ch0;
    for (int c = threadIdx.x; c < b.width; c += kGnThreads) {
        cp[c] = make_float2(ra[c], rb[c]);
        const float w = a.weight ? a.weight[b.ch0 + c] : 1.0f;
        ra[c] *= w;
        rb[c] *= w;
    }
    __syncthreads();
    const int per = a.upg == 1 ? a.cpg : b.width;
    unit_sums(ra, 1, b.width, per, b.nunits, 1.0, ua);
    unit_sums(rb, 1, b.width, per, b.nunits, 1.0, ub);
    float2* up = a.unit_part + ((int64_t)n * a.chunks + chunk) * a.units + b.unit0;
    for (int u = threadIdx.x; u < b.nunits; u += kGnThreads) up[u] = make_float2(ua[u], ub[u]);
}

// grad_weight and grad_bias of 16 channels from the chunks' sums: as many as there are images
// and chunks, so joined in binary64.
constexpr int kGnChanBlock = 16;
__device__ __forceinline__ void channel_sums(const GnArgs& a, int block) {
    __shared__ double2 red[kGnThreads];
    const int c = block * kGnChanBlock + threadIdx.x % kGnChanBlock;
    double2 t = make_double2(0.0, 0.0);
    const int64_t parts = (int64_t)a.N * a.chunks;
    if (c < a.C)
        for (int64_t e = threadIdx.x / kGnChanBlock; e < parts; e += kGnThreads / kGnChanBlock) {
            const float2 q = a.chan_part[e * a.C + c];
            t.x += q.x;
            t.y += q.y;
        }
    red[threadIdx.x] = t;
    __syncthreads();
    if (threadIdx.x < kGnChanBlock && c < a.C) {
        for (int e = threadIdx.x + kGnChanBlock; e < kGnThreads; e += kGnChanBlock) {
            t.x += red[e].x;
            t.y += red[e].y;
        }
        if (a.grad_bias) a.grad_bias[c] = (float)t.x;
        if (a.grad_weight) a.grad_weight[c] = (float)t.y;
    }
}

// The averages over (image n, groups g0 .. g0 + ngroups - 1) of weight * dz and weight * dz *
// xhat from the chunks' sums, as join_stats.
__device__ __forceinline__ void join_sums(const GnArgs& a, int n, int g0, int ngroups, float* m1,
                                          float* m2) {
    const int run = ngroups <= 4 ? 64 : ngroups <= 8 ? 32 : ngroups <= 16 ? 16 : 8;
    const int lane = threadIdx.x & (run - 1), entries = a.chunks * a.upg;
    const double inv = 1.0 / ((double)a.S * a.cpg);
    for (int j0 = 0; j0 < ngroups; j0 += kGnThreads / run) {
        const int j = j0 + (int)threadIdx.x / run, g = g0 + min(j, ngroups - 1);
        const float2* part = a.unit_part + (int64_t)n * a.chunks * a.units + (int64_t)g * a.upg;
        double t1 = 0.0, t2 = 0.0;
        for (int e = lane; e < entries; e += run) {
            const int c = a.upg == 1 ? e : e / a.upg;
            const float2 q = part[(int64_t)c * a.units + e - c * a.upg];
            t1 += q.x;
            t2 += q.y;
        }
        for (int m = run / 2; m; m >>= 1) {
            t1 += __shfl_xor(t1, m);
            t2 += __shfl_xor(t2, m);
        }
        if (lane == 0 && j < ngroups) {
            m1[j] = (float)(t1 * inv);
            m2[j] = (float)(t2 * inv);
        }
    }
    __syncthreads();
}

// grad_x of one chunk; the workgroups after the last chunk's form grad_weight and
// grad_bias.
template <typename T, int V>
__global__ __launch_bounds__(kGnThreads) void gn_bwd_apply_kernel(GnArgs a, int64_t chunk_blocks) {
    if (blockIdx.x >= chunk_blocks) {
        channel_sums(a, blockIdx.x - chunk_blocks);
        return;
    }
    __shared__ float m1[kGnUnits], m2[kGnUnits];
    const int s = blockIdx.x % a.slabs;
    const int chunk = (blockIdx.x / a.slabs) % a.chunks;
    const int n = blockIdx.x / a.slabs / a.chunks;
    const Slab b = slab_of<V>(a, s, kGnThreads);
    join_sums(a, n, b.g0, a.upg == 1 ? b.nunits : 1, m1, m2);
    if (b.r >= b.R) return;
    float mu[V], rs[V], w[V], bi[V], c1[V], c2[V];
    int u[V];
    units_of(b, a.upg == 1 ? a.cpg : b.width, u);
#pragma unroll
    for (int e = 0; e < V; ++e) {
        const int c = b.v * V + e, j = u[e];
        mu[e] = a.mean[(int64_t)n * a.G + b.g0 + j];
        rs[e] = a.rstd[(int64_t)n * a.G + b.g0 + j];
        w[e] = a.weight ? a.weight[b.ch0 + c] : 1.0f;
        bi[e] = a.bias ? a.bias[b.ch0 + c] : 0.0f;
        c1[e] = m1[j];
        c2[e] = m2[j];
    }
    const int64_t r0 = chunk * a.rows_per_chunk, r1 = min(r0 + a.rows_per_chunk, a.S);
    const int64_t base = ((int64_t)n * a.S) * a.C + b.ch0 + b.v * V;
    const T* p = static_cast<const T*>(a.x) + base;
    constexpr int U = 2;
    for (int64_t row = r0 + b.r; row < r1; row += U * b.R) {
        Raw<T, V> q[U];
        float d[U][V];
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (row + i * b.R < r1) {
                q[i] = Raw<T, V>::load(p + (row + i * b.R) * a.C);
                load_vec(a.grad_out, base + (row + i * b.R) * a.C, d[i], a.out_dtype);
            }
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (row + i * b.R < r1) {
                float x[V], z[V];
                q[i].unpack(x);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    x[e] = (x[e] - mu[e]) * rs[e];
                    z[e] = fmaf(x[e], w[e], bi[e]);
                }
                activate_grad(d[i], z, a.act);
#pragma unroll
                for (int e = 0; e < V; ++e)
                    z[e] = rs[e] * (fmaf(w[e], d[i][e], -c1[e]) - x[e] * c2[e]);
                store_as(static_cast<T*>(a.grad_x) + base + (row + i * b.R) * a.C, z);
            }
    }
}

// ---- an image's slab in one workgroup ----------------------------------------------------
//
// Where a slab of one image fits the registers of a workgroup, it is read once, its
// statistics are formed there and it is normalised and written from there: the floor of
// traffic, one launch.  Consecutive slabs go to one XCD, whose L2 then holds the 128-byte
// lines that two slabs share.  64 x 3136 x 128 bfloat16 (103 MB in and out) takes 29 us, 3.5
// TB/s: each compute unit has one workgroup, which reads, then computes, then writes, and no
// other fills the gaps (a copy of as much takes 21 us).  Small maps are bound by the launch:
// 6 x 176 x 256 binary32 takes 6.0 us.
__device__ __forceinline__ int xcd_run(int id, int total) {
    const int x = id % 8, i = id / 8;
    return x * (total / 8) + min(x, total % 8) + i;
}

template <typename T, int V, int NV, bool STORE>
__global__ __launch_bounds__(kGnWholeThreads) void gn_whole_kernel(GnArgs a) {
    __shared__ float red[kGnWholeThreads * V];
    __shared__ double um[kGnUnits], uq[kGnUnits];
    __shared__ float gm[kGnUnits], gr[kGnUnits];
    const int id = xcd_run(blockIdx.x, a.N * a.slabs);
    const int n = id / a.slabs, s = id - n * a.slabs;
    const Slab b = slab_of<V>(a, s, blockDim.x);
    const int64_t base = (int64_t)n * a.S * a.C + b.ch0 + b.v * V;
    const T* p = static_cast<const T*>(a.x) + base;
    const int S = b.r < b.R ? (int)a.S : 0;
    Raw<T, V> q[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int row = b.r + i * b.R;
        if (row < S) q[i] = Raw<T, V>::load(p + (int64_t)row * a.C);
        else q[i] = Raw<T, V>::zero();
    }
    float first[V], sum[V], sq[V];
    q[0].unpack(first);
    int cnt = b.r < S;
#pragma unroll
    for (int e = 0; e < V; ++e) sum[e] = sq[e] = 0.0f;
    const auto count = [&](const Raw<T, V>& r) {
        float x[V];
        r.unpack(x);
        ++cnt;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const float d = x[e] - first[e];
            sum[e] += d;
            sq[e] = fmaf(d, d, sq[e]);
        }
    };
#pragma unroll
    for (int i = 1; i < NV; ++i)
        if (b.r + i * b.R < S) count(q[i]);
#pragma unroll
    for (int i = 0; i < NV; ++i) q[i].forget();
    join_threads(a, b, n, a.share, cnt, first, sum, sq, red, um, uq);
    for (int u = threadIdx.x; u < b.nunits; u += blockDim.x) {
        gm[u] = (float)(um[u] + (double)origin_of(a, n, b.g0 + u));
        gr[u] = rstd_of(uq[u] * a.share, a.eps);
        if (a.mean) a.mean[(int64_t)n * a.G + b.g0 + u] = gm[u];
        if (a.rstd) a.rstd[(int64_t)n * a.G + b.g0 + u] = gr[u];
    }
    if constexpr (STORE) {
        __syncthreads();
        float mu[V], sc[V], bi[V];
        int u[V];
        units_of(b, a.cpg, u);
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const int c = b.v * V + e;
            mu[e] = gm[u[e]];
            sc[e] = gr[u[e]] * (a.weight ? a.weight[b.ch0 + c] : 1.0f);
            bi[e] = a.bias ? a.bias[b.ch0 + c] : 0.0f;
        }
        const auto write = [&](auto act, auto same) {
            const auto put = [&](const Raw<T, V>& r, int row) {
                float z[V];
                r.unpack(z);
#pragma unroll
                for (int e = 0; e < V; ++e) z[e] = fmaf(z[e] - mu[e], sc[e], bi[e]);
                activate(z, act);
                const int64_t at = base + (int64_t)row * a.C;
                if constexpr (same) store_as(static_cast<T*>(a.out) + at, z);
                else store_vec(a.out, at, z, a.out_dtype);
            };
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (b.r + i * b.R < S) put(q[i], b.r + i * b.R);
        };
        with_activation(a.act, [&](auto act) {
            if (a.out_dtype == a.x_dtype) write(act, std::true_type{});
            else write(act, std::false_type{});
        });
    }
}

// The same for the gradients (grad_out of x's type): dz stays in registers in binary32, so the
// derivative of the activation is formed once.  64 x 784 x 256 bfloat16 with SiLU (77 MB in and
// out) takes 30.8 us and 4.0 us for the channels' sums behind it (floor 12 us); as in the
// forward a compute unit reads, computes and writes by turns.  Where no slab fits, 3 x 1665 x 96
// binary16 (2.9 MB) takes 16 us by chunks: 10 and 7 us of two launches of 60 workgroups, whose
// loads, joins and exchanges follow one another.
template <typename T, int V, int NV>
__global__ __launch_bounds__(kGnWholeBwdThreads) void gn_bwd_whole_kernel(GnArgs a) {
    __shared__ float ra[kGnWholeBwdThreads * V], rb[kGnWholeBwdThreads * V];
    __shared__ float ua[kGnUnits], ub[kGnUnits];
    const int id = xcd_run(blockIdx.x, a.N * a.slabs);
    const int n = id / a.slabs, s = id - n * a.slabs;
    const Slab b = slab_of<V>(a, s, blockDim.x);
    const int64_t base = (int64_t)n * a.S * a.C + b.ch0 + b.v * V;
    const T* p = static_cast<const T*>(a.x) + base;
    const T* gp = static_cast<const T*>(a.grad_out) + base;
    const int S = b.r < b.R ? (int)a.S : 0;
    Raw<T, V> q[NV], dq[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int row = b.r + i * b.R;
        if (row < S) {
            q[i] = Raw<T, V>::load(p + (int64_t)row * a.C);
            dq[i] = Raw<T, V>::load(gp + (int64_t)row * a.C);
        } else {
            q[i] = dq[i] = Raw<T, V>::zero();
        }
    }
    const float* mean = a.mean + (int64_t)n * a.G + b.g0;
    const float* rstd = a.rstd + (int64_t)n * a.G + b.g0;
    float dz[NV][V], A[V], B[V];
    int u[V];
    units_of(b, a.cpg, u);
    {
        float mu[V], sc[V], bi[V];
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const int c = b.v * V + e, j = u[e];
            mu[e] = mean[j];
            sc[e] = rstd[j] * (a.weight ? a.weight[b.ch0 + c] : 1.0f);
            bi[e] = a.bias ? a.bias[b.ch0 + c] : 0.0f;
            A[e] = B[e] = 0.0f;
        }
        with_activation(a.act, [&](auto act) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float x[V], z[V];
                q[i].unpack(x);
                dq[i].unpack(dz[i]);   // zeros past the last row
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    x[e] -= mu[e];
                    z[e] = fmaf(x[e], sc[e], bi[e]);
                }
                activate_grad(dz[i], z, act);
                if (b.r + i * b.R < S) {
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        A[e] += dz[i][e];
                        B[e] = fmaf(dz[i][e], x[e], B[e]);
                    }
                }
            }
        });
#pragma unroll
        for (int e = 0; e < V; ++e) B[e] *= rstd[u[e]];
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) q[i].forget();
    fold_rows(b, A, B, ra, rb);
    float2* cp = a.chan_part + (int64_t)n * a.C + b.ch0;
    for (int c = threadIdx.x; c < b.width; c += blockDim.x) {
        cp[c] = make_float2(ra[c], rb[c]);
        const float w = a.weight ? a.weight[b.ch0 + c] : 1.0f;
        ra[c] *= w;
        rb[c] *= w;
    }
    if (!a.grad_x) return;
    __syncthreads();
    unit_sums(ra, 1, b.width, a.cpg, b.nunits, a.share, ua);
    unit_sums(rb, 1, b.width, a.cpg, b.nunits, a.share, ub);
    // rstd * (w dz - m1 - xhat m2) as two multiply-adds
    float mu[V], k1[V], k2[V], k3[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
        const int c = b.v * V + e, j = u[e];
        mu[e] = mean[j];
        const float rs = rstd[j];
        k1[e] = rs * (a.weight ? a.weight[b.ch0 + c] : 1.0f);
        k2[e] = -rs * rs * ub[j];
        k3[e] = -rs * ua[j];
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int row = b.r + i * b.R;
        if (row < S) {
            float x[V];
            q[i].unpack(x);
#pragma unroll
            for (int e = 0; e < V; ++e)
                x[e] = fmaf(dz[i][e], k1[e], fmaf(x[e] - mu[e], k2[e], k3[e]));
            store_as(static_cast<T*>(a.grad_x) + base + (int64_t)row * a.C, x);
        }
    }
}

// ---- launches ----------------------------------------------------------------------------

template <typename T, int V, bool STORE>
hipError_t forward_whole(const GnArgs& a, hipStream_t stream) {
    const uint32_t blocks = (uint32_t)(a.N * a.slabs);
    if (a.vecs <= 4) gn_whole_kernel<T, V, 4, STORE><<<blocks, a.threads, 0, stream>>>(a);
    else if (a.vecs <= 8) gn_whole_kernel<T, V, 8, STORE><<<blocks, a.threads, 0, stream>>>(a);
    else gn_whole_kernel<T, V, kGnWholeVecs, STORE><<<blocks, a.threads, 0, stream>>>(a);
    return hipGetLastError();
}

uint32_t join_blocks(const GnArgs& a) {
    return (uint32_t)(a.N * ((a.G + kGnJoin - 1) / kGnJoin));
}

template <typename T, int V>
hipError_t forward_stats(const GnArgs& a, hipStream_t stream) {
    if (a.threads) return forward_whole<T, V, false>(a, stream);
    const uint32_t blocks = (uint32_t)((int64_t)a.N * a.chunks * a.slabs);
    gn_stats_kernel<T, V><<<blocks, kGnThreads, 0, stream>>>(a);
    gn_join_kernel<<<join_blocks(a), kGnThreads, 0, stream>>>(a);
    return hipGetLastError();
}

template <typename T, int V>
hipError_t forward(const GnArgs& a, hipStream_t stream) {
    if (a.threads) return forward_whole<T, V, true>(a, stream);
    const uint32_t blocks = (uint32_t)((int64_t)a.N * a.chunks * a.slabs);
    gn_stats_kernel<T, V><<<blocks, kGnThreads, 0, stream>>>(a);
    gn_apply_kernel<T, V><<<blocks, kGnThreads, 0, stream>>>(a);
    return hipGetLastError();
}

template <typename T, int V>
hipError_t backward(const GnArgs& a, hipStream_t stream) {
    const int64_t blocks = (int64_t)a.N * a.chunks * a.slabs;
    const int64_t ch = a.grad_weight || a.grad_bias ? (a.C + kGnChanBlock - 1) / kGnChanBlock : 0;
    int64_t dx = 0;
    if (blocks && a.threads) {
        if (a.vecs <= 2)
            gn_bwd_whole_kernel<T, V, 2><<<(uint32_t)blocks, a.threads, 0, stream>>>(a);
        else if (a.vecs <= 4)
            gn_bwd_whole_kernel<T, V, 4><<<(uint32_t)blocks, a.threads, 0, stream>>>(a);
        else
            gn_bwd_whole_kernel<T, V, 8><<<(uint32_t)blocks, a.threads, 0, stream>>>(a);
    } else if (blocks) {
        gn_bwd_stats_kernel<T, V><<<(uint32_t)blocks, kGnThreads, 0, stream>>>(a);
        if (a.grad_x) dx = blocks;
    }
    if (dx + ch)
        gn_bwd_apply_kernel<T, V><<<(uint32_t)(dx + ch), kGnThreads, 0, stream>>>(a, dx);
    return hipGetLastError();
}

template <typename F>
hipError_t by_type(int dtype, bool vec, F&& f) {
    switch (dtype) {
        case DA_BF16: return vec ? f(__bf16{}, std::integral_constant<int, 8>{})
                                 : f(__bf16{}, std::integral_constant<int, 1>{});
        case DA_F16: return vec ? f(_Float16{}, std::integral_constant<int, 8>{})
                                : f(_Float16{}, std::integral_constant<int, 1>{});
        default: return vec ? f(float{}, std::integral_constant<int, 4>{})
                            : f(float{}, std::integral_constant<int, 1>{});
    }
}

}  // namespace

hipError_t launch_gn_stats(const GnArgs& a, bool vec, hipStream_t stream) {
    return by_type(a.x_dtype, vec, [&](auto t, auto v) {
        return forward_stats<decltype(t), decltype(v)::value>(a, stream);
    });
}

hipError_t launch_gn_forward(const GnArgs& a, bool vec, hipStream_t stream) {
    return by_type(a.x_dtype, vec, [&](auto t, auto v) {
        return forward<decltype(t), decltype(v)::value>(a, stream);
    });
}

hipError_t launch_gn_backward(const GnArgs& a, bool vec, hipStream_t stream) {
    return by_type(a.x_dtype, vec, [&](auto t, auto v) {
        return backward<decltype(t), decltype(v)::value>(a, stream);
    });
}

}  // namespace da
