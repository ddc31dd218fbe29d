// Group-norm statistics as kernels read them: the chunks' partial results (gn.hip) joined
// into means and reciprocal standard deviations.  Device code.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "act_device.h"
#include "gn_internal.h"

namespace da {

__device__ __forceinline__ double wave_sum(double t) {
    for (int m = kWave / 2; m; m >>= 1) t += __shfl_xor(t, m);
    return t;
}

// The group's first value in image n: all of the group's means are formed and kept as
// differences from it, so that a large common offset cancels before anything is rounded.
__device__ __forceinline__ float origin_of(const GnArgs& a, int n, int g) {
    return load_elem(a.x, (int64_t)n * a.S * a.C + (int64_t)g * a.cpg, a.x_dtype);
}

// The chunks' statistics of groups g0 .. g0 + ngroups - 1 joined in binary64, one wave
// per group: mean and rstd into LDS.  Every thread of the workgroup calls it.
__device__ __forceinline__ void join_stats(const GnArgs& a, int n, int g0, int ngroups, float* gm,
                                           float* gr) {
    const int lane = threadIdx.x & (kWave - 1), nw = blockDim.x / kWave;
    const double total = (double)a.S * a.cpg;
    for (int j = threadIdx.x / kWave; j < ngroups; j += nw) {
        const int g = g0 + j;
        const float2* part = a.unit_part + (int64_t)n * a.chunks * a.units + (int64_t)g * a.upg;
        const int entries = a.chunks * a.upg;
        double sum = 0.0, m2 = 0.0;
        for (int e = lane; e < entries; e += kWave) {
            const int c = e / a.upg, u = e - c * a.upg;
            const int64_t r0 = c * a.rows_per_chunk;
            const double cnt = (double)(min(r0 + a.rows_per_chunk, a.S) - r0) *
                               min(a.cpu, a.cpg - u * a.cpu);
            sum += cnt * part[(int64_t)c * a.units + u].x;
        }
        const double mean = wave_sum(sum) / total;
        for (int e = lane; e < entries; e += kWave) {
            const int c = e / a.upg, u = e - c * a.upg;
            const int64_t r0 = c * a.rows_per_chunk;
            const double cnt = (double)(min(r0 + a.rows_per_chunk, a.S) - r0) *
                               min(a.cpu, a.cpg - u * a.cpu);
            const float2 q = part[(int64_t)c * a.units + u];
            m2 += q.y + cnt * (q.x - mean) * (q.x - mean);
        }
        const double var = wave_sum(m2) / total;
        if (lane == 0) {
            gm[j] = (float)(mean + (double)origin_of(a, n, g));
            // squares past binary32: no number
            gr[j] = var < 0x1p1000 ? (float)(1.0 / sqrt(var + (double)a.eps))
                                   : __uint_as_float(0x7fc00000u);
        }
    }
    __syncthreads();
}

}  // namespace da
