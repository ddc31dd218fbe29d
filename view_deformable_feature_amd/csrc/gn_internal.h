// Internal launch description of the group-norm kernels (gn.hip), filled by the host
// API (gn_api.cpp).  Not part of the public ABI.
//
// A workgroup covers a slab: slab_ch consecutive channels (whole groups, and whole
// vectors of VEC channels) of some rows of one image.  Its threads form R rows of
// slab_ch / VEC vectors; a thread keeps its vector of channels and walks the rows.  A
// group wider than kGnThreads vectors is cut into upg units of cpu channels (the last
// one shorter), one to a slab; otherwise a unit is a group.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#include "group_norm.h"

namespace da {

constexpr int kGnThreads = 256;
// A slab of a whole image in one workgroup: at most so many threads, and vectors to a thread.
// The forward keeps 64 registers of x of the 128 that 1024 threads may have (with 16 vectors of 16
// bits it spills 4 of the others), the backward 32 of x and 64 of dz (with 1024 threads it
// spilled 45 of them at half as many vectors).
constexpr int kGnWholeThreads = 1024, kGnWholeVecs = 16;
constexpr int kGnWholeBwdThreads = 512, kGnWholeBwdVecs = 8;
// Units of any slab: groups of one channel each, 256 bytes of a row hold the most (a slab is wider
// only where a single group, or a few that share vectors, are).
constexpr int kGnUnits = 128;

struct GnArgs {
    const void* x;            // [N, S, C] of x_dtype
    const float* weight;      // [C] or NULL
    const float* bias;        // [C] or NULL
    void* out;                // [N, S, C] of out_dtype
    float* mean;              // [N, G] or NULL (read in the backward)
    float* rstd;              // [N, G] or NULL
    const void* grad_out;     // [N, S, C] of out_dtype
    void* grad_x;             // [N, S, C] of x_dtype, or NULL
    float* grad_weight;       // [C] or NULL
    float* grad_bias;         // [C] or NULL
    float* origins;           // [N, G]: the groups' first values, which means are taken from
    double2* stat_part;       // [N, chunks, units]: mean less that, sum of squared deviations
    float2* unit_part;        // backward: [N, chunks, units] sums of weight * dz and weight * dz * xhat
    float2* chan_part;        // backward: [N, chunks, C] sums of dz and dz * xhat
    int64_t S;
    int64_t rows_per_chunk;
    double share;             // 1 / (S * cpg), the weight of a value in its group's averages
    int32_t N, C, G, cpg;
    int32_t slab_ch, slabs;
    int32_t upg, cpu, units;
    int32_t chunks;           // row chunks of an image (statistics and apply alike)
    int32_t threads, vecs;    // an image's slab in one workgroup (chunks 1): threads, vectors
                              // per thread; 0: by chunks
    int32_t act, x_dtype, out_dtype;
    float eps;
};

// Statistics alone, for a kernel that normalises as it reads: workspace bytes (and the
// problem's checks); then a filled in and mean and rstd [N, G] enqueued into that workspace
// (256-byte aligned).
da_status gn_stats_bytes(const gn_problem* p, uint64_t& bytes);
hipError_t enqueue_gn_stats(const gn_problem* p, const void* x, void* workspace, GnArgs& a,
                            hipStream_t stream);

hipError_t launch_gn_stats(const GnArgs& a, bool vec, hipStream_t stream);
hipError_t launch_gn_forward(const GnArgs& a, bool vec, hipStream_t stream);
hipError_t launch_gn_backward(const GnArgs& a, bool vec, hipStream_t stream);

}  // namespace da
