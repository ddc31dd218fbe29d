// Internal launch description of the rotation kernels (rope.hip), filled by the host API
// (rope_api.cpp).  Not part of the public ABI.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#include "rotary.h"

namespace da {

constexpr int kRopeThreads = 256;

// One tensor of a launch.
struct RopeSide {
    const void* x;            // [B, N, H, D], strided
    void* y;                  // the result, strided; in the backward grad_y
    void* dx;                 // backward: [B, N, H, D] or NULL
    const void* positions;
    const float* weight;      // [D] or NULL
    float* grad_weight;       // backward: [D] or NULL
    float* part;              // backward: [blocks, D] sums of the workgroups
    int64_t x_batch, x_token, x_head;   // strides in elements
    int64_t y_batch, y_token, y_head;
    int64_t pos_batch;
    int64_t tokens;           // of all batch entries
    int32_t N, H;
    int32_t pos_type;
    int32_t abreast;          // heads of a token that a workgroup has side by side
    int32_t blocks;           // workgroups
};

struct RopeArgs {
    RopeSide side[2];
    const double* freqs;
    int32_t sides, D, R;
    int32_t units;            // pairs of vectors of a head
    int32_t lanes;            // of a head: a power of two, units <= lanes * units a lane
    float eps, magnitude, sign;
    int32_t layout, dtype;
};

// vec: numbers of a vector (1, 2, 4, 8); per_lane: units to a lane (1, 2, 4)
hipError_t launch_rope(const RopeArgs& a, bool norm, int vec, int per_lane, hipStream_t stream);
hipError_t launch_rope_norm_backward(const RopeArgs& a, int vec, int per_lane, hipStream_t stream);

}  // namespace da
