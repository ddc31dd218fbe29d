// Internal launch description of the 8-bit products (i8.hip), filled by the host API
// (i8_api.cpp).  Not part of the public ABI.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#include "gn_internal.h"

namespace da {

struct I8Args {
    const void* x;            // [M, K] of x_dtype (quantising kernels)
    int8_t* a;                // [M, K] codes (workspace where x is quantised first)
    float* a_scale;           // [M]
    const int8_t* w;          // [N, K]
    const float* w_scale;     // [N]
    const float* bias;        // [N] or NULL
    void* out;                // [M, N] of out_dtype
    int64_t M;
    int32_t K, N;
    int32_t act, x_dtype, out_dtype;
    int32_t slices;           // rows kernel: slices of the output channels
    int32_t tiles_per_slice;  // rows kernel: 16-channel tiles of a slice
    int32_t blocks_per_image; // rows kernel: workgroups that share an image's rows
    int32_t staged;           // rows kernel: results leave by way of LDS
    // a row passes through group norm and an activation before it is quantised
    const float* norm_weight; // [K] or NULL
    const float* norm_bias;   // [K] or NULL
};

// Which kernels a problem takes; the workspace goes by it.
enum class I8Path {
    kRows,      // one kernel that quantises its rows itself
    kSkinny,    // one kernel, few rows: the weights are streamed once
    kTiles,     // quantised rows in memory, then a tiled product
    kSkinnyCodes,  // quantised rows in memory, then the streaming kernel
};
I8Path i8_path(int64_t M, int64_t K, int64_t N, bool codes, bool norm);

hipError_t launch_i8_quantize(const I8Args& a, const GnArgs* norm, hipStream_t stream);
// The product on `path`; quantising paths read x, the others a and a_scale.
hipError_t launch_i8_product(const I8Args& a, I8Path path, bool codes, const GnArgs* norm,
                             hipStream_t stream);

}  // namespace da
