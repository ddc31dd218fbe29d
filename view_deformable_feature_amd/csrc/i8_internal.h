// Internal launch description of the 8-bit products (i8.hip), filled by the host API
// (i8_api.cpp).  Not part of the public ABI.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

namespace da {

struct I8Args {
    const void* x;            // [M, K] of x_dtype (quantising kernels)
    int8_t* a;                // [M, K] codes
    float* a_scale;           // [M]
    const int8_t* w;          // [N, K]
    const float* w_scale;     // [N]
    const float* bias;        // [N] or NULL
    void* out;                // [M, N] of out_dtype
    int64_t M;
    int32_t K, N;
    int32_t act, x_dtype, out_dtype;
    // a row passes through group norm and an activation before it is quantised
    const float* mean;        // [images, G], or NULL
    const float* rstd;        // [images, G]
    const float* norm_weight; // [K] or NULL
    const float* norm_bias;   // [K] or NULL
    int64_t S;                // rows of an image
    int32_t G, cpg, norm_act;
};

hipError_t launch_i8_quantize(const I8Args& a, hipStream_t stream);
hipError_t launch_i8_matmul(const I8Args& a, hipStream_t stream);

}  // namespace da
