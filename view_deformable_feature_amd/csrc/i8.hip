// Products of 8-bit codes with a scale per row and output channel, and the quantisation
// of rows to such codes.  Contract and formulas: include/int8.h.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "act_device.h"
#include "i8_internal.h"

namespace da {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

// A row's scale and the factor its codes are formed with, from the largest magnitude's
// bits (magnitudes order as their bits do, infinities and NaNs last).
__device__ __forceinline__ void row_scale(uint32_t big_bits, float& scale, float& inverse) {
    const float big = __uint_as_float(big_bits);
    if (big_bits >= 0x7f800000u) {
        scale = __uint_as_float(0x7fc00000u);
        inverse = 0.0f;
    } else if (big < 0x1p-100f) {
        scale = inverse = 0.0f;
    } else {
        scale = big / 127.0f;
        inverse = 127.0f / big;
    }
}

__device__ __forceinline__ int code_of(float x, float inverse) {
    // a row with a NaN or an infinity has inverse 0 and its codes are 0 whatever x is
    const float q = rintf(x * inverse);
    return inverse == 0.0f ? 0 : (int)q;
}

// One wave per row, read twice (the second time from cache).
constexpr int kQuantThreads = 256;
__global__ __launch_bounds__(kQuantThreads) void i8_quantize_kernel(I8Args a) {
    const int64_t m = (int64_t)blockIdx.x * (kQuantThreads / kWave) + threadIdx.x / kWave;
    const int lane = threadIdx.x & (kWave - 1);
    if (m >= a.M) return;
    const auto value = [&](int k) {
        float v[1] = {load_elem(a.x, m * a.K + k, a.x_dtype)};
        if (a.mean) {
            const int64_t j = m / a.S * a.G + k / a.cpg;
            const float w = a.norm_weight ? a.norm_weight[k] : 1.0f;
            v[0] = fmaf(v[0] - a.mean[j], a.rstd[j] * w, a.norm_bias ? a.norm_bias[k] : 0.0f);
            activate(v, a.norm_act);
        }
        return v[0];
    };
    uint32_t big = 0;
    for (int k = lane; k < a.K; k += kWave) big = max(big, __float_as_uint(value(k)) & 0x7fffffffu);
    for (int s = kWave / 2; s; s >>= 1) big = max(big, (uint32_t)__shfl_xor((int)big, s));
    float scale, inverse;
    row_scale(big, scale, inverse);
    for (int k = lane; k < a.K; k += kWave) a.a[m * a.K + k] = (int8_t)code_of(value(k), inverse);
    if (lane == 0) a.a_scale[m] = scale;
}

// 16 bytes of row `row` from column k on, zeros outside the matrix.
__device__ __forceinline__ i32x4 piece(const int8_t* p, int64_t row, int64_t rows, int k, int K) {
    i32x4 q = {0, 0, 0, 0};
    if (row < rows)
        for (int i = 0; i < 16; ++i)
            if (k + i < K) q[i / 4] |= (int)((uint32_t)(uint8_t)p[row * K + k + i] << (8 * (i % 4)));
    return q;
}

// A wave forms 16 rows x 64 columns.
__global__ __launch_bounds__(256) void i8_matmul_kernel(I8Args a) {
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int tiles = (a.N + 63) / 64;
    const int64_t m0 = (int64_t)(blockIdx.x / tiles) * 64 + wave * 16;
    const int n0 = (int)(blockIdx.x % tiles) * 64;
    i32x4 acc[4] = {};
    for (int k = 0; k < a.K; k += 64) {
        const i32x4 fa = piece(a.a, m0 + lane % 16, a.M, k + lane / 16 * 16, a.K);
        for (int j = 0; j < 4; ++j) {
            const i32x4 fb = piece(a.w, n0 + j * 16 + lane % 16, a.N, k + lane / 16 * 16, a.K);
            acc[j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fa, fb, acc[j], 0, 0, 0);
        }
    }
    for (int j = 0; j < 4; ++j) {
        const int n = n0 + j * 16 + lane % 16;
        for (int i = 0; i < 4; ++i) {
            const int64_t m = m0 + lane / 16 * 4 + i;
            if (m < a.M && n < a.N) {
                float y[1] = {(float)acc[j][i] * a.a_scale[m] * a.w_scale[n]};
                if (a.bias) y[0] += a.bias[n];
                activate(y, a.act);
                store_vec(a.out, m * a.N + n, y, a.out_dtype);
            }
        }
    }
}

}  // namespace

hipError_t launch_i8_quantize(const I8Args& a, hipStream_t stream) {
    const uint32_t blocks = (uint32_t)((a.M + 3) / 4);
    i8_quantize_kernel<<<blocks, kQuantThreads, 0, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_i8_matmul(const I8Args& a, hipStream_t stream) {
    const uint32_t blocks = (uint32_t)((a.M + 63) / 64 * ((a.N + 63) / 64));
    i8_matmul_kernel<<<blocks, 256, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace da
