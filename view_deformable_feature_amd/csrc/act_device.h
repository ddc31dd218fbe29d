// Activations and 16-byte vector access shared by the group norm (gn.hip) and the
// 8-bit products (i8.hip).  Device code.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "da_device.h"
#include "group_norm.h"

namespace da {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// sigmoid(z) by the hardware's exponential and reciprocal (one unit in the last place
// each): exp(-z) is off by 2^-23 + |z| 2^-24 of itself, so the result is off by that
// share of 1 - sigmoid(z) at most.
__device__ __forceinline__ float sigmoid_f(float z) {
    return __builtin_amdgcn_rcpf(1.0f + __expf(-z));
}

// Phi(z), the standard normal distribution function; e is exp(-z^2 / 2), which the density
// needs as well.  Phi(-|z|) = e * f(t) with t = 1 / (1 + 0.4 |z| / sqrt 2), and f, half the
// scaled complementary error function, is t times the polynomial of degree 8 in t whose largest
// relative deviation over |z| <= 13.4 (beyond, e leaves binary32) is least: 2^-24, found by
// exchanging its extrema.  With the roundings of t, the sum and the exponential the result is off
// by at most (24 + 2 z^2) 2^-24 of itself, in the lower tail too, where 1 + erf(z / sqrt 2) has no
// digits left.  One range for all arguments: erff has two, which a wave runs through one after
// the other.
__device__ __forceinline__ float normal_cdf(float z, float& e) {
    e = __expf(-0.5f * z * z);
    const float t = __builtin_amdgcn_rcpf(fmaf(0.28284271f, fabsf(z), 1.0f));
    float p = fmaf(t, 0.0201337319f, -0.0677354659f);
    p = fmaf(t, p, 0.0369209123f);
    p = fmaf(t, p, 0.0498649666f);
    p = fmaf(t, p, 0.0357540387f);
    p = fmaf(t, p, 0.0984815590f);
    p = fmaf(t, p, 0.1004792810f);
    p = fmaf(t, p, 0.1132878560f);
    p = fmaf(t, p, 0.1128131490f);
    const float tail = t * p * e;
    return z < 0.0f ? tail : 1.0f - tail;
}

template <int V>
__device__ __forceinline__ void activate(float (&z)[V], int act) {
    if (act == DA_ACT_RELU) {
#pragma unroll
        for (int e = 0; e < V; ++e) z[e] = z[e] < 0.0f ? 0.0f : z[e];   // a NaN stays one
    } else if (act == DA_ACT_SILU) {
#pragma unroll
        for (int e = 0; e < V; ++e) z[e] *= sigmoid_f(z[e]);
    } else if (act == DA_ACT_GELU) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
            float density;
            z[e] *= normal_cdf(z[e], density);
        }
    }
}

// d[e] *= act'(z[e])
template <int V>
__device__ __forceinline__ void activate_grad(float (&d)[V], const float (&z)[V], int act) {
    if (act == DA_ACT_RELU) {
#pragma unroll
        for (int e = 0; e < V; ++e) d[e] = z[e] <= 0.0f ? 0.0f : d[e];
    } else if (act == DA_ACT_SILU) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const float s = sigmoid_f(z[e]);
            d[e] *= s * (1.0f + z[e] * (1.0f - s));
        }
    } else if (act == DA_ACT_GELU) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
            float density;
            const float cdf = normal_cdf(z[e], density);
            d[e] *= fmaf(z[e] * 0.39894228f, density, cdf);
        }
    }
}

// f with the activation as a constant: loops inside f then have no branch on it.
template <typename F>
__device__ __forceinline__ void with_activation(int act, F&& f) {
    switch (act) {
        case DA_ACT_RELU: f(std::integral_constant<int, DA_ACT_RELU>{}); break;
        case DA_ACT_SILU: f(std::integral_constant<int, DA_ACT_SILU>{}); break;
        case DA_ACT_GELU: f(std::integral_constant<int, DA_ACT_GELU>{}); break;
        default: f(std::integral_constant<int, DA_ACT_NONE>{});
    }
}

// Raw storage of V elements of T, moved in one access: V = 16 bytes' worth, or 1.
template <typename T, int V>
struct Raw {
    u32x4 q;
    static __device__ __forceinline__ Raw load(const T* p) {
        return {*reinterpret_cast<const u32x4*>(p)};
    }
    static __device__ __forceinline__ Raw zero() { return {u32x4{0, 0, 0, 0}}; }
    // Makes the compiler forget what it knows of the value, so that what was unpacked from it
    // before is not kept in registers for the next time.
    __device__ __forceinline__ void forget() { asm volatile("" : "+v"(q)); }
    __device__ __forceinline__ void unpack(float (&v)[V]) const {
        typedef T vec __attribute__((ext_vector_type(V)));
        const vec t = __builtin_bit_cast(vec, q);
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] = (float)t[e];
    }
};
template <typename T>
struct Raw<T, 1> {
    T t;
    static __device__ __forceinline__ Raw load(const T* p) { return {*p}; }
    static __device__ __forceinline__ Raw zero() { return {(T)0.0f}; }
    __device__ __forceinline__ void forget() {}
    __device__ __forceinline__ void unpack(float (&v)[1]) const { v[0] = (float)t; }
};

// Store V floats as elements of D at p (aligned to min(16, V * sizeof(D)) bytes), each
// rounded once to nearest even.
template <typename D, int V>
__device__ __forceinline__ void store_as(D* p, const float (&v)[V]) {
    if constexpr (V == 1) {
        *p = (D)v[0];
    } else {
        constexpr int kPer = V * (int)sizeof(D) <= 16 ? V : 16 / (int)sizeof(D);
        typedef D vec __attribute__((ext_vector_type(kPer)));
#pragma unroll
        for (int b = 0; b < V; b += kPer) {
            vec t;
#pragma unroll
            for (int e = 0; e < kPer; ++e) t[e] = (D)v[b + e];
            *reinterpret_cast<vec*>(p + b) = t;
        }
    }
}
template <int V>
__device__ __forceinline__ void store_vec(void* base, int64_t i, const float (&v)[V], int dtype) {
    if (dtype == DA_BF16)
        store_as(static_cast<__bf16*>(base) + i, v);
    else if (dtype == DA_F16)
        store_as(static_cast<_Float16*>(base) + i, v);
    else
        store_as(static_cast<float*>(base) + i, v);
}

template <typename D, int V>
__device__ __forceinline__ void load_as(const D* p, float (&v)[V]) {
    if constexpr (V == 1) {
        v[0] = (float)*p;
    } else {
        constexpr int kPer = V * (int)sizeof(D) <= 16 ? V : 16 / (int)sizeof(D);
        typedef D vec __attribute__((ext_vector_type(kPer)));
#pragma unroll
        for (int b = 0; b < V; b += kPer) {
            const vec t = *reinterpret_cast<const vec*>(p + b);
#pragma unroll
            for (int e = 0; e < kPer; ++e) v[b + e] = (float)t[e];
        }
    }
}
template <int V>
__device__ __forceinline__ void load_vec(const void* base, int64_t i, float (&v)[V], int dtype) {
    if (dtype == DA_BF16)
        load_as(static_cast<const __bf16*>(base) + i, v);
    else if (dtype == DA_F16)
        load_as(static_cast<const _Float16*>(base) + i, v);
    else
        load_as(static_cast<const float*>(base) + i, v);
}

}  // namespace da
