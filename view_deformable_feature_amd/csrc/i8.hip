// Products of 8-bit codes with a scale per row and output channel, and the quantisation
// of rows to such codes.  Contract and formulas: include/int8.h.
//
// The matrix instruction v_mfma_i32_16x16x64_i8 takes 16 rows of 64 consecutive codes of
// either operand, 16 bytes of row l % 16 at byte 16 * (l / 16) in lane l, and leaves in
// lane l four sums: rows 4 * (l / 16) .. + 3 of the first operand with row l % 16 of the
// second.  The weights are the first operand throughout, so a lane ends up with four
// consecutive output channels of one row and stores them at once.
//
// Columns past K are zeros in both operands.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "act_device.h"
#include "i8_internal.h"

namespace da {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ i32x4 mfma(i32x4 w, i32x4 x, i32x4 acc) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(w, x, acc, 0, 0, 0);
}

// ---- quantisation ------------------------------------------------------------------------

// A row's scale and the factor its codes are formed with, from the largest magnitude's
// bits (magnitudes order as their bits do, infinities and NaNs last).  Both quotients are
// the correctly rounded ones.
struct RowScale {
    float scale, inverse;
    uint32_t mask;   // 0 where every code is 0 whatever x * inverse is
};
__device__ __forceinline__ RowScale row_scale(uint32_t big_bits) {
    const float big = __uint_as_float(big_bits);
    if (big_bits >= 0x7f800000u) return {__uint_as_float(0x7fc00000u), 0.0f, 0u};
    if (big < 0x1p-100f) return {0.0f, 0.0f, 0u};
    return {big / 127.0f, 127.0f / big, ~0u};
}

// Four codes.  Adding 1.5 * 2^23 to the rounded product rounds it once more, to the nearest
// whole number, ties to even, and leaves it in the low byte in two's complement; the two
// steps must not become one multiply-add, which would round once.
__device__ __forceinline__ uint32_t pack_codes(const float* x, const RowScale& s) {
#pragma clang fp contract(off)
    constexpr float kMagic = 12582912.0f;
    const uint32_t q0 = __float_as_uint(x[0] * s.inverse + kMagic);
    const uint32_t q1 = __float_as_uint(x[1] * s.inverse + kMagic);
    const uint32_t q2 = __float_as_uint(x[2] * s.inverse + kMagic);
    const uint32_t q3 = __float_as_uint(x[3] * s.inverse + kMagic);
    const uint32_t lo = __builtin_amdgcn_perm(q1, q0, 0x0c0c0400u);
    const uint32_t hi = __builtin_amdgcn_perm(q3, q2, 0x0c0c0400u);
    return __builtin_amdgcn_perm(hi, lo, 0x05040100u) & s.mask;
}

// Eight numbers of a row from column c on, XB bytes each; zeros past column K.  Any
// alignment.
template <int XB>
struct Eight {
    u32x4 q[XB / 2];
    __device__ __forceinline__ void load(const void* x, int64_t row, int c, int K) {
        const char* p = static_cast<const char*>(x) + (row * K + c) * XB;
        if (c + 8 <= K) {
            __builtin_memcpy(q, p, 8 * XB);
        } else {
            uint32_t w[2 * XB];
#pragma unroll
            for (int e = 0; e < 2 * XB; ++e) w[e] = 0;
#pragma unroll
            for (int e = 0; e < 7; ++e)
                if (c + e < K) {
                    if constexpr (XB == 4) {
                        __builtin_memcpy(&w[e], p + 4 * e, 4);
                    } else {
                        uint16_t h;
                        __builtin_memcpy(&h, p + 2 * e, 2);
                        w[e / 2] |= (uint32_t)h << (16 * (e & 1));
                    }
                }
            __builtin_memcpy(q, w, 8 * XB);
        }
    }
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t voff) {
#pragma unroll
        for (int i = 0; i < XB / 2; ++i)
            q[i] = __builtin_bit_cast(
                u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, voff + 16 * i, 0, 0));
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < XB / 2; ++i) q[i] = u32x4{0, 0, 0, 0};
    }
    __device__ __forceinline__ void merge(const Eight& o, bool take) {
#pragma unroll
        for (int i = 0; i < XB / 2; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) q[i][e] = take ? o.q[i][e] : q[i][e];
    }
    // the largest magnitude's bits, in the type's own format
    __device__ __forceinline__ uint32_t magnitude() const {
        uint32_t big = 0;
        if constexpr (XB == 4) {
#pragma unroll
            for (int i = 0; i < 8; ++i) big = max(big, q[i / 4][i % 4] & 0x7fffffffu);
            return big;
        } else {
            typedef uint16_t vec __attribute__((ext_vector_type(2)));
            vec m = {0, 0};
#pragma unroll
            for (int i = 0; i < 4; ++i)
                m = __builtin_elementwise_max(m, __builtin_bit_cast(vec, q[0][i] & 0x7fff7fffu));
            return max((uint32_t)m[0], (uint32_t)m[1]);
        }
    }
    static __device__ __forceinline__ uint32_t widen(uint32_t bits, bool bf16) {
        if constexpr (XB == 4) return bits;
        return bf16 ? bits << 16
                    : __float_as_uint((float)__builtin_bit_cast(_Float16, (uint16_t)bits));
    }
    __device__ __forceinline__ void unpack(float (&v)[8], bool bf16) const {
        if constexpr (XB == 4) {
            __builtin_memcpy(v, q, 32);
        } else if (bf16) {
            typedef __bf16 vec __attribute__((ext_vector_type(8)));
            const vec t = __builtin_bit_cast(vec, q[0]);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = (float)t[e];
        } else {
            typedef _Float16 vec __attribute__((ext_vector_type(8)));
            const vec t = __builtin_bit_cast(vec, q[0]);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = (float)t[e];
        }
    }
};

__device__ __forceinline__ uint32_t magnitude(const float (&v)[8]) {
    uint32_t big = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) big = max(big, __float_as_uint(v[e]) & 0x7fffffffu);
    return big;
}

// The normalisation of eight channels of a row, which a lane keeps for all its rows, and the
// activation behind it; columns past K give 0.
struct NormCoef {
    float mu[8], sc[8], bi[8];
    __device__ __forceinline__ void apply(float (&v)[8], int act) const {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = fmaf(v[e] - mu[e], sc[e], bi[e]);
        activate(v, act);
    }
    // of channels c .. c + 7 of image n
    __device__ __forceinline__ void load(const I8Args& a, const GnArgs& g, int64_t n, int c) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            mu[e] = sc[e] = bi[e] = 0.0f;   // a column past K holds 0
            if (c + e < a.K) {
                const int64_t j = n * g.G + (c + e) / g.cpg;
                mu[e] = g.mean[j];
                sc[e] = g.rstd[j] * (a.norm_weight ? a.norm_weight[c + e] : 1.0f);
                if (a.norm_bias) bi[e] = a.norm_bias[c + e];
            }
        }
    }
};

// Rows to codes and scales in memory: for a caller, and before the kernels that read codes.
// Bound by memory (65536 x 1024 bfloat16, 201 MB, 47 us, 4.3 TB/s), and by its own latency for few
// rows (1237 x 1000 of 16 bits, 3.7 MB: 4.4 us).
// L lanes to a row, 64 / L rows to a wave; a row's first HOLD pieces per lane stay in
// registers, what is past them is read again.  Behind a norm L is 64, and a wave has up to 8
// consecutive rows of one image, for which it keeps the coefficients of the pieces held.
constexpr int kQuantThreads = 256, kQuantWaves = kQuantThreads / kWave;
template <int XB, bool NORM, int L, int HOLD>
__global__ __launch_bounds__(kQuantThreads) void i8_quantize_kernel(I8Args a, GnArgs g,
                                                                     int rows_per_wave) {
    const int lane = threadIdx.x & (kWave - 1);
    const int64_t wave = (int64_t)blockIdx.x * kQuantWaves + threadIdx.x / kWave;
    const bool bf16 = a.x_dtype == DA_BF16;
    int64_t m = wave * (kWave / L) + lane / L, end = min(m + 1, a.M), image = 0;
    NormCoef f[NORM ? HOLD : 1];
    if constexpr (NORM) {
        const int64_t per = (g.S + rows_per_wave - 1) / rows_per_wave;   // waves of an image
        image = wave / per;
        if (image >= g.N) return;
        m = image * g.S + (wave - image * per) * rows_per_wave;
        end = min(m + rows_per_wave, (image + 1) * g.S);
#pragma unroll
        for (int i = 0; i < HOLD; ++i) f[i].load(a, g, image, (i * L + lane) * 8);
    }
    for (; m < end; ++m) {
        Eight<XB> hold[HOLD];
        float v[8];
        uint32_t big = 0;
#pragma unroll
        for (int i = 0; i < HOLD; ++i) {
            const int c = (i * L + lane % L) * 8;
            if (c < a.K) hold[i].load(a.x, m, c, a.K);
            else hold[i].zero();
        }
        // numbers from column c on, normalised where a norm stands in front
        const auto of = [&](const Eight<XB>& q, const NormCoef& coef) {
            q.unpack(v, bf16);
            if constexpr (NORM) coef.apply(v, g.act);
        };
        const auto again = [&](int c) {
            Eight<XB> q;
            q.load(a.x, m, c, a.K);
            NormCoef coef;
            if constexpr (NORM) coef.load(a, g, image, c);
            of(q, coef);
        };
#pragma unroll
        for (int i = 0; i < HOLD; ++i) {
            of(hold[i], f[NORM ? i : 0]);
            big = max(big, magnitude(v));
        }
        for (int c = (HOLD * L + lane % L) * 8; c < a.K; c += L * 8) {
            again(c);
            big = max(big, magnitude(v));
        }
#pragma unroll
        for (int s = L / 2; s; s >>= 1) big = max(big, (uint32_t)__shfl_xor((int)big, s));
        const RowScale s = row_scale(big);
        const auto put = [&](int c) {
            const u32x2 q = {pack_codes(v, s), pack_codes(v + 4, s)};
            int8_t* p = a.a + m * a.K + c;
            if (c + 8 <= a.K) {
                __builtin_memcpy(p, &q, 8);
            } else {
#pragma unroll
                for (int e = 0; e < 7; ++e)
                    if (c + e < a.K) p[e] = (int8_t)(q[e / 4] >> (8 * (e & 3)));
            }
        };
#pragma unroll
        for (int i = 0; i < HOLD; ++i) {
            const int c = (i * L + lane % L) * 8;
            if (c < a.K) {
                of(hold[i], f[NORM ? i : 0]);
                put(c);
            }
        }
        for (int c = (HOLD * L + lane % L) * 8; c < a.K; c += L * 8) {
            again(c);
            put(c);
        }
        if (lane % L == 0) a.a_scale[m] = s.scale;
    }
}

// How many of a tile's `most` rows are left.  In whole numbers, so that the ranges of the buffer
// resources that are made of it are scalars: HIP's min of 64-bit numbers goes by binary64, in
// vector registers, and every access through such a resource then runs in a loop over the lanes'
// values of it.
__device__ __forceinline__ int rows_left(int64_t left, int most) {
    return left < most ? (int)left : most;
}

// ---- pieces of the operands --------------------------------------------------------------

// The 16 codes of row `row` of [.., K] from column k on (k < K), zeros past K.  Any alignment.
// A row's broken last piece is the end of its last 16 codes, shifted down.
__device__ __forceinline__ i32x4 bytes_of(const int8_t* base, int64_t row, int k, int K) {
    const int8_t* p = base + row * K;
    uint64_t lo = 0, hi = 0;
    if (K >= 16) {
        const int at = min(k, K - 16), s = (k - at) * 8;   // 0 .. 120 bits
        __builtin_memcpy(&lo, p + at, 8);
        __builtin_memcpy(&hi, p + at + 8, 8);
        if (s >= 64) {
            lo = hi >> (s - 64);
            hi = 0;
        } else if (s) {
            lo = lo >> s | hi << (64 - s);
            hi >>= s;
        }
    } else {
        for (int i = 0; k + i < K; ++i) {
            const uint64_t b = (uint64_t)(uint8_t)p[k + i] << (8 * (i & 7));
            lo |= i < 8 ? b : 0;
            hi |= i < 8 ? 0 : b;
        }
    }
    return i32x4{(int)lo, (int)(lo >> 32), (int)hi, (int)(hi >> 32)};
}

// A piece of a row as it lies in memory: eight numbers, or sixteen codes.
struct Sixteen {
    i32x4 q;
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t voff) {
        q = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(r, voff, 0, 0));
    }
    __device__ __forceinline__ void load(const void* base, int64_t row, int c, int K) {
        q = bytes_of(static_cast<const int8_t*>(base), row, c, K);
    }
    __device__ __forceinline__ void zero() { q = i32x4{0, 0, 0, 0}; }
    __device__ __forceinline__ void merge(const Sixteen& o, bool take) {
#pragma unroll
        for (int e = 0; e < 4; ++e) q[e] = take ? o.q[e] : q[e];
    }
};
template <int XB>
struct RowPiece {
    typedef Eight<XB> type;
};
template <>
struct RowPiece<0> {
    typedef Sixteen type;
};
template <int XB>
__device__ __forceinline__ void numbers(const Eight<XB> (&q)[2], float (&v)[16], bool bf16) {
    q[0].unpack(reinterpret_cast<float(&)[8]>(v[0]), bf16);
    q[1].unpack(reinterpret_cast<float(&)[8]>(v[8]), bf16);
}

// ---- results -----------------------------------------------------------------------------

// Scales and bias of the four output channels from n on (0 past N).
struct ColumnScale {
    float s[4], b[4];
};
__device__ __forceinline__ ColumnScale column_scale(const I8Args& a, int n) {
    ColumnScale c;
    if (n + 4 <= a.N) {
        __builtin_memcpy(c.s, a.w_scale + n, 16);
        if (a.bias) {
            __builtin_memcpy(c.b, a.bias + n, 16);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) c.b[i] = 0.0f;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            c.s[i] = n + i < a.N ? a.w_scale[n + i] : 0.0f;
            c.b[i] = n + i < a.N && a.bias ? a.bias[n + i] : 0.0f;
        }
    }
    return c;
}

template <typename D>
__device__ __forceinline__ void store_four(D* p, const float (&y)[4], int count) {
    typedef D vec __attribute__((ext_vector_type(4)));
    const vec t = {(D)y[0], (D)y[1], (D)y[2], (D)y[3]};
    if (count >= 4) {
        __builtin_memcpy(p, &t, sizeof t);
    } else {
#pragma unroll
        for (int i = 0; i < 3; ++i)
            if (i < count) p[i] = t[i];
    }
}

// Four elements through a buffer resource: dropped past its range.
__device__ __forceinline__ void store_four(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff,
                                           const float (&y)[4], int dtype) {
    if (dtype == DA_F32) {
        typedef float vec __attribute__((ext_vector_type(4)));
        const vec t = {y[0], y[1], y[2], y[3]};
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, t), r, voff, soff, 0);
    } else if (dtype == DA_BF16) {
        typedef __bf16 vec __attribute__((ext_vector_type(4)));
        const vec t = {(__bf16)y[0], (__bf16)y[1], (__bf16)y[2], (__bf16)y[3]};
        __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, t), r, voff, soff, 0);
    } else {
        typedef _Float16 vec __attribute__((ext_vector_type(4)));
        const vec t = {(_Float16)y[0], (_Float16)y[1], (_Float16)y[2], (_Float16)y[3]};
        __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, t), r, voff, soff, 0);
    }
}

// The sums as numbers: conversion, row scale, and column scale with the bias round once each.
__device__ __forceinline__ void scaled(const i32x4& acc, float row, const ColumnScale& c,
                                       float (&y)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = fmaf((float)acc[i] * row, c.s[i], c.b[i]);
}

// out[m, n .. n + 3] from the sums, as far as n stays below N.
__device__ __forceinline__ void finish(const I8Args& a, int64_t m, int n, const i32x4& acc,
                                       float row, const ColumnScale& c, int act) {
    float y[4];
    scaled(acc, row, c, y);
    activate(y, act);
    const int64_t at = m * a.N + n;
    if (a.out_dtype == DA_BF16)
        store_four(static_cast<__bf16*>(a.out) + at, y, a.N - n);
    else if (a.out_dtype == DA_F16)
        store_four(static_cast<_Float16*>(a.out) + at, y, a.N - n);
    else
        store_four(static_cast<float*>(a.out) + at, y, a.N - n);
}

// ---- rows kernel -------------------------------------------------------------------------
//
// At most 256 columns.  A workgroup holds a slice of the weights in LDS; each of its waves
// takes 16 rows at a time, by itself: a lane reads 16 consecutive numbers of row l % 16 for
// every 64 columns, which is where the matrix instruction wants their codes, so a row's
// largest magnitude is two lane exchanges away, the codes never leave the registers, no
// wave waits for another, and the next rows are on their way while these are multiplied.
// x is read once per slice (the second time from cache), out is written once, and no codes
// go through memory.
//
// Memory bounds it where rows are many: 200704 x 128 x 108 from bfloat16 into binary32 (138
// MB) takes 30 us, 4.6 TB/s (a copy of as much 28 us).  900 x 256 x 2496 codes take 9 us:
// a launch, the fill of LDS and the first rows are waited for before the first product.  Behind
// a norm 50176 x 256 x 216 takes 25 us and the statistics 9 us; by their instructions 12.8
// million activations and codes are some 11 us, and with one unit of rows to a wave nothing
// overlaps its loads and stores but the other workgroup of the compute unit.  That takes 128
// registers: with 256, and half the waves, the call is 37.1 us in place of 31.9.

constexpr int kRowsThreads = 512;
constexpr int kRowsWaves = kRowsThreads / kWave;
constexpr size_t kRowsLdsAll = 80 * 1024;   // two workgroups to a compute unit
constexpr size_t kRowsLds = 60 * 1024;      // of weights

// Whole pieces of x go through a buffer resource: what lies past the wave's rows reads as
// zero, without a comparison.
constexpr uint32_t kOutside = 0x80000000u;   // past every range (each is below 2^31 bytes)

// Bytes between rows of codes in LDS: an odd number of 16-byte units, so that the 16 rows of
// an operand start in different banks.
__host__ __device__ constexpr int rows_stride(int kt) { return kt * 64 + 16; }

template <int XB, bool NORM, int KT>
__global__ __launch_bounds__(kRowsThreads, KT == 4 && XB == 4 ? 2 : 4) void i8_rows_kernel(I8Args a,
                                                                                       GnArgs g) {
    constexpr int kStride = rows_stride(KT);
    constexpr int kPieces = XB == 0 ? 1 : 2;   // per 16 numbers of a lane
    constexpr int xbytes = XB ? XB : 1, per = XB ? 8 : 16;
    extern __shared__ __align__(16) unsigned char lds[];
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int col = lane % 16, part = lane / 16;
    const int tiles = (a.N + 15) / 16;
    const int slice = blockIdx.x % a.slices, block = blockIdx.x / a.slices;
    const int t0 = slice * a.tiles_per_slice, t1 = min(tiles, t0 + a.tiles_per_slice);
    const int wrows = (t1 - t0) * 16;
    unsigned char* ws = lds;
    float* scale = reinterpret_cast<float*>(lds + a.tiles_per_slice * 16 * kStride);
    float* bias = scale + a.tiles_per_slice * 16;
    float* mu = bias + a.tiles_per_slice * 16;   // [64 * KT] each
    float* sc = mu + 64 * KT;
    float* bi = sc + 64 * KT;
    unsigned char* stage = reinterpret_cast<unsigned char*>(NORM ? bi + 64 * KT : mu) +
                           wave * 16 * a.N * (a.out_dtype == DA_F32 ? 4 : 2);

    // rows: units of 16, within one image behind a norm
    int64_t base = 0, rows_end = a.M, u = (int64_t)block * kRowsWaves + wave;
    int64_t step = (int64_t)a.blocks_per_image * kRowsWaves;
    if constexpr (NORM) {
        const int64_t image = block / a.blocks_per_image;
        base = image * g.S;
        rows_end = base + g.S;
        u -= image * step;
        for (int c = threadIdx.x; c < 64 * KT; c += kRowsThreads) {
            float m = 0.0f, s = 0.0f, b = 0.0f;   // a column past K holds 0
            if (c < a.K) {
                const int64_t j = image * g.G + c / g.cpg;
                m = g.mean[j];
                s = g.rstd[j] * (a.norm_weight ? a.norm_weight[c] : 1.0f);
                if (a.norm_bias) b = a.norm_bias[c];
            }
            mu[c] = m;
            sc[c] = s;
            bi[c] = b;
        }
    }
    const int64_t units = (rows_end - base + 15) / 16;

    // A unit's numbers: kc * 64 + part * 16 .. + 15 of row `col`.  The row's broken last piece,
    // where it has one, is piece odd_piece of run odd_run in the lanes of odd_part.
    typename RowPiece<XB>::type q[KT][kPieces];
    const int odd_c = a.K / per * per, odd_run = a.K % per ? odd_c / 64 : -1;
    const int odd_part = odd_c % 64 / 16, odd_piece = odd_c % 16 / per;
    const auto fetch = [&](int64_t unit) {
        const int64_t m0 = base + unit * 16;
        const int rows = rows_left(rows_end - m0, 16);
        const void* x = XB ? a.x : a.a;
        const auto r = make_rsrc(static_cast<const char*>(x) + m0 * a.K * xbytes,
                                 (uint32_t)(rows * a.K * xbytes));
#pragma unroll
        for (int kc = 0; kc < KT; ++kc)
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                const int c = kc * 64 + part * 16 + i * per;
                q[kc][i].load(r, c + per <= a.K ? (col * a.K + c) * xbytes : kOutside);
            }
        if (odd_run >= 0) {
            typename RowPiece<XB>::type odd;
            odd.zero();
            if (part == odd_part && col < rows) odd.load(x, m0 + col, odd_c, a.K);
#pragma unroll
            for (int kc = 0; kc < KT; ++kc)
#pragma unroll
                for (int i = 0; i < kPieces; ++i)
                    if (kc == odd_run && i == odd_piece) q[kc][i].merge(odd, part == odd_part);
        }
    };
    if (u < units) fetch(u);

    const auto wr = make_rsrc(a.w + (int64_t)t0 * 16 * a.K, (uint32_t)min(wrows, a.N - t0 * 16) * a.K);
    for (int e = threadIdx.x; e < wrows * KT * 4; e += kRowsThreads) {
        const int r = e / (KT * 4), c = e % (KT * 4) * 16, n = t0 * 16 + r;
        Sixteen w;
        w.load(wr, c + 16 <= a.K ? r * a.K + c : kOutside);
        if (a.K % 16 && n < a.N && c < a.K && c + 16 > a.K) w.load(a.w, n, c, a.K);
        *reinterpret_cast<i32x4*>(ws + r * kStride + c) = w.q;
    }
    for (int e = threadIdx.x; e < wrows; e += kRowsThreads) {
        const int n = t0 * 16 + e;
        scale[e] = n < a.N ? a.w_scale[n] : 0.0f;
        bias[e] = n < a.N && a.bias ? a.bias[n] : 0.0f;
    }
    __syncthreads();

    const bool bf16 = a.x_dtype == DA_BF16;
    const int ob = a.out_dtype == DA_F32 ? 4 : 2;
    const uint32_t out_at = (uint32_t)((col * a.N + part * 4) * ob);
    for (; u < units; u += step) {
        i32x4 x[KT];
        float rs;
        const int64_t m0 = base + u * 16;
        const int rows = rows_left(rows_end - m0, 16);
        if constexpr (XB == 0) {
            rs = col < rows ? a.a_scale[m0 + col] : 0.0f;
#pragma unroll
            for (int kc = 0; kc < KT; ++kc) x[kc] = q[kc][0].q;
        } else {
            // normalised numbers are kept between the two steps; the barriers to the scheduler
            // keep the numbers from being worked on all at once (four at a time behind a norm:
            // 8 registers spilled)
            float z[KT][16];
            uint32_t big = 0;
#pragma unroll
            for (int kc = 0; kc < KT; ++kc) {
                if constexpr (NORM) {
                    numbers(q[kc], z[kc], bf16);
                    const int c = kc * 64 + part * 16;
#pragma unroll
                    for (int e = 0; e < 16; e += 4) {
                        const f32x4 m4 = *reinterpret_cast<const f32x4*>(mu + c + e);
                        const f32x4 s4 = *reinterpret_cast<const f32x4*>(sc + c + e);
                        const f32x4 b4 = *reinterpret_cast<const f32x4*>(bi + c + e);
                        float y[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            y[i] = fmaf(z[kc][e + i] - m4[i], s4[i], b4[i]);
                        activate(y, g.act);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            z[kc][e + i] = y[i];
                            big = max(big, __float_as_uint(y[i]) & 0x7fffffffu);
                        }
                        __builtin_amdgcn_sched_barrier(0);
                    }
                } else {
                    big = max(big, max(q[kc][0].magnitude(), q[kc][1].magnitude()));
                }
            }
            if constexpr (!NORM) big = Eight<XB>::widen(big, bf16);
            big = max(big, (uint32_t)__shfl_xor((int)big, 16));
            big = max(big, (uint32_t)__shfl_xor((int)big, 32));
            const RowScale s = row_scale(big);
            rs = s.scale;
#pragma unroll
            for (int kc = 0; kc < KT; ++kc) {
                if constexpr (!NORM) numbers(q[kc], z[kc], bf16);
                const float* v = z[kc];
                x[kc] = i32x4{(int)pack_codes(v, s), (int)pack_codes(v + 4, s),
                              (int)pack_codes(v + 8, s), (int)pack_codes(v + 12, s)};
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        if (u + step < units) fetch(u + step);

        const auto outr = make_rsrc(static_cast<char*>(a.out) + m0 * a.N * ob,
                                    (uint32_t)(rows * a.N * ob));
        const unsigned char* wp = ws + col * kStride + part * 16;
        const float* sp = scale + part * 4;
        for (int t = t0; t < t1; ++t, wp += 16 * kStride, sp += 16) {
            i32x4 acc = {0, 0, 0, 0};
#pragma unroll
            for (int kc = 0; kc < KT; ++kc)
                acc = mfma(*reinterpret_cast<const i32x4*>(wp + kc * 64), x[kc], acc);
            ColumnScale cs;
            __builtin_memcpy(cs.s, sp, 16);
            __builtin_memcpy(cs.b, sp + a.tiles_per_slice * 16, 16);
            if (a.staged) {
                float y[4];
                scaled(acc, rs, cs, y);
                activate(y, a.act);
                if (t * 16 + part * 4 < a.N) {
                    const int at = col * a.N + t * 16 + part * 4;
                    if (ob == 4) *reinterpret_cast<f32x4*>(stage + at * 4) = f32x4{y[0], y[1], y[2], y[3]};
                    else store_vec(static_cast<void*>(stage), at, y, a.out_dtype);
                }
            } else if (t * 16 + 16 <= a.N) {
                float y[4];
                scaled(acc, rs, cs, y);
                activate(y, a.act);
                store_four(outr, out_at, (uint32_t)(t * 16 * ob), y, a.out_dtype);
            } else {   // the last tile, not all of it in the row
                const int n = t * 16 + part * 4;
                if (n < a.N && col < rows) finish(a, m0 + col, n, acc, rs, cs, a.act);
            }
        }
        if (a.staged) {
            // the unit's rows are one run of memory: lines are written whole.  The wave's own LDS
            // accesses complete in order; the fences keep the compiler to it.
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
            for (int p = lane * 16; p < rows * a.N * ob; p += kWave * 16)
                __builtin_amdgcn_raw_buffer_store_b128(*reinterpret_cast<const u32x4*>(stage + p),
                                                       outr, (uint32_t)p, 0, 0);
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
        }
    }
}

// ---- streaming kernel --------------------------------------------------------------------
//
// Few rows, 16 * MT at a time: a wave takes 16 output channels and every KW-th run of 64 columns,
// the weights going from memory into operand registers, several runs in flight; the KW
// waves' sums meet in LDS.  The rows' codes come from memory (XB 0), or the workgroup
// quantises up to 16 rows of x into LDS first.  One row of 4096 by 4096 x 4096 codes takes 7.6
// us, 2.2 TB/s of weights (floor 4 us): the launch, the row's scale and the sums' meeting are
// waited for one after the other; the first weights are on their way before the row is read.

constexpr int kSkinnyThreads = 512;
constexpr int kSkinnyWaves = kSkinnyThreads / kWave;
constexpr size_t kSkinnyLds = 48 * 1024;       // of codes

template <int XB, int MT>
__global__ __launch_bounds__(kSkinnyThreads) void i8_skinny_kernel(I8Args a, int kw_count) {
    extern __shared__ __align__(16) unsigned char codes[];   // [M][stride], XB != 0
    __shared__ __align__(16) i32x4 meet[kSkinnyWaves][MT][kWave];
    __shared__ uint32_t bigs[16][kSkinnyWaves];
    __shared__ float scales[16];
    constexpr int kRuns = MT == 1 ? 8 : 4;   // of a wave in flight, in pairs of 128 columns
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int col = lane % 16, part = lane / 16;
    const int kw = wave % kw_count;
    const int tiles = (a.N + 15) / 16, runs = (a.K + 63) / 64;
    const int blocks = (tiles + kSkinnyWaves / kw_count - 1) / (kSkinnyWaves / kw_count);
    const int64_t m0 = (int64_t)(blockIdx.x / blocks) * (16 * MT);
    const int rows = rows_left(a.M - m0, 16 * MT);
    const int tile = blockIdx.x % blocks * (kSkinnyWaves / kw_count) + wave / kw_count;
    const int stride = runs * 64 + 16, step = kRuns * kw_count;
    const bool live = tile < tiles;
    const int n = tile * 16 + col, wrows = live ? min(16, a.N - tile * 16) : 0;

    struct Runs {
        Sixteen w[kRuns], x[XB == 0 ? MT : 1][XB == 0 ? kRuns : 1];
    } next;
    const auto column = [&](int c, int i) {
        return (c + i / 2 * 2 * kw_count + 2 * kw + i % 2) * 64 + part * 16;
    };
    const auto wr = make_rsrc(a.w + (live ? (int64_t)tile * 16 * a.K : 0), (uint32_t)wrows * a.K);
    const auto xr = make_rsrc(a.a + (XB == 0 ? m0 * a.K : 0), XB == 0 ? (uint32_t)rows * a.K : 0u);
    const auto fetch = [&](int c) {
#pragma unroll
        for (int i = 0; i < kRuns; ++i) {
            const int k = column(c, i);
            next.w[i].load(wr, k + 16 <= a.K ? col * a.K + k : kOutside);
            if constexpr (XB == 0) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
                    next.x[mt][i].load(xr, k + 16 <= a.K ? (mt * 16 + col) * a.K + k : kOutside);
            }
        }
        if (a.K % 16 && (c + step) * 64 > a.K) {   // the rows' broken last pieces are among these
#pragma unroll
            for (int i = 0; i < kRuns; ++i) {
                const int k = column(c, i);
                if (k < a.K && k + 16 > a.K) {
                    if (col < wrows) next.w[i].load(a.w, n, k, a.K);
                    if constexpr (XB == 0) {
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt)
                            if (mt * 16 + col < rows)
                                next.x[mt][i].load(a.a, m0 + mt * 16 + col, k, a.K);
                    }
                }
            }
        }
    };
    fetch(0);   // on its way while the rows are quantised

    if constexpr (XB != 0) {
        // 8 / 2^j waves to a row; a lane keeps the first two pieces of it
        const bool bf16 = a.x_dtype == DA_BF16;
        int share = 1;
        while (share < kSkinnyWaves && kSkinnyWaves / (2 * share) >= rows) share *= 2;
        const int part_of = wave % share, skip = share * kWave * 8;
        constexpr int kHold = 2;
        for (int first = 0; first < rows; first += kSkinnyWaves / share) {
            const int m = first + wave / share, c0 = (part_of * kWave + lane) * 8;
            Eight<XB> hold[kHold];
            float v[8];
            uint32_t big = 0;
#pragma unroll
            for (int i = 0; i < kHold; ++i) {
                if (m < rows && c0 + i * skip < a.K) hold[i].load(a.x, m, c0 + i * skip, a.K);
                else hold[i].zero();
            }
#pragma unroll
            for (int i = 0; i < kHold; ++i) big = max(big, hold[i].magnitude());
            if (m < rows)
                for (int c = c0 + kHold * skip; c < a.K; c += skip) {
                    Eight<XB> q;
                    q.load(a.x, m, c, a.K);
                    big = max(big, q.magnitude());
                }
            big = Eight<XB>::widen(big, bf16);
#pragma unroll
            for (int s = kWave / 2; s; s >>= 1) big = max(big, (uint32_t)__shfl_xor((int)big, s));
            if (share > 1) {
                if (lane == 0) bigs[wave / share][part_of] = big;
                __syncthreads();
                for (int i = 0; i < share; ++i) big = max(big, bigs[wave / share][i]);
            }
            if (m < rows) {
                const RowScale s = row_scale(big);
                const auto put = [&](const Eight<XB>& q, int c) {
                    q.unpack(v, bf16);
                    *reinterpret_cast<u32x2*>(codes + m * stride + c) =
                        u32x2{pack_codes(v, s), pack_codes(v + 4, s)};
                };
#pragma unroll
                for (int i = 0; i < kHold; ++i)
                    if (c0 + i * skip < runs * 64) put(hold[i], c0 + i * skip);
                for (int c = c0 + kHold * skip; c < runs * 64; c += skip) {
                    Eight<XB> q;
                    if (c < a.K) q.load(a.x, m, c, a.K);
                    else q.zero();
                    put(q, c);
                }
                if (part_of == 0 && lane == 0) scales[m] = s.scale;
            }
            if (share > 1) __syncthreads();   // bigs is written again for the next rows
        }
        __syncthreads();
    }

    i32x4 acc[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) acc[mt] = i32x4{0, 0, 0, 0};
    for (int c = 0; c < runs; c += step) {
        const Runs now = next;
        if (c + step < runs) fetch(c + step);
#pragma unroll
        for (int i = 0; i < kRuns; ++i)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                i32x4 x = {0, 0, 0, 0};
                if constexpr (XB != 0) {
                    const int k = column(c, i);
                    if (col < rows && k < runs * 64)
                        x = *reinterpret_cast<const i32x4*>(codes + col * stride + k);
                } else {
                    x = now.x[mt][i].q;
                }
                acc[mt] = mfma(now.w[i].q, x, acc[mt]);
            }
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) meet[wave][mt][lane] = acc[mt];
    __syncthreads();
    // the waves of a tile deal its row tiles
    const int nn = tile * 16 + part * 4;
    if (!live || nn >= a.N) return;
    const ColumnScale cs = column_scale(a, nn);
    for (int mt = kw; mt < MT; mt += kw_count) {
        i32x4 t = meet[wave - kw][mt][lane];
        for (int i = 1; i < kw_count; ++i) t += meet[wave - kw + i][mt][lane];
        const int m = mt * 16 + col;
        if (m < rows)
            finish(a, m0 + m, nn, t, XB != 0 ? scales[m] : a.a_scale[m0 + m], cs, a.act);
    }
}

// ---- tiled product -----------------------------------------------------------------------
//
// 64 rows by 64 output channels to a workgroup of four waves, 128 columns at a time through
// LDS, the next 128 on their way to registers meanwhile.  For products too small to fill the
// chip with larger tiles, so bound by a tile's walk along its columns (0.6 us per 128): 1237 x
// 1000 x 777 takes 11.2 us, 12544 x 512 x 432 with its quantisation 23 us.  A 16-byte piece p of
// an LDS row r sits at place p ^ (r / 2 % 8): the 16 rows an operand is read from then fall into
// different banks.

constexpr int kTileK = 128, kTile = 64, kTileThreads = 256;

// Workgroups go round the 8 XCDs: each gets a run of consecutive tiles, and runs go down 8 row
// tiles before the next column tile, so that an XCD's L2 sees few operands.
__device__ __forceinline__ void tile_of(int id, int mt, int nt, int& m, int& n) {
    const int total = mt * nt, x = id % 8, i = id / 8;
    id = x * (total / 8) + min(x, total % 8) + i;
    const int band = id / (8 * nt), in_band = id - band * 8 * nt;
    const int rows = min(8, mt - band * 8);
    m = band * 8 + in_band % rows;
    n = in_band / rows;
}

__global__ __launch_bounds__(kTileThreads) void i8_tile_kernel(I8Args a) {
    constexpr int kPieces = kTileK / 16, kLoads = kTile * kPieces / kTileThreads, W = 32;
    __shared__ __align__(16) i32x4 xs[2][kTile * kPieces], ws[2][kTile * kPieces];
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int col = lane % 16, part = lane / 16;
    const int wm = wave % 2 * W, wn = wave / 2 * W;
    const int mt = (int)((a.M + kTile - 1) / kTile), nt = (a.N + kTile - 1) / kTile;
    int tile_m, tile_n;
    tile_of(blockIdx.x, mt, nt, tile_m, tile_n);
    const int64_t m0 = (int64_t)tile_m * kTile;
    const int n0 = tile_n * kTile;
    const int rows = rows_left(a.M - m0, kTile), cols = min(a.N - n0, kTile);

    // A thread's pieces: rows `row` and row + 32 of either operand, at one place of theirs.
    // Whole pieces come through buffer resources whose ranges end with the block's last row,
    // so that no row is looked at; a row's broken last piece is put together from bytes.
    struct Stage {
        i32x4 x[kLoads], w[kLoads];
    } next;
    const int piece = threadIdx.x % kPieces * 16, row = threadIdx.x / kPieces;
    constexpr int kRowStep = kTileThreads / kPieces;
    const auto xr = make_rsrc(a.a + m0 * a.K, (uint32_t)rows * a.K);
    const auto wr = make_rsrc(a.w + (int64_t)n0 * a.K, (uint32_t)cols * a.K);
    const auto load = [](__amdgpu_buffer_rsrc_t r, uint32_t voff, int k0) {
        return __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(r, voff, k0, 0));
    };
    const auto fetch = [&](int k0, Stage& s) {
        if (k0 >= a.K) return;
        const int k = k0 + piece;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const uint32_t at = k + 16 <= a.K ? (row + i * kRowStep) * a.K + piece : kOutside;
            s.x[i] = load(xr, at, k0);
            s.w[i] = load(wr, at, k0);
        }
        if (a.K % 16 && k0 + kTileK > a.K && k < a.K && k + 16 > a.K) {
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const int r = row + i * kRowStep;
                if (r < rows) s.x[i] = bytes_of(a.a, m0 + r, k, a.K);
                if (r < cols) s.w[i] = bytes_of(a.w, n0 + r, k, a.K);
            }
        }
    };
    const auto place = [](int r, int p) { return r * kPieces + (p ^ ((r >> 1) & 7)); };
    const auto put = [&](int b, const Stage& s) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            xs[b][place(row + i * kRowStep, piece / 16)] = s.x[i];
            ws[b][place(row + i * kRowStep, piece / 16)] = s.w[i];
        }
    };

    i32x4 acc[W / 16][W / 16];
#pragma unroll
    for (int i = 0; i < W / 16; ++i)
#pragma unroll
        for (int j = 0; j < W / 16; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
    const auto multiply = [&](int b) {
#pragma unroll
        for (int kc = 0; kc < kTileK / 64; ++kc) {
            i32x4 xf[W / 16], wf[W / 16];
#pragma unroll
            for (int j = 0; j < W / 16; ++j) {
                wf[j] = ws[b][place(wn + j * 16 + col, kc * 4 + part)];
                xf[j] = xs[b][place(wm + j * 16 + col, kc * 4 + part)];
            }
#pragma unroll
            for (int i = 0; i < W / 16; ++i)
#pragma unroll
                for (int j = 0; j < W / 16; ++j) acc[i][j] = mfma(wf[j], xf[i], acc[i][j]);
        }
    };
    fetch(0, next);
    float rs[W / 16];
    ColumnScale cs[W / 16];
#pragma unroll
    for (int i = 0; i < W / 16; ++i) {
        const int m = wm + i * 16 + col;
        rs[i] = m < rows ? a.a_scale[m0 + m] : 0.0f;
        cs[i] = column_scale(a, min(n0 + wn + i * 16 + part * 4, a.N));
    }
    put(0, next);
    __syncthreads();
    int b = 0;
    for (int k0 = 0; k0 < a.K; k0 += kTileK, b ^= 1) {
        fetch(k0 + kTileK, next);
        multiply(b);
        if (k0 + kTileK < a.K) put(b ^ 1, next);
        __syncthreads();
    }
#pragma unroll
    for (int j = 0; j < W / 16; ++j) {
        const int n = n0 + wn + j * 16 + part * 4;
        if (n >= a.N) continue;
#pragma unroll
        for (int i = 0; i < W / 16; ++i) {
            const int m = wm + i * 16 + col;
            if (m < rows) finish(a, m0 + m, n, acc[i][j], rs[i], cs[j], a.act);
        }
    }
}

// ---- large products ----------------------------------------------------------------------
//
// 256 rows by 256 output channels to a workgroup of eight waves, 128 x 64 to a wave, columns
// in whole runs of 128.  8192 x 4096 x 4096 takes 109 us into the same result each time, 129 us
// with operands and results in rotation: 2.1 to 2.5 POP/s, bound by the matrix cores (the
// library's 8-bit product without scales reaches 2.2 in rotation).  Tiles of 64 took 200 us; a
// grid of as many workgroups as are resident, each with several tiles, spilled and was slower.
// The next 128 columns go from memory straight into the other half of LDS while these are
// multiplied, and a run's operands are read while the run before it is in the matrix cores.
// An instruction that fills LDS puts lane l's 16 bytes at place l of a run of 1 KB, so the
// swizzle of the tiled kernel is in the addresses the lanes fetch from.

constexpr int kBigTile = 256, kBigThreads = 512;
constexpr int kSchedMatrix = 0x8, kSchedLdsRead = 0x100;   // instruction classes of a schedule

__global__ __launch_bounds__(kBigThreads, 2) void i8_big_kernel(I8Args a) {
    constexpr int kPieces = kTileK / 16, WM = 128, WN = 64;
    // four arrays, not one: the compiler then sees that what is filled is not what is read
    __shared__ __align__(16) i32x4 x0[kBigTile * kPieces], x1[kBigTile * kPieces];
    __shared__ __align__(16) i32x4 w0[kBigTile * kPieces], w1[kBigTile * kPieces];
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int col = lane % 16, part = lane / 16;
    const int wm = wave % 2 * WM, wn = wave / 2 * WN;
    const int mt = (int)((a.M + kBigTile - 1) / kBigTile), nt = (a.N + kBigTile - 1) / kBigTile;
    int tile_m, tile_n;
    tile_of(blockIdx.x, mt, nt, tile_m, tile_n);
    const int64_t m0 = (int64_t)tile_m * kBigTile;
    const int n0 = tile_n * kBigTile;
    const int rows = rows_left(a.M - m0, kBigTile);

    const auto xr = make_rsrc(a.a + m0 * a.K, (uint32_t)rows * a.K);
    const auto wr = make_rsrc(a.w + (int64_t)n0 * a.K, (uint32_t)min(a.N - n0, kBigTile) * a.K);
    // rows i * 64 + wave * 8 + lane / 8
    const int row = wave * 8 + lane / kPieces;
    const uint32_t at = row * a.K + ((lane % kPieces) ^ ((row >> 1) & 7)) * 16;
    const auto fetch = [&](int k0, i32x4* xs, i32x4* ws) {
#pragma unroll
        for (int i = 0; i < kBigTile / 64; ++i) {
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                xr, (__attribute__((address_space(3))) void*)(xs + (i * 64 + wave * 8) * kPieces), 16,
                at + i * 64 * a.K, k0, 0, 0);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                wr, (__attribute__((address_space(3))) void*)(ws + (i * 64 + wave * 8) * kPieces), 16,
                at + i * 64 * a.K, k0, 0, 0);
        }
    };
    const auto place = [](int r, int p) { return r * kPieces + (p ^ ((r >> 1) & 7)); };

    i32x4 acc[WM / 16][WN / 16];
#pragma unroll
    for (int i = 0; i < WM / 16; ++i)
#pragma unroll
        for (int j = 0; j < WN / 16; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
    const auto step = [&](const i32x4* xs, const i32x4* ws) {
#pragma unroll
        for (int kc = 0; kc < kTileK / 64; ++kc) {
            i32x4 xf[WM / 16], wf[WN / 16];
#pragma unroll
            for (int j = 0; j < WN / 16; ++j) wf[j] = ws[place(wn + j * 16 + col, kc * 4 + part)];
#pragma unroll
            for (int i = 0; i < WM / 16; ++i) xf[i] = xs[place(wm + i * 16 + col, kc * 4 + part)];
#pragma unroll
            for (int i = 0; i < WM / 16; ++i)
#pragma unroll
                for (int j = 0; j < WN / 16; ++j) acc[i][j] = mfma(wf[j], xf[i], acc[i][j]);
        }
        // the order of the step: the first run's operands, then a read to every two products
        // while there are any, so that the second run's are there when the first is done
        __builtin_amdgcn_sched_group_barrier(kSchedLdsRead, 12, 0);
#pragma unroll
        for (int i = 0; i < 12; ++i) {
            __builtin_amdgcn_sched_group_barrier(kSchedMatrix, 2, 0);
            __builtin_amdgcn_sched_group_barrier(kSchedLdsRead, 1, 0);
        }
        __builtin_amdgcn_sched_group_barrier(kSchedMatrix, 40, 0);
    };
    fetch(0, x0, w0);
    __syncthreads();
    for (int k0 = 0;;) {
        if (k0 + kTileK < a.K) fetch(k0 + kTileK, x1, w1);
        step(x0, w0);
        __syncthreads();
        k0 += kTileK;
        if (k0 >= a.K) break;
        if (k0 + kTileK < a.K) fetch(k0 + kTileK, x0, w0);
        step(x1, w1);
        __syncthreads();
        k0 += kTileK;
        if (k0 >= a.K) break;
    }

    // all scales at once, then stores only
    const int ob = a.out_dtype == DA_F32 ? 4 : 2;
    const auto outr = make_rsrc(static_cast<char*>(a.out) + m0 * a.N * ob, (uint32_t)rows * a.N * ob);
    const auto rr = make_rsrc(a.a_scale + m0, rows * 4u);
    const auto sr = make_rsrc(a.w_scale, a.N * 4u), br = make_rsrc(a.bias, a.bias ? a.N * 4u : 0u);
    float rs[WM / 16];
    ColumnScale cs[WN / 16];
#pragma unroll
    for (int i = 0; i < WM / 16; ++i)
        rs[i] = __uint_as_float(
            __builtin_amdgcn_raw_buffer_load_b32(rr, (wm + i * 16 + col) * 4, 0, 0));
#pragma unroll
    for (int j = 0; j < WN / 16; ++j) {
        Sixteen s, b;
        s.load(sr, (n0 + wn + j * 16 + part * 4) * 4u);
        b.load(br, (n0 + wn + j * 16 + part * 4) * 4u);
        __builtin_memcpy(cs[j].s, &s.q, 16);
        __builtin_memcpy(cs[j].b, &b.q, 16);
    }
    // the activation is chosen outside the loops: 32 places with every activation in them do not
    // fit the instruction cache
    with_activation(a.act, [&](auto act) {
#pragma unroll
        for (int i = 0; i < WM / 16; ++i) {
            const int m = wm + i * 16 + col;
            const uint32_t out_at = (uint32_t)((m * a.N + part * 4) * ob);
#pragma unroll
            for (int j = 0; j < WN / 16; ++j) {
                const int nt0 = n0 + wn + j * 16;
                if (nt0 + 16 <= a.N) {
                    float y[4];
                    scaled(acc[i][j], rs[i], cs[j], y);
                    activate(y, act);
                    store_four(outr, out_at, (uint32_t)(nt0 * ob), y, a.out_dtype);
                } else if (nt0 + part * 4 < a.N && m < rows) {
                    finish(a, m0 + m, nt0 + part * 4, acc[i][j], rs[i], cs[j], act);
                }
            }
        }
    });
}

// ---- launches ----------------------------------------------------------------------------

constexpr int kRowsMostK = 256;

template <int XB, bool NORM, int KT>
hipError_t launch_rows(I8Args a, const GnArgs& g, hipStream_t stream) {
    const int tiles = (a.N + 15) / 16;
    const int64_t images = NORM ? g.N : 1, S = NORM ? g.S : a.M;
    const int64_t blocks = ((S + 15) / 16 + kRowsWaves - 1) / kRowsWaves;   // of an image
    // a slice is what fits, or less where the rows alone leave compute units without work
    const int most = (int)(kRowsLds / (16 * rows_stride(KT)));
    const int64_t want = std::max<int64_t>(1, 512 / (images * blocks));
    a.tiles_per_slice = (int32_t)std::max<int64_t>(1, std::min<int64_t>(most, tiles / want));
    a.slices = (tiles + a.tiles_per_slice - 1) / a.tiles_per_slice;
    a.tiles_per_slice = (tiles + a.slices - 1) / a.slices;
    // workgroups beyond what is resident at once would bring the weights in again
    const int64_t cap = std::max<int64_t>(1, 512 / (images * a.slices));
    a.blocks_per_image = (int32_t)std::min(blocks, cap);
    size_t lds = (size_t)a.tiles_per_slice * 16 * (rows_stride(KT) + 8) +
                 (NORM ? 3 * 64 * KT * 4 : 0);
    // Results by way of LDS where whole rows of whole 16-byte pieces fit, two workgroups to a
    // compute unit: 200704 x 128 x 108 into binary32 takes 33 us so, 42 us from the registers,
    // whose 64-byte pieces of 432-byte rows no line of memory begins or ends with.  Parts of
    // rows gained nothing: 50176 x 256 x 216 took 23 us by pieces of 128 bytes, 20 us directly.
    const size_t row = (size_t)a.N * (a.out_dtype == DA_F32 ? 4 : 2);
    a.staged = a.slices == 1 && row % 16 == 0 && lds + kRowsWaves * 16 * row <= kRowsLdsAll;
    if (a.staged) lds += kRowsWaves * 16 * row;
    i8_rows_kernel<XB, NORM, KT>
        <<<(uint32_t)(images * a.blocks_per_image * a.slices), kRowsThreads, lds, stream>>>(a, g);
    return hipGetLastError();
}

template <int XB, bool NORM>
hipError_t rows_by_depth(const I8Args& a, const GnArgs& g, hipStream_t stream) {
    if (a.K <= 128) return launch_rows<XB, NORM, 2>(a, g, stream);
    return launch_rows<XB, NORM, 4>(a, g, stream);
}

template <int XB>
hipError_t launch_skinny(const I8Args& a, hipStream_t stream) {
    const int runs = (a.K + 63) / 64, tiles = (a.N + 15) / 16;
    int kw = kSkinnyWaves;
    while (kw > 1 && runs < 4 * kw) kw /= 2;   // at least two pairs of runs to a wave
    const int mt = XB != 0 || a.M <= 16 ? 1 : a.M <= 32 ? 2 : 4;
    const uint32_t blocks = (uint32_t)((tiles + kSkinnyWaves / kw - 1) / (kSkinnyWaves / kw) *
                                       ((a.M + 16 * mt - 1) / (16 * mt)));
    const size_t lds = XB ? (size_t)a.M * (runs * 64 + 16) : 0;
    if constexpr (XB != 0) {
        i8_skinny_kernel<XB, 1><<<blocks, kSkinnyThreads, lds, stream>>>(a, kw);
    } else {
        if (mt == 1) i8_skinny_kernel<XB, 1><<<blocks, kSkinnyThreads, 0, stream>>>(a, kw);
        else if (mt == 2) i8_skinny_kernel<XB, 2><<<blocks, kSkinnyThreads, 0, stream>>>(a, kw);
        else i8_skinny_kernel<XB, 4><<<blocks, kSkinnyThreads, 0, stream>>>(a, kw);
    }
    return hipGetLastError();
}

// A product with a 256 x 256 tile for every other compute unit or more (us, against 64 x 64 tiles):
// 4096 x 1024 x 4096, 256 tiles, takes 25 (49); 1024 x 4096 x 8192, 128 tiles, 53 (72); 1792 x
// 4096 x 4096, 112 tiles, 52 (61), but 1792 x 512 x 4096 16.8 (14.7) and 1536 x 512 x 4096, 96
// tiles, 16.3 (14.1).  Its 16-byte fills of LDS are for aligned addresses: codes that begin
// elsewhere go by the smaller tiles, whose loads into registers may lie anywhere.
bool big(const I8Args& a) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(a.a) | reinterpret_cast<uintptr_t>(a.w);
    return (a.M + 255) / 256 * ((a.N + 255) / 256) >= 128 && a.K % kTileK == 0 && at % 16 == 0 &&
           a.N < (1 << 20);
}

hipError_t launch_tiles(const I8Args& a, hipStream_t stream) {
    const auto blocks = [&](int t) {
        return (uint32_t)((a.M + t - 1) / t * ((a.N + t - 1) / t));
    };
    if (big(a)) i8_big_kernel<<<blocks(kBigTile), kBigThreads, 0, stream>>>(a);
    else i8_tile_kernel<<<blocks(kTile), kTileThreads, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace

// Which kernel, by times measured on an MI355X (us a call of i8_linear in a captured graph):
//  - up to 256 columns the rows kernel: 50176 x 256 x 216 takes 19 (quantised in memory, then
//    tiled 25), 200704 x 128 x 108 24 (52), 100 x 256 x 2496 5.9 (7.5), but 900 x 256 x 2496, whose
//    78 slices read x as many times, 11.5 (9.2);
//  - up to 16 rows the streaming kernel: one row of 4096 x 4096 takes 6.7, and quantising on
//    the way saves a launch where the rows fit LDS; up to 64, and beyond them with 1024 columns
//    or more up to 128 rows or 64 tiles (one 64 x 64 tile walks its columns at 0.6 us per
//    128): 64 x 4096 x 4096 takes 19 (tiled 31), 128 x 4096 x 256 18 (31), 100 x 4096 x 4096 28
//    (31), 200 x 2048 x 1024 12 (18), but 48 x 512 x 432 10 (9), 256 x 1024 x 4096 18 (13) and
//    256 x 512 x 512 11 (9);
//  - else tiles.
I8Path i8_path(int64_t M, int64_t K, int64_t N, bool codes, bool norm) {
    // 16 rows of a binary32 result are the range of a buffer resource
    const bool rows = K <= kRowsMostK && N < (1 << 22);
    if (norm) return rows ? I8Path::kRows : I8Path::kTiles;
    if (M <= 16 && !codes && (size_t)M * ((K + 63) / 64 * 64 + 16) <= kSkinnyLds)
        return I8Path::kSkinny;
    if (M <= 16) return I8Path::kSkinnyCodes;
    if (rows) return I8Path::kRows;
    const int64_t tiles = (M + kTile - 1) / kTile * ((N + kTile - 1) / kTile);
    if (M <= 64 || (K >= 1024 && M <= 256 && (M <= 128 || tiles <= 64))) return I8Path::kSkinnyCodes;
    return I8Path::kTiles;
}

namespace {

template <int XB, bool NORM, int L, int HOLD>
hipError_t quantize(const I8Args& a, const GnArgs& g, hipStream_t stream) {
    // rows one after the other only where there are waves enough without
    const int rows = (int)std::min<int64_t>(8, std::max<int64_t>(1, a.M / 2048));
    const int64_t waves = NORM ? g.N * ((g.S + rows - 1) / rows)
                               : (a.M + kWave / L - 1) / (kWave / L);
    i8_quantize_kernel<XB, NORM, L, HOLD>
        <<<(uint32_t)((waves + kQuantWaves - 1) / kQuantWaves), kQuantThreads, 0, stream>>>(a, g, rows);
    return hipGetLastError();
}

template <int XB>
hipError_t quantize(const I8Args& a, const GnArgs* norm, hipStream_t stream) {
    if (norm)
        return a.K <= 1024 ? quantize<XB, true, 64, 2>(a, *norm, stream)
                           : quantize<XB, true, 64, 4>(a, *norm, stream);
    const GnArgs none{};
    if (a.K <= 64) return quantize<XB, false, 8, 1>(a, none, stream);
    if (a.K <= 128) return quantize<XB, false, 16, 1>(a, none, stream);
    if (a.K <= 256) return quantize<XB, false, 32, 1>(a, none, stream);
    if (a.K <= 512) return quantize<XB, false, 64, 1>(a, none, stream);
    return quantize<XB, false, 64, 4>(a, none, stream);
}

}  // namespace

hipError_t launch_i8_quantize(const I8Args& a, const GnArgs* norm, hipStream_t stream) {
    return a.x_dtype == DA_F32 ? quantize<4>(a, norm, stream) : quantize<2>(a, norm, stream);
}

hipError_t launch_i8_product(const I8Args& a, I8Path path, bool codes, const GnArgs* norm,
                             hipStream_t stream) {
    const bool wide = a.x_dtype == DA_F32;
    switch (path) {
        case I8Path::kRows:
            if (norm)
                return wide ? rows_by_depth<4, true>(a, *norm, stream)
                            : rows_by_depth<2, true>(a, *norm, stream);
            if (codes) return rows_by_depth<0, false>(a, GnArgs{}, stream);
            return wide ? rows_by_depth<4, false>(a, GnArgs{}, stream)
                        : rows_by_depth<2, false>(a, GnArgs{}, stream);
        case I8Path::kSkinny:
            return wide ? launch_skinny<4>(a, stream) : launch_skinny<2>(a, stream);
        case I8Path::kSkinnyCodes:
            return launch_skinny<0>(a, stream);
        default:
            return launch_tiles(a, stream);
    }
}

}  // namespace da
