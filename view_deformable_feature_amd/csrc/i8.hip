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

// One wave per row; a row's first 2048 numbers stay in registers, what is past them is read
// again.
constexpr int kQuantThreads = 256;
template <int XB>
__global__ __launch_bounds__(kQuantThreads) void i8_quantize_kernel(I8Args a) {
    constexpr int kHold = 4;
    const int64_t m = (int64_t)blockIdx.x * (kQuantThreads / kWave) + threadIdx.x / kWave;
    const int lane = threadIdx.x & (kWave - 1);
    if (m >= a.M) return;
    const bool bf16 = a.x_dtype == DA_BF16;
    Eight<XB> hold[kHold];
    float v[8];
    uint32_t big = 0;
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
        const int c = (i * kWave + lane) * 8;
        if (c < a.K) hold[i].load(a.x, m, c, a.K);
        else hold[i].zero();
    }
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
        hold[i].unpack(v, bf16);
        big = max(big, magnitude(v));
    }
    for (int c = (kHold * kWave + lane) * 8; c < a.K; c += kWave * 8) {
        Eight<XB> t;
        t.load(a.x, m, c, a.K);
        t.unpack(v, bf16);
        big = max(big, magnitude(v));
    }
    for (int s = kWave / 2; s; s >>= 1) big = max(big, (uint32_t)__shfl_xor((int)big, s));
    const RowScale s = row_scale(big);
    const auto put = [&](const Eight<XB>& t, int c) {
        t.unpack(v, bf16);
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
    for (int i = 0; i < kHold; ++i)
        if ((i * kWave + lane) * 8 < a.K) put(hold[i], (i * kWave + lane) * 8);
    for (int c = (kHold * kWave + lane) * 8; c < a.K; c += kWave * 8) {
        Eight<XB> t;
        t.load(a.x, m, c, a.K);
        put(t, c);
    }
    if (lane == 0) a.a_scale[m] = s.scale;
}

// The same behind a group norm whose means and rstds are in memory: rows past the rows
// kernel's depth, read twice.
template <int XB>
__global__ __launch_bounds__(kQuantThreads) void i8_norm_quantize_kernel(I8Args a, GnArgs g) {
    const int64_t m = (int64_t)blockIdx.x * (kQuantThreads / kWave) + threadIdx.x / kWave;
    const int lane = threadIdx.x & (kWave - 1);
    if (m >= a.M) return;
    const bool bf16 = a.x_dtype == DA_BF16;
    const int64_t image = m / g.S;
    const auto value = [&](int c, float (&v)[8]) {
        Eight<XB> q;
        q.load(a.x, m, c, a.K);
        q.unpack(v, bf16);
        NormCoef f;
        f.load(a, g, image, c);
        f.apply(v, g.act);
    };
    float v[8];
    uint32_t big = 0;
    for (int c = lane * 8; c < a.K; c += kWave * 8) {
        value(c, v);
        big = max(big, magnitude(v));
    }
    for (int s = kWave / 2; s; s >>= 1) big = max(big, (uint32_t)__shfl_xor((int)big, s));
    const RowScale s = row_scale(big);
    for (int c = lane * 8; c < a.K; c += kWave * 8) {
        value(c, v);
        const u32x2 q = {pack_codes(v, s), pack_codes(v + 4, s)};
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (c + e < a.K) a.a[m * a.K + c + e] = (int8_t)(q[e / 4] >> (8 * (e & 3)));
    }
    if (lane == 0) a.a_scale[m] = s.scale;
}

// ---- pieces of the operands --------------------------------------------------------------

// 16 codes of row `row` of [.., K] from column k on (k < K), zeros past K.  Any alignment.
__device__ __forceinline__ i32x4 bytes_of(const int8_t* base, int64_t row, int k, int K) {
    const int8_t* p = base + row * K + k;
    i32x4 q = {0, 0, 0, 0};
    if (k + 16 <= K) {
        __builtin_memcpy(&q, p, 16);
    } else {
#pragma unroll
        for (int i = 0; i < 15; ++i)
            if (k + i < K) q[i / 4] |= (int)((uint32_t)(uint8_t)p[i] << (8 * (i & 3)));
    }
    return q;
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
                                       float row, const ColumnScale& c) {
    float y[4];
    scaled(acc, row, c, y);
    activate(y, a.act);
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

constexpr int kRowsThreads = 512;
constexpr int kRowsWaves = kRowsThreads / kWave;
constexpr size_t kRowsLds = 64 * 1024;   // of weights: two workgroups to a compute unit

// Whole pieces of x go through a buffer resource: what lies past the wave's rows reads as
// zero, without a comparison.
constexpr uint32_t kOutside = 0x80000000u;   // past every range (each is below 2^31 bytes)

// Bytes between rows of codes in LDS: an odd number of 16-byte units, so that the 16 rows of
// an operand start in different banks.
__host__ __device__ constexpr int rows_stride(int kt) { return kt * 64 + 16; }

template <int XB, bool NORM, int KT>
__global__ __launch_bounds__(kRowsThreads, KT == 4 && (NORM || XB == 4) ? 2 : 4) void i8_rows_kernel(I8Args a,
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
        const int rows = (int)min<int64_t>(rows_end - m0, 16);
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

    for (int e = threadIdx.x; e < wrows * KT * 4; e += kRowsThreads) {
        const int r = e / (KT * 4), c = e % (KT * 4) * 16, n = t0 * 16 + r;
        i32x4 w = {0, 0, 0, 0};
        if (n < a.N && c < a.K) w = bytes_of(a.w, n, c, a.K);
        *reinterpret_cast<i32x4*>(ws + r * kStride + c) = w;
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
        const int rows = (int)min<int64_t>(rows_end - m0, 16);
        if constexpr (XB == 0) {
            rs = col < rows ? a.a_scale[m0 + col] : 0.0f;
#pragma unroll
            for (int kc = 0; kc < KT; ++kc) x[kc] = q[kc][0].q;
        } else {
            // normalised numbers are kept between the two steps; the barriers to the scheduler
            // keep the runs of 64 columns from being unpacked all at once
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
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            z[kc][e + i] = fmaf(z[kc][e + i] - m4[i], s4[i], b4[i]);
                    }
                    activate(z[kc], g.act);
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        big = max(big, __float_as_uint(z[kc][e]) & 0x7fffffffu);
                    __builtin_amdgcn_sched_barrier(0);
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
            if (t * 16 + 16 <= a.N) {
                float y[4];
                scaled(acc, rs, cs, y);
                activate(y, a.act);
                store_four(outr, out_at, (uint32_t)(t * 16 * ob), y, a.out_dtype);
            } else {   // the last tile, not all of it in the row
                const int n = t * 16 + part * 4;
                if (n < a.N && col < rows) finish(a, m0 + col, n, acc, rs, cs);
            }
        }
    }
}

// ---- panel kernel ------------------------------------------------------------------------
//
// 257 to 1024 columns, where a wave's rows no longer fit its registers twice over: a
// workgroup brings 16 * MT rows into LDS as codes, and its waves deal the 16-channel tiles
// of the output among them, the weights coming from L2 into registers a tile ahead.

constexpr int kPanelThreads = 256;
constexpr int kPanelWaves = kPanelThreads / kWave;

template <int XB, bool NORM, int KT, int MT>
__global__ __launch_bounds__(kPanelThreads, 3) void i8_panel_kernel(I8Args a, GnArgs g) {
    constexpr int kBM = 16 * MT, kStride = rows_stride(KT);
    __shared__ __align__(16) unsigned char codes[kBM * kStride];
    __shared__ uint32_t row_info[kBM];   // scale (codes), or the largest magnitude's bits
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int slice = blockIdx.x % a.slices;
    int64_t m0 = blockIdx.x / a.slices, mend = a.M, image = 0;
    if constexpr (NORM) {   // a workgroup stays in one image
        image = m0 / a.blocks_per_image;
        m0 = image * g.S + (m0 - image * a.blocks_per_image) * kBM;
        mend = (image + 1) * g.S;
    } else {
        m0 *= kBM;
    }
    const int rows = (int)min<int64_t>(mend - m0, kBM);

    if constexpr (XB == 0) {
        const auto xr = make_rsrc(a.a + m0 * a.K, rows * a.K);
        constexpr int kPer = KT * 4;   // pieces of 16 to a row
#pragma unroll
        for (int i = 0; i < kBM * kPer / kPanelThreads; ++i) {
            const int e = i * kPanelThreads + threadIdx.x, r = e / kPer, c = e % kPer * 16;
            Sixteen q;
            if (a.K % 16 == 0) q.load(xr, c < a.K ? r * a.K + c : kOutside);
            else if (r < rows && c < a.K) q.load(a.a, m0 + r, c, a.K);
            else q.zero();
            *reinterpret_cast<i32x4*>(codes + r * kStride + c) = q.q;
        }
        if (threadIdx.x < kBM)
            row_info[threadIdx.x] =
                (int)threadIdx.x < rows ? __float_as_uint(a.a_scale[m0 + threadIdx.x]) : 0u;
    } else {
        // a wave's 4 * MT rows one after the other, NV vectors of eight to a lane
        constexpr int NV = KT / 8, kIters = 4 * MT, kBatch = 8 / NV;
        const auto xr = make_rsrc(static_cast<const char*>(a.x) + m0 * a.K * XB, rows * a.K * XB);
        const bool bf16 = a.x_dtype == DA_BF16, pieces = a.K % 8 == 0;
        const int c0 = lane * 8, r0 = wave * kIters;
        NormCoef f[NORM ? NV : 1];
        if constexpr (NORM) {
#pragma unroll
            for (int j = 0; j < NV; ++j) f[j].load(a, g, image, c0 + j * kWave * 8);
        }
#pragma unroll 1
        for (int b = 0; b < kIters; b += kBatch) {
            Eight<XB> q[kBatch][NV];
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    const int r = r0 + b + i, c = c0 + j * kWave * 8;
                    if (pieces) q[i][j].load(xr, c < a.K ? (r * a.K + c) * XB : kOutside);
                    else if (r < rows && c < a.K) q[i][j].load(a.x, m0 + r, c, a.K);
                    else q[i][j].zero();
                }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int r = r0 + b + i;
                float v[NV][8];
                uint32_t big = 0;
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    q[i][j].unpack(v[j], bf16);
                    if constexpr (NORM) {
                        f[j].apply(v[j], g.act);
                        big = max(big, magnitude(v[j]));
                    } else {
                        big = max(big, q[i][j].magnitude());
                    }
                }
                if constexpr (!NORM) big = Eight<XB>::widen(big, bf16);
#pragma unroll
                for (int s = kWave / 2; s; s >>= 1) big = max(big, (uint32_t)__shfl_xor((int)big, s));
                const RowScale s = row_scale(big);
#pragma unroll
                for (int j = 0; j < NV; ++j)
                    *reinterpret_cast<u32x2*>(codes + r * kStride + c0 + j * kWave * 8) =
                        u32x2{pack_codes(v[j], s), pack_codes(v[j] + 4, s)};
                if (lane == 0) row_info[r] = big;
            }
        }
    }
    __syncthreads();

    const int col = lane % 16, part = lane / 16;
    int at_row = col * kStride + part * 16;
    float rs[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
        rs[mt] = XB == 0 ? __uint_as_float(row_info[mt * 16 + col])
                         : row_scale(row_info[mt * 16 + col]).scale;

    // a wave's weights come in halves of 512 columns, the next half and the next tile's scales
    // on their way while one is multiplied; what is fetched past a row of the weights meets
    // codes that are zero
    const int tiles = (a.N + 15) / 16;
    const int t1 = min(tiles, (slice + 1) * a.tiles_per_slice);
    const auto wr = make_rsrc(a.w, (uint32_t)((int64_t)a.N * a.K) & ~3u);
    const auto sr = make_rsrc(a.w_scale, a.N * 4u), br = make_rsrc(a.bias, a.bias ? a.N * 4u : 0u);
    const uint32_t w_at = col * a.K + part * 16;
    const auto weights = [&](int t, int kc0, i32x4 (&wf)[8]) {
        if (a.K % 16 && t == tiles - 1) {   // the matrix may end inside a piece
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int k = (kc0 + i) * 64 + part * 16;
                wf[i] = k < a.K ? bytes_of(a.w, min(t * 16 + col, a.N - 1), k, a.K)
                                : i32x4{0, 0, 0, 0};
            }
        } else {
            Sixteen q;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                q.load(wr, w_at + (uint32_t)(t * 16 * a.K) + (kc0 + i) * 64);
                wf[i] = q.q;
            }
        }
    };
    const auto scales = [&](int t) {
        ColumnScale c;
        Sixteen s, b;
        s.load(sr, part * 16 + t * 64);
        b.load(br, part * 16 + t * 64);
        __builtin_memcpy(c.s, &s.q, 16);
        __builtin_memcpy(c.b, &b.q, 16);
        return c;
    };
    const int ob = a.out_dtype == DA_F32 ? 4 : 2;
    const auto outr = make_rsrc(static_cast<char*>(a.out) + m0 * a.N * ob, rows * a.N * ob);
    uint32_t out_at[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) out_at[mt] = (uint32_t)(((mt * 16 + col) * a.N + part * 4) * ob);

    int t = slice * a.tiles_per_slice + wave;
    if (t >= t1) return;
    i32x4 wf[8];
    weights(t, 0, wf);
    ColumnScale cs = scales(t);
    for (; t < t1; t += kPanelWaves) {
        const int tn = t + kPanelWaves;
        // the rows' operands are read anew for each tile: kept, they would fill the registers
        asm volatile("" : "+v"(at_row));
        ColumnScale csn = cs;
        i32x4 acc[MT];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) acc[mt] = i32x4{0, 0, 0, 0};
#pragma unroll
        for (int kc0 = 0; kc0 < KT; kc0 += 8) {
            i32x4 next[8] = {};
            if (kc0 + 8 < KT) {
                weights(t, kc0 + 8, next);
            } else if (tn < t1) {
                weights(tn, 0, next);
                csn = scales(tn);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
                    acc[mt] = mfma(wf[i], *reinterpret_cast<const i32x4*>(
                                              codes + at_row + mt * 16 * kStride + (kc0 + i) * 64),
                                   acc[mt]);
#pragma unroll
            for (int i = 0; i < 8; ++i) wf[i] = next[i];
        }
        if (t * 16 + 16 <= a.N) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                float y[4];
                scaled(acc[mt], rs[mt], cs, y);
                activate(y, a.act);
                store_four(outr, out_at[mt], (uint32_t)(t * 16 * ob), y, a.out_dtype);
            }
        } else {   // the last tile, not all of it in the row
            const int n = t * 16 + part * 4;
            if (n < a.N) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
                    if (mt * 16 + col < rows)
                        finish(a, m0 + mt * 16 + col, n, acc[mt], rs[mt], cs);
            }
        }
        cs = csn;
    }
}

// ---- streaming kernel --------------------------------------------------------------------
//
// At most 16 * MT rows: a wave takes 16 output channels and every KW-th run of 64 columns,
// the weights going from memory into operand registers, several runs in flight; the KW
// waves' sums meet in LDS.  The rows' codes come from memory (XB 0), or the workgroup
// quantises up to 16 rows of x into LDS first.

constexpr int kSkinnyThreads = 512;
constexpr int kSkinnyWaves = kSkinnyThreads / kWave;
constexpr int kSkinnyRuns = 8;                 // weight runs of a wave in flight
constexpr size_t kSkinnyLds = 48 * 1024;       // of codes

template <int XB, int MT>
__global__ __launch_bounds__(kSkinnyThreads) void i8_skinny_kernel(I8Args a, int kw_count) {
    extern __shared__ __align__(16) unsigned char codes[];   // [M][stride], XB != 0
    __shared__ __align__(16) i32x4 meet[kSkinnyWaves][MT][kWave];
    __shared__ uint32_t bigs[16][kSkinnyWaves];
    __shared__ float scales[16];
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int col = lane % 16, part = lane / 16;
    const int kw = wave % kw_count;
    const int tile = blockIdx.x * (kSkinnyWaves / kw_count) + wave / kw_count;
    const int tiles = (a.N + 15) / 16, runs = (a.K + 63) / 64;
    const int stride = runs * 64 + 16;
    const int n = min(tile * 16 + col, a.N - 1);
    const bool live = tile < tiles;

    i32x4 wf[kSkinnyRuns];
    const auto fetch = [&](int c) {
#pragma unroll
        for (int i = 0; i < kSkinnyRuns; ++i) {
            const int k = (c + i * kw_count) * 64 + part * 16;
            wf[i] = live && k < a.K ? bytes_of(a.w, n, k, a.K) : i32x4{0, 0, 0, 0};
        }
    };
    fetch(kw);   // on its way while the rows are quantised

    if constexpr (XB != 0) {
        // 8 / 2^j waves to a row
        const bool bf16 = a.x_dtype == DA_BF16;
        int share = 1;
        while (share < kSkinnyWaves && kSkinnyWaves / (2 * share) >= (int)a.M) share *= 2;
        const int part_of = wave % share;
        for (int m = wave / share; m < (int)a.M; m += kSkinnyWaves / share) {
            uint32_t big = 0;
            for (int c = (part_of * kWave + lane) * 8; c < a.K; c += share * kWave * 8) {
                Eight<XB> q;
                float v[8];
                q.load(a.x, m, c, a.K);
                q.unpack(v, bf16);
                big = max(big, magnitude(v));
            }
            for (int s = kWave / 2; s; s >>= 1) big = max(big, (uint32_t)__shfl_xor((int)big, s));
            if (lane == 0) bigs[m][part_of] = big;
        }
        __syncthreads();
        for (int m = wave / share; m < (int)a.M; m += kSkinnyWaves / share) {
            uint32_t big = 0;
            for (int i = 0; i < share; ++i) big = max(big, bigs[m][i]);
            const RowScale s = row_scale(big);
            for (int c = (part_of * kWave + lane) * 8; c < runs * 64; c += share * kWave * 8) {
                Eight<XB> q;
                float v[8];
                if (c < a.K) q.load(a.x, m, c, a.K);
                else q.zero();
                q.unpack(v, bf16);
                *reinterpret_cast<u32x2*>(codes + m * stride + c) =
                    u32x2{pack_codes(v, s), pack_codes(v + 4, s)};
            }
            if (part_of == 0 && lane == 0) scales[m] = s.scale;
        }
        __syncthreads();
    }

    i32x4 acc[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) acc[mt] = i32x4{0, 0, 0, 0};
    for (int c = kw; c < runs;) {
        i32x4 now[kSkinnyRuns];
#pragma unroll
        for (int i = 0; i < kSkinnyRuns; ++i) now[i] = wf[i];
        const int at = c;
        c += kSkinnyRuns * kw_count;
        if (c < runs) fetch(c);
#pragma unroll
        for (int i = 0; i < kSkinnyRuns; ++i) {
            const int k = (at + i * kw_count) * 64 + part * 16;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                i32x4 x = {0, 0, 0, 0};
                const int m = mt * 16 + col;
                if constexpr (XB != 0) {
                    if (m < (int)a.M && k < runs * 64)
                        x = *reinterpret_cast<const i32x4*>(codes + m * stride + k);
                } else {
                    if (m < (int)a.M && k < a.K) x = bytes_of(a.a, m, k, a.K);
                }
                acc[mt] = mfma(now[i], x, acc[mt]);
            }
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
        if (m < (int)a.M) finish(a, m, nn, t, XB != 0 ? scales[m] : a.a_scale[m], cs);
    }
}

// ---- tiled product -----------------------------------------------------------------------
//
// BM rows by BN output channels to a workgroup, 128 columns at a time through LDS, each
// wave WM x WN of it; the next 128 columns are on their way to registers while the matrix
// cores work.  A 16-byte piece p of an LDS row r sits at place p ^ f(r), so that the 16 rows
// an operand is read from fall into different banks.

constexpr int kTileK = 128;

template <int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(BM / WM * (BN / WN) * kWave) void i8_tile_kernel(I8Args a) {
    constexpr int kThreads = BM / WM * (BN / WN) * kWave;
    constexpr int kPieces = kTileK / 16;                       // of a row
    constexpr int kXLoads = BM * kPieces / kThreads, kWLoads = BN * kPieces / kThreads;
    static_assert(BM * kPieces % kThreads == 0 && BN * kPieces % kThreads == 0, "whole loads");
    __shared__ __align__(16) i32x4 xs[2][BM * kPieces], ws[2][BN * kPieces];
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int col = lane % 16, part = lane / 16;
    const int wm = wave % (BM / WM) * WM, wn = wave / (BM / WM) * WN;

    // Workgroups go round the 8 XCDs: each gets a run of consecutive tiles, and runs go down
    // 8 row tiles before the next column tile, so that an XCD's L2 sees few operands.
    const int mt = (int)((a.M + BM - 1) / BM), nt = (a.N + BN - 1) / BN;
    int id = blockIdx.x;
    {
        const int total = mt * nt, per = total / 8, extra = total % 8;
        const int x = id % 8, i = id / 8;
        id = x * per + min(x, extra) + i;
    }
    const int band = id / (8 * nt), in_band = id - band * 8 * nt;
    const int rows = min(8, mt - band * 8);
    const int64_t m0 = (int64_t)(band * 8 + in_band % rows) * BM;
    const int n0 = in_band / rows * BN;

    i32x4 xq[kXLoads], wq[kWLoads];
    const auto fetch = [&](int k0) {
#pragma unroll
        for (int i = 0; i < kXLoads; ++i) {
            const int e = i * kThreads + threadIdx.x;
            const int64_t m = min(m0 + e / kPieces, a.M - 1);
            const int k = k0 + e % kPieces * 16;
            xq[i] = k < a.K ? bytes_of(a.a, m, k, a.K) : i32x4{0, 0, 0, 0};
        }
#pragma unroll
        for (int i = 0; i < kWLoads; ++i) {
            const int e = i * kThreads + threadIdx.x;
            const int n = min(n0 + e / kPieces, a.N - 1);
            const int k = k0 + e % kPieces * 16;
            wq[i] = k < a.K ? bytes_of(a.w, n, k, a.K) : i32x4{0, 0, 0, 0};
        }
    };
    const auto place = [](int r, int p) { return r * kPieces + (p ^ ((r >> 1) & 7)); };
    const auto put = [&](int b) {
#pragma unroll
        for (int i = 0; i < kXLoads; ++i) {
            const int e = i * kThreads + threadIdx.x;
            xs[b][place(e / kPieces, e % kPieces)] = xq[i];
        }
#pragma unroll
        for (int i = 0; i < kWLoads; ++i) {
            const int e = i * kThreads + threadIdx.x;
            ws[b][place(e / kPieces, e % kPieces)] = wq[i];
        }
    };

    i32x4 acc[WM / 16][WN / 16];
#pragma unroll
    for (int i = 0; i < WM / 16; ++i)
#pragma unroll
        for (int j = 0; j < WN / 16; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
    fetch(0);
    put(0);
    __syncthreads();
    int b = 0;
    for (int k0 = 0; k0 < a.K; k0 += kTileK, b ^= 1) {
        const bool more = k0 + kTileK < a.K;
        if (more) fetch(k0 + kTileK);
#pragma unroll
        for (int kc = 0; kc < kTileK / 64; ++kc) {
            i32x4 xf[WM / 16], wf[WN / 16];
#pragma unroll
            for (int i = 0; i < WM / 16; ++i) xf[i] = xs[b][place(wm + i * 16 + col, kc * 4 + part)];
#pragma unroll
            for (int j = 0; j < WN / 16; ++j) wf[j] = ws[b][place(wn + j * 16 + col, kc * 4 + part)];
#pragma unroll
            for (int i = 0; i < WM / 16; ++i)
#pragma unroll
                for (int j = 0; j < WN / 16; ++j) acc[i][j] = mfma(wf[j], xf[i], acc[i][j]);
        }
        if (more) put(b ^ 1);
        __syncthreads();
    }
#pragma unroll
    for (int j = 0; j < WN / 16; ++j) {
        const int n = n0 + wn + j * 16 + part * 4;
        if (n >= a.N) continue;
        const ColumnScale c = column_scale(a, n);
#pragma unroll
        for (int i = 0; i < WM / 16; ++i) {
            const int64_t m = m0 + wm + i * 16 + col;
            if (m < a.M) finish(a, m, n, acc[i][j], a.a_scale[m], c);
        }
    }
}

// ---- launches ----------------------------------------------------------------------------

constexpr int kRowsMostK = 256, kPanelMostK = 1024;

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
    const size_t lds = (size_t)a.tiles_per_slice * 16 * (rows_stride(KT) + 8) +
                       (NORM ? 3 * 64 * KT * 4 : 0);
    i8_rows_kernel<XB, NORM, KT>
        <<<(uint32_t)(images * a.blocks_per_image * a.slices), kRowsThreads, lds, stream>>>(a, g);
    return hipGetLastError();
}

template <int XB, bool NORM, int KT, int MT>
hipError_t launch_panel(I8Args a, const GnArgs& g, hipStream_t stream) {
    constexpr int kBM = 16 * MT;
    int64_t blocks = (a.M + kBM - 1) / kBM;
    if (NORM) {
        a.blocks_per_image = (int32_t)((g.S + kBM - 1) / kBM);
        blocks = (int64_t)g.N * a.blocks_per_image;
    }
    // output tiles are shared out where the row blocks alone leave compute units idle
    const int tiles = (a.N + 15) / 16;
    const int64_t want = std::max<int64_t>(1, 512 / blocks);
    a.tiles_per_slice = (int32_t)std::max<int64_t>(std::min(tiles, kPanelWaves),
                                                   (tiles + want - 1) / want);
    a.slices = (tiles + a.tiles_per_slice - 1) / a.tiles_per_slice;
    i8_panel_kernel<XB, NORM, KT, MT>
        <<<(uint32_t)(blocks * a.slices), kPanelThreads, 0, stream>>>(a, g);
    return hipGetLastError();
}

template <int XB, bool NORM>
hipError_t rows_by_depth(const I8Args& a, const GnArgs& g, hipStream_t stream) {
    if (a.K <= 128) return launch_rows<XB, NORM, 2>(a, g, stream);
    if (a.K <= kRowsMostK) return launch_rows<XB, NORM, 4>(a, g, stream);
    const int64_t blocks = NORM ? (int64_t)g.N * ((g.S + 63) / 64) : (a.M + 63) / 64;
    // 64 rows share what is fetched of the weights; 32 where that many row blocks are few
    if (a.K <= 512)
        return blocks < 128 ? launch_panel<XB, NORM, 8, 2>(a, g, stream)
                            : launch_panel<XB, NORM, 8, 4>(a, g, stream);
    return blocks < 128 ? launch_panel<XB, NORM, 16, 2>(a, g, stream)
                        : launch_panel<XB, NORM, 16, 4>(a, g, stream);
}

template <int XB>
hipError_t launch_skinny(const I8Args& a, hipStream_t stream) {
    const int runs = (a.K + 63) / 64, tiles = (a.N + 15) / 16;
    int kw = kSkinnyWaves;
    while (kw > 1 && runs < 2 * kw) kw /= 2;
    const uint32_t blocks = (uint32_t)((tiles + kSkinnyWaves / kw - 1) / (kSkinnyWaves / kw));
    const size_t lds = XB ? (size_t)a.M * (runs * 64 + 16) : 0;
    if constexpr (XB != 0) {
        i8_skinny_kernel<XB, 1><<<blocks, kSkinnyThreads, lds, stream>>>(a, kw);
    } else {
        if (a.M <= 16) i8_skinny_kernel<XB, 1><<<blocks, kSkinnyThreads, 0, stream>>>(a, kw);
        else if (a.M <= 32) i8_skinny_kernel<XB, 2><<<blocks, kSkinnyThreads, 0, stream>>>(a, kw);
        else i8_skinny_kernel<XB, 4><<<blocks, kSkinnyThreads, 0, stream>>>(a, kw);
    }
    return hipGetLastError();
}

template <int BM, int BN, int WM, int WN>
hipError_t launch_tile(const I8Args& a, hipStream_t stream) {
    const int64_t blocks = (a.M + BM - 1) / BM * ((a.N + BN - 1) / BN);
    i8_tile_kernel<BM, BN, WM, WN>
        <<<(uint32_t)blocks, BM / WM * (BN / WN) * kWave, 0, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_tiles(const I8Args& a, hipStream_t stream) {
    const auto blocks = [&](int bm, int bn) {
        return (a.M + bm - 1) / bm * ((a.N + bn - 1) / bn);
    };
    if (blocks(256, 256) >= 200) return launch_tile<256, 256, 128, 64>(a, stream);
    if (blocks(128, 128) >= 256) return launch_tile<128, 128, 64, 64>(a, stream);
    return launch_tile<64, 64, 32, 32>(a, stream);
}

}  // namespace

I8Path i8_path(int64_t M, int64_t K, int64_t N, bool codes, bool norm) {
    // ranges of buffer resources: the weights, and 64 rows of a binary32 result
    const bool rows = K <= kPanelMostK && N * K < (int64_t(1) << 31) && N < (1 << 22);
    if (norm) return rows ? I8Path::kRows : I8Path::kTiles;
    if (M <= 16 && !codes && (size_t)M * ((K + 63) / 64 * 64 + 16) <= kSkinnyLds)
        return I8Path::kSkinny;
    if (M <= 64) return I8Path::kSkinnyCodes;
    if (rows) return I8Path::kRows;
    return I8Path::kTiles;
}

hipError_t launch_i8_quantize(const I8Args& a, const GnArgs* norm, hipStream_t stream) {
    const uint32_t blocks = (uint32_t)((a.M + kQuantThreads / kWave - 1) / (kQuantThreads / kWave));
    if (norm) {
        if (a.x_dtype == DA_F32)
            i8_norm_quantize_kernel<4><<<blocks, kQuantThreads, 0, stream>>>(a, *norm);
        else
            i8_norm_quantize_kernel<2><<<blocks, kQuantThreads, 0, stream>>>(a, *norm);
        return hipGetLastError();
    }
    if (a.x_dtype == DA_F32) i8_quantize_kernel<4><<<blocks, kQuantThreads, 0, stream>>>(a);
    else i8_quantize_kernel<2><<<blocks, kQuantThreads, 0, stream>>>(a);
    return hipGetLastError();
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
