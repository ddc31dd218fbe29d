// What the attention kernels share: tiles in LDS, their products with columns in registers.
//
// Every kernel holds 32 columns to a wave in registers (queries, or keys for their gradients)
// and streams tiles of rows through LDS.  With the matrix instruction of 32 x 32 results lane l
// has column l % 32, and of each 32 rows those at 8 (i / 4) + 4 (l / 32) + i % 4, i = 0 .. 15.
// Two products suffice:
//  * rows times columns, over the numbers of a head: lane l takes 16 bytes of row l % 32,
//    pieces l / 32, 2 + l / 32, ... (the order of a sum's terms is free, the columns' pieces
//    are taken alike);
//  * the transposed tile times such a result, over the rows: a lane's 16 results of 32 rows are,
//    eight by eight, the second operand as they stand, if the first one takes its rows in the
//    same order: 16 s + 4 (l / 32) + 0 .. 3 and 8 more, which the transposing read of LDS
//    delivers four by four.
// So nothing of the scores is exchanged between lanes, and a column's maximum, sum and
// gradient statistics are one register each.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "act_device.h"
#include "attn_internal.h"

namespace da {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef const __attribute__((address_space(3))) char* LdsBytes;

constexpr float kInf = __builtin_inff();
constexpr float kLn2 = 0.69314718f;

// acc += a b^T over one 16-byte piece of either operand's 32 rows and lane half.
template <typename T>
__device__ __forceinline__ f32x16 mul_pieces(u32x4 a, u32x4 b, f32x16 acc) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            acc = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a[e]), __uint_as_float(b[e]),
                                                       acc, 0, 0, 0);
        return acc;
    } else {
        typedef T vec __attribute__((ext_vector_type(8)));
        const vec x = __builtin_bit_cast(vec, a), y = __builtin_bit_cast(vec, b);
        if constexpr (std::is_same<T, __bf16>::value)
            return __builtin_amdgcn_mfma_f32_32x32x16_bf16(x, y, acc, 0, 0, 0);
        else
            return __builtin_amdgcn_mfma_f32_32x32x16_f16(x, y, acc, 0, 0, 0);
    }
}

// The largest of a value over the two lanes of a column; its sum.
__device__ __forceinline__ float column_max(float v) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float column_sum(float v) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// A tile of ROWS rows of DP numbers, in pieces of 16 bytes.  A row's pieces are turned by an
// exclusive or that depends on the row, so that neither 16 rows' equal pieces (rows times
// columns) nor 64 bytes of four rows in a row (the transposing read) meet in the banks.
// THREADS fill it together.
template <typename T, int DP, int ROWS, int THREADS = kAttnThreads>
struct Tile {
    static constexpr int kUsed = DP * (int)sizeof(T) / 16;
    static constexpr int kRow = kUsed <= 4 ? 4 : kUsed <= 8 ? 8 : kUsed <= 16 ? 16 : 32;
    static constexpr int kPieces = ROWS * kRow;
    static constexpr int kBytesRow = kRow * 16;
    static constexpr int kThreads = THREADS;
    static constexpr int kFetches = kPieces / THREADS;
    static constexpr int kSteps = DP * (int)sizeof(T) / 32;   // pieces of a lane half
    static constexpr int kRowsFetch = THREADS / kRow;

    static __host__ __device__ constexpr int turn(int row) {
        return kRow >= 16 ? ((row & 3) << 2) | ((row >> 2) & 3)
               : kRow == 8 ? (((row >> 1) & 1) << 2) | ((row >> 2) & 3)
                           : (row >> 2) & 3;
    }
};

// A lane's places in tiles.  All rows that differ by multiples of 16 are turned alike, and the
// other parts of a piece's number have bits of their own, so that what a loop adds to them is
// an exclusive or with a constant.
template <typename T, int DP>
struct Places {
    using Tl = Tile<T, DP, 64>;
    uint32_t row;   // piece l / 32 of row l % 32
    uint32_t col;   // transposed: 16 bits, row 4 (l / 32) + l % 16 / 4, numbers 16 (l / 16 % 2) +
                    // 4 (l % 4) ..; 32 bits, row 4 (l / 32), number l % 32
    __device__ __forceinline__ Places(int lane) {
        const int c = lane % 32, h = lane / 32;
        row = c * Tl::kBytesRow + ((h ^ Tl::turn(c)) * 16);
        if constexpr (sizeof(T) == 2) {
            const int r = 4 * h + lane % 16 / 4;
            col = r * Tl::kBytesRow + (((lane / 16 % 2 * 2 + lane % 4 / 2) ^ Tl::turn(r)) * 16) +
                  lane % 2 * 8;
        } else {
            const int r = 4 * h;
            col = r * Tl::kBytesRow + ((c / 4) ^ Tl::turn(r)) * 16 + c % 4 * 4;
        }
    }
    // pieces 2 t + l / 32 of the block's rows
    __device__ __forceinline__ u32x4 row_piece(LdsBytes tile, int block, int t) const {
        return *reinterpret_cast<const __attribute__((address_space(3))) u32x4*>(
            tile + (row ^ (t * 32)) + block * 32 * Tl::kBytesRow);
    }
    // rows 16 s + 4 (l / 32) + 0 .. 3 and 8 more of the block, number 32 d + l % 32
    __device__ __forceinline__ u32x4 col_piece(LdsBytes tile, int block, int s, int d) const {
        typedef short four __attribute__((ext_vector_type(4)));
        const auto read = [&](int j) {
            return __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (__attribute__((address_space(3))) four*)(
                    const_cast<__attribute__((address_space(3))) char*>(tile) +
                    (col ^ (d * 64) ^ (j * 32)) + (block * 32 + s * 16 + j * 8) * Tl::kBytesRow));
        };
        const u32x2 a = __builtin_bit_cast(u32x2, read(0)), b = __builtin_bit_cast(u32x2, read(1));
        return u32x4{a[0], a[1], b[0], b[1]};
    }
    // row 8 (i / 4) + 4 (l / 32) + i % 4 of the block, number 32 d + l % 32
    __device__ __forceinline__ float col_number(LdsBytes tile, int block, int i, int d) const {
        const int r = 8 * (i / 4) + i % 4;
        return *reinterpret_cast<const __attribute__((address_space(3))) float*>(
            tile + (col ^ ((d * 8) ^ Tl::turn(r)) * 16) + (block * 32 + r) * Tl::kBytesRow);
    }
};

// A block's 16 results of a lane, as the second operand of a product over its rows.  LOW: with
// a second term, the rest that the rounding to 16 bits left.
template <typename T, bool LOW>
struct Weights {
    u32x4 high[2], low[2];
    __device__ __forceinline__ explicit Weights(const f32x16& p) {
        typedef T vec __attribute__((ext_vector_type(8)));
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            vec h, l;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                h[e] = (T)p[8 * s + e];
                if constexpr (LOW) l[e] = (T)(p[8 * s + e] - (float)h[e]);
            }
            high[s] = __builtin_bit_cast(u32x4, h);
            if constexpr (LOW) low[s] = __builtin_bit_cast(u32x4, l);
        }
    }
};
template <bool LOW>
struct Weights<float, LOW> {
    f32x16 p;
    __device__ __forceinline__ explicit Weights(const f32x16& v) : p(v) {}
};

// acc[d] += the block's rows, transposed, times w
template <typename T, int DP, bool LOW>
__device__ __forceinline__ void mul_rows(const Places<T, DP>& at, LdsBytes tile, int block,
                                         const Weights<T, LOW>& w, f32x16 (&acc)[DP / 32]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
#pragma unroll
            for (int d = 0; d < DP / 32; ++d)
                acc[d] = __builtin_amdgcn_mfma_f32_32x32x2f32(at.col_number(tile, block, i, d), w.p[i],
                                                              acc[d], 0, 0, 0);
    } else {
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int d = 0; d < DP / 32; ++d) {
                const u32x4 v = at.col_piece(tile, block, s, d);
                acc[d] = mul_pieces<T>(v, w.high[s], acc[d]);
                if constexpr (LOW) acc[d] = mul_pieces<T>(v, w.low[s], acc[d]);
            }
    }
}

__device__ __forceinline__ f32x16 all_equal(float v) {
    f32x16 x;
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = v;
    return x;
}

// The block's rows times the columns in registers, added to acc.
template <typename T, int DP>
__device__ __forceinline__ f32x16 mul_columns(const Places<T, DP>& at, LdsBytes tile, int block,
                                              const u32x4 (&cols)[Tile<T, DP, 64>::kSteps],
                                              f32x16 acc = all_equal(0.0f)) {
#pragma unroll
    for (int t = 0; t < Tile<T, DP, 64>::kSteps; ++t)
        acc = mul_pieces<T>(at.row_piece(tile, block, t), cols[t], acc);
    return acc;
}

// A lane's pieces of its column: D numbers at p, zeros past them and without a column.
template <typename T, int DP>
__device__ __forceinline__ void load_column(const char* p, bool there, int D, int half,
                                            u32x4 (&cols)[Tile<T, DP, 64>::kSteps]) {
    const int pieces = there ? D * (int)sizeof(T) / 16 : 0;
#pragma unroll
    for (int t = 0; t < Tile<T, DP, 64>::kSteps; ++t) {
        cols[t] = u32x4{0, 0, 0, 0};
        if (2 * t + half < pieces)
            cols[t] = *reinterpret_cast<const u32x4*>(p + (2 * t + half) * 16);
    }
}

// Which of up to 64 keys are visible, a bit each, from their number and their bytes of a mask; the
// bytes are read a tile ahead, a key to a lane.
struct Visible {
    uint64_t bits;
    __device__ __forceinline__ bool operator()(int row) const { return (bits >> row) & 1; }
    __device__ __forceinline__ uint32_t block(int b) const { return (uint32_t)(bits >> (b * 32)); }
};
// Fills a tile in LDS straight from memory: a filling instruction puts lane l's 16 bytes at
// place l of a run of 1 KB, so the turned order is in the addresses that the lanes fetch
// from.  Rows past `rows`, numbers past D and, with a mask, rows that are not visible become zeros.
template <class Tl>
struct Filler {
    int row, piece;        // of the first fetch, the piece as it is turned there
    uint32_t pieces;       // of a row, D numbers
    __device__ __forceinline__ Filler(int thread, int row_bytes)
        : row(thread / Tl::kRow), piece(thread % Tl::kRow), pieces(row_bytes / 16) {}
    template <bool MASK>
    __device__ __forceinline__ void run(const char* base, int rows, uint32_t stride, u32x4* tile,
                                        int wave, const Visible& vis) const {
        // whole numbers in scalar registers, or every fetch becomes a loop over a lane's values
        rows = __builtin_amdgcn_readfirstlane(rows);
        const uint64_t place = reinterpret_cast<uint64_t>(base);
        // (the builtin's result is signed)
        const uint32_t high = __builtin_amdgcn_readfirstlane((uint32_t)(place >> 32));
        const uint32_t low = __builtin_amdgcn_readfirstlane((uint32_t)place);
        const uint64_t from = (uint64_t)high << 32 | low;
        const uint32_t bytes = rows <= 0 ? 0u : (uint32_t)(rows - 1) * stride + pieces * 16;
        const auto r = make_rsrc(reinterpret_cast<const void*>(from), bytes);
#pragma unroll
        for (int i = 0; i < Tl::kFetches; ++i) {
            const int at = row + i * Tl::kRowsFetch;
            const uint32_t p = piece ^ Tl::turn(at);
            const bool there = p < pieces && (!MASK || vis(at));
            const uint32_t off = there ? at * stride + p * 16 : 0x80000000u;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                r, (__attribute__((address_space(3))) void*)(tile + i * Tl::kThreads + wave * 64), 16,
                off, 0, 0, 0);
        }
    }
};

// Ends a tile: the wave's fills of LDS have arrived, which a barrier by itself does not wait for,
// and every wave has done with the tile.
__device__ __forceinline__ void tile_barrier() {
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __syncthreads();
}

// Walks over `tiles` tiles with two buffers: a tile is worked on while the next one fills the other.
// fetch(i) starts the next tile's fills of buffer i, keep(i) puts down what else of it came by
// registers, step(i) works on it; i is a constant, so that what is filled and what is read are
// arrays of their own.  The loop has no branches of its own, so that results stay in their registers,
// and fetches past the end, where fetch gives zeros.  (Three buffers gained nothing with heads of 64
// numbers, for which there is room: 6 x 900 on up to 1201 keys, gradients, 62 us, 63 so.)
template <class Fetch, class Step, class Keep>
__device__ __forceinline__ void walk(int tiles, Fetch fetch, Step step, Keep keep) {
    constexpr std::integral_constant<int, 0> first{};
    constexpr std::integral_constant<int, 1> second{};
    if (tiles <= 0) return;
    fetch(first);
    keep(first);
    tile_barrier();
    for (int j = 0; j + 1 < tiles; j += 2) {
        fetch(second);
        step(first);
        keep(second);
        tile_barrier();
        fetch(first);
        step(second);
        keep(first);
        tile_barrier();
    }
    if (tiles % 2) step(first);
}

// The wave's own fills of LDS have arrived and its reads are done.
__device__ __forceinline__ void own_fills() {
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
}

__device__ __forceinline__ uint32_t mask_byte(const uint8_t* mask, int keys, int lane) {
    uint32_t byte = 0;
    if (lane < keys) byte = mask[lane];
    return byte;
}
__device__ __forceinline__ Visible visible(uint32_t byte, int keys, int lane) {
    return {__ballot(byte && lane < keys)};
}
// Scores (or dS) of a block of keys, `other` where the key is not visible
__device__ __forceinline__ void hide(f32x16& s, uint32_t see, float other) {
    if (see == ~0u) return;
    // a row's bit, for the lanes of either half, as a mask of lanes in scalar registers
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int at = 8 * (i / 4) + i % 4;
        const uint32_t low = see & (1u << at) ? ~0u : 0u, high = see & (1u << (at + 4)) ? ~0u : 0u;
        s[i] = __builtin_amdgcn_inverse_ballot_w64((uint64_t)high << 32 | low) ? s[i] : other;
    }
}

// The workgroup's place: (batch entry, key head), tile of columns, split of keys.  Workgroups go
// to the eight XCDs in turn, and those of a key head stay on one, whose L2 then has its states:
// by whole key heads where they divide by eight, so that entries of different lengths spread,
// else by runs of workgroups.
struct Spot {
    int unit, tile, split;
    bool there;
};
__device__ __forceinline__ Spot spot_of(const AttnArgs& a, uint32_t n, uint32_t blocks) {
    const uint32_t per = (uint32_t)(a.col_tiles * a.splits);
    uint32_t unit, rest;
    bool there = true;
    if ((uint32_t)(a.B * a.Hk) % 8 == 0) {
        unit = n % 8 + n / 8 / per * 8;
        rest = n / 8 % per;
    } else {
        const uint32_t line = n % 8 * (blocks / 8) + n / 8;
        there = line < (uint32_t)a.blocks;
        unit = line / per;
        rest = line % per;
    }
    return {(int)unit, (int)(rest / a.splits), (int)(rest % a.splits), there};
}

// The number of keys of a batch entry.
__device__ __forceinline__ int keys_of(const AttnArgs& a, int b) {
    return a.lens ? min(max(a.lens[b], 0), a.Nk) : a.Nk;
}

// A lane's part of its column's result, numbers 32 d + 8 j + 4 (l / 32) + 0 .. 3 each times
// `factor`, to p (the column's D numbers in memory).
template <typename T, int ND>
__device__ __forceinline__ void store_column(T* p, int D, int half, const f32x16 (&acc)[ND],
                                             float factor) {
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int at = d * 32 + j * 8 + half * 4;
            if (at >= D) continue;
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = acc[d][4 * j + e] * factor;
            store_as(p + at, v);
        }
}

// Gradients' weights p (dP - delta) in binary16: its range is short, so each column scales them by
// a power of two of its own, chosen when the first that is not 0 comes, at 2^8, and again
// when one passes 2^15.  In the other types they stay as they are.
template <typename T, int ND>
struct Lift {
    float up = 0.0f, limit = 0.0f;   // limit: 2^15 / up
    __device__ __forceinline__ void apply(f32x16& ds, f32x16 (&acc)[ND]) {
        if constexpr (std::is_same<T, _Float16>::value) {
            float big = 0.0f;
#pragma unroll
            for (int i = 0; i < 16; ++i) big = fmaxf(big, fabsf(ds[i]));
            big = column_max(big);
            if (__any(big > limit)) {
                const int e = (int)(__float_as_uint(big) >> 23);   // exponent and 127
                const float to = __uint_as_float((uint32_t)min(254 + 8 - e, 254) << 23);
                const bool raise = big > limit;
                const float change = up == 0.0f ? 0.0f : to / up;
                if (raise) {
                    up = to;
                    limit = 32768.0f / to;
                }
#pragma unroll
                for (int d = 0; d < ND; ++d)
#pragma unroll
                    for (int i = 0; i < 16; ++i) acc[d][i] *= raise ? change : 1.0f;
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) ds[i] *= up;
        }
    }
    __device__ __forceinline__ float down() const {
        if constexpr (std::is_same<T, _Float16>::value) return up == 0.0f ? 0.0f : 1.0f / up;
        return 1.0f;
    }
};

}  // namespace da
