// Attention, forward.  Contract and formulas: include/attention.h; tiles and products:
// attn_device.h.
//
// Columns are rows of queries, keys and values are streamed.  One pass with a running maximum:
// of a tile's scores s (keys by queries) a column keeps its maximum m and
// sum l, its weights are 2^(s scale / log 2 - m), and the result, [numbers, queries], is scaled
// again only when a maximum grows by more than 2^8, which is rare after the first tiles and
// costs no digits in binary32.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "attn_device.h"

namespace da {
namespace {

// In binary16 weights lie at 2^7 below the running maximum's, up to 2^15, so that small ones
// keep their digits.
template <typename T>
constexpr float kLiftLog2 = std::is_same<T, _Float16>::value ? 7.0f : 0.0f;
constexpr float kGrowth = 8.0f;

// Waves to a SIMD that the registers leave room for.
template <typename T, int DP, bool DEEP>
constexpr int kForwardWaves = DEEP || sizeof(T) == 4 ? 1 : 2;

template <typename T, int DP, bool DEEP>
__global__ __launch_bounds__(kAttnThreads, (kForwardWaves<T, DP, DEEP>))
void attn_forward_kernel(AttnArgs a) {
    constexpr int TILE = DEEP ? kAttnDeepTile : kAttnWideTile, NB = DEEP ? 1 : 2, ND = DP / 32;
    using Tl = Tile<T, DP, TILE>;
    constexpr bool TWICE = Tl::kPieces * 16 * 4 <= 128 * 1024;   // room for the next tile
    // arrays of their own: the compiler then sees that what is filled is not what is read
    __shared__ u32x4 k0[Tl::kPieces], v0[Tl::kPieces];
    __shared__ u32x4 k1[TWICE ? Tl::kPieces : 1], v1[TWICE ? Tl::kPieces : 1];
    const Spot spot = spot_of(a);
    if (!spot.there) return;
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int col = lane % 32, half = lane / 32;
    const int b = spot.unit / a.Hk, hk = spot.unit % a.Hk;
    const int all = keys_of(a, b);
    const int first = spot.split * a.split_keys;
    const int keys = min(all - first, a.split_keys);   // of this workgroup; may be none
    const int tiles = keys > 0 ? (keys + TILE - 1) / TILE : 0;

    const int r = spot.tile * (DEEP ? kAttnDeep : kAttnWide) + (DEEP ? 0 : wave * 32) + col;
    const int query = (uint32_t)r / (uint32_t)a.group, head = hk * a.group + (uint32_t)r % (uint32_t)a.group;
    const bool there = r < a.rows;
    u32x4 qc[Tl::kSteps];
    load_column<T, DP>(static_cast<const char*>(a.q) + b * a.q_batch + query * a.q_token + head * a.q_head,
                       there, a.D, half, qc);

    const char* kp = static_cast<const char*>(a.k) + b * a.k_batch + hk * a.k_head + first * a.k_token;
    const char* vp = static_cast<const char*>(a.v) + b * a.v_batch + hk * a.v_head + first * a.v_token;
    const uint8_t* mask = a.mask ? a.mask + (int64_t)b * a.Nk + first : nullptr;
    const Places<T, DP> at(lane);
    const Filler<Tl> filler(threadIdx.x, a.D * (int)sizeof(T));
    MaskBytes<Tl::kWords> bytes;

    const auto fetch = [&](int j, const Visible<Tl::kWords>& vis, u32x4* ks, u32x4* vs) {
        const int rows = min(keys - j * TILE, TILE);
        const auto see = [&](int row) { return !mask || vis(row); };
        filler.run(kp + (int64_t)j * TILE * a.k_token, rows, (uint32_t)a.k_token, ks, wave, see);
        filler.run(vp + (int64_t)j * TILE * a.v_token, rows, (uint32_t)a.v_token, vs, wave, see);
    };
    const auto ahead = [&](int j) {   // the mask of tile j
        bytes.load(mask ? mask + j * TILE : nullptr, keys - j * TILE, lane);
    };

    f32x16 acc[ND];
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[d][i] = 0.0f;
    float top = -kInf, shift = 0.0f, sum = 0.0f;   // the maximum; what exponents are less by
    const float growth = kGrowth / a.scale2;

    const auto step = [&](LdsBytes ks, LdsBytes vs, const Visible<Tl::kWords>& vis) {
        f32x16 s[NB];
        float big = -kInf;
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            const int block = DEEP ? wave : n;
            s[n] = mul_columns<T, DP>(at, ks, block, qc);
            const uint32_t see = vis.block(block);
            if (see != ~0u) {
                const uint32_t mine = see >> (4 * half);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    s[n][i] = mine & (1u << (8 * (i / 4) + i % 4)) ? s[n][i] : -kInf;
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) big = fmaxf(big, s[n][i]);
        }
        big = column_max(big);
        if (__any(big > top + growth)) {
            const float now = fmaxf(top, big);
            const float to = now == -kInf ? 0.0f : fmaf(now, a.scale2, -kLiftLog2<T>);
            const float change = top == -kInf ? 0.0f : __builtin_amdgcn_exp2f(shift - to);
            top = now;
            shift = to;
            sum *= change;
#pragma unroll
            for (int d = 0; d < ND; ++d)
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[d][i] *= change;
        }
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            float part[2] = {0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                s[n][i] = __builtin_amdgcn_exp2f(fmaf(s[n][i], a.scale2, -shift));
                part[i % 2] += s[n][i];
            }
            sum += part[0] + part[1];
            mul_rows<T, DP, DEEP>(at, vs, DEEP ? wave : n, Weights<T, DEEP>(s[n]), acc);
        }
    };

    if (tiles > 0) {
        ahead(0);
        Visible<Tl::kWords> here = bytes.visible(keys, lane);
        if (tiles > 1) ahead(1);
        fetch(0, here, k0, v0);
        tile_barrier();
        int j = 0;
        // tile j from (ks, vs) while tile j + 1 fills (kn, vn)
        const auto turn = [&](u32x4* ks, u32x4* vs, u32x4* kn, u32x4* vn) {
            Visible<Tl::kWords> next = here;
            if (j + 1 < tiles) {
                next = bytes.visible(keys - (j + 1) * TILE, lane);
                if (j + 2 < tiles) ahead(j + 2);
                if constexpr (TWICE) fetch(j + 1, next, kn, vn);
            }
            step((LdsBytes)ks, (LdsBytes)vs, here);
            tile_barrier();
            if constexpr (!TWICE) {
                if (j + 1 < tiles) fetch(j + 1, next, kn, vn);
                tile_barrier();
            }
            here = next;
            return ++j < tiles;
        };
        if constexpr (TWICE) {
            while (turn(k0, v0, k1, v1) && turn(k1, v1, k0, v0)) {}
        } else {
            while (turn(k0, v0, k0, v0)) {}
        }
    }

    sum = column_sum(sum);
    if constexpr (DEEP) {
        // the waves' parts meet at their largest exponent
        float2* stat = reinterpret_cast<float2*>(k0);
        __syncthreads();
        if (half == 0) stat[wave * 32 + col] = make_float2(top == -kInf ? -kInf : shift, sum);
        __syncthreads();
        float most = -kInf, total = 0.0f;
#pragma unroll
        for (int w = 0; w < 4; ++w) most = fmaxf(most, stat[w * 32 + col].x);
        most = most == -kInf ? 0.0f : most;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const float2 s = stat[w * 32 + col];
            total += s.y == 0.0f ? 0.0f : s.y * __builtin_amdgcn_exp2f(s.x - most);
        }
        const float factor = top == -kInf ? 0.0f : __builtin_amdgcn_exp2f(shift - most);
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[d][i] *= factor;
        sum = total;
        shift = most;
        add_waves<ND>(acc, reinterpret_cast<float*>(k0), wave, lane);
        if (wave != 0) return;
    }
    if (!there) return;
    if (a.splits > 1) {
        const int64_t at_row = ((int64_t)spot.split * a.B * a.Hk + spot.unit) * a.rows + r;
        if (half == 0) a.part_stat[at_row] = make_float2(shift, sum);
        store_column<float, ND>(a.part + at_row * a.D, a.D, half, acc, 1.0f);
        return;
    }
    char* out = static_cast<char*>(a.out) + b * a.o_batch + query * a.o_token + head * a.o_head;
    store_column<T, ND>(reinterpret_cast<T*>(out), a.D, half, acc, sum == 0.0f ? 0.0f : 1.0f / sum);
    if (a.lse && half == 0)
        a.lse[((int64_t)b * a.H + head) * a.Nq + query] =
            sum == 0.0f ? -kInf : fmaf(shift, kLn2, logf(sum));
}

// ---- splits of keys joined ---------------------------------------------------------------
//
// `threads` threads to a row, a power of two: the splits' statistics go through LDS, then each
// four numbers of each split are a thread's, whose sums meet in LDS.  All reads of a row are on
// their way at once, since a launch of so little work is bound by their latency (one wave to a
// row, split after split, took 7 us for 12 splits of 8 rows of 64 numbers).
template <typename T>
__global__ __launch_bounds__(kAttnThreads) void attn_join_kernel(AttnArgs a, int threads) {
    __shared__ float2 stat[kAttnThreads];
    __shared__ f32x4 meet[kAttnThreads];
    const int64_t units = (int64_t)a.B * a.Hk, lines = units * a.rows;
    const int t = threadIdx.x % threads, base = threadIdx.x - t;
    const int64_t line = (int64_t)blockIdx.x * (kAttnThreads / threads) + threadIdx.x / threads;
    const bool there = line < lines;
    const int unit = there ? (int)(line / a.rows) : 0, r = there ? (int)(line % a.rows) : 0;
    const int b = unit / a.Hk, hk = unit % a.Hk;
    const int splits = there ? (keys_of(a, b) + a.split_keys - 1) / a.split_keys : 0;   // with keys
    float2 mine = make_float2(-kInf, 0.0f);
    if (t < splits) mine = a.part_stat[t * lines + line];
    if (mine.y == 0.0f) mine.x = -kInf;
    stat[threadIdx.x] = mine;
    // 4 numbers to a thread, threads / vectors of them side by side
    const int vectors = a.D / 4, abreast = threads / vectors, at = t % vectors * 4;
    f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    __syncthreads();
    float most = -kInf, sum = 0.0f;
    for (int s = 0; s < splits; ++s) most = fmaxf(most, stat[base + s].x);
    most = most == -kInf ? 0.0f : most;
    const auto weight = [&](float2 p) { return p.y == 0.0f ? 0.0f : __builtin_amdgcn_exp2f(p.x - most); };
    for (int s = 0; s < splits; ++s) sum = fmaf(stat[base + s].y, weight(stat[base + s]), sum);
    if (t < abreast * vectors) {
#pragma unroll 8
        for (int s = t / vectors; s < splits; s += abreast) {
            const f32x4 p = *reinterpret_cast<const f32x4*>(a.part + (s * lines + line) * a.D + at);
            v += p * weight(stat[base + s]);
        }
    }
    meet[threadIdx.x] = v;
    __syncthreads();
    if (!there || t >= vectors) return;
    for (int i = 1; i < abreast; ++i) v += meet[threadIdx.x + i * vectors];
    const float inverse = sum == 0.0f ? 0.0f : 1.0f / sum;
    const float result[4] = {v[0] * inverse, v[1] * inverse, v[2] * inverse, v[3] * inverse};
    const int query = (uint32_t)r / (uint32_t)a.group, head = hk * a.group + (uint32_t)r % (uint32_t)a.group;
    char* out = static_cast<char*>(a.out) + b * a.o_batch + query * a.o_token + head * a.o_head;
    store_as(reinterpret_cast<T*>(out) + at, result);
    if (a.lse && at == 0)
        a.lse[((int64_t)b * a.H + head) * a.Nq + query] =
            sum == 0.0f ? -kInf : fmaf(most, kLn2, logf(sum));
}

template <typename T, int DP>
void launch(const AttnArgs& a, hipStream_t stream) {
    const uint32_t blocks = (uint32_t)(a.blocks + 7) / 8 * 8;
    if (a.deep)
        attn_forward_kernel<T, DP, true><<<blocks, kAttnThreads, 0, stream>>>(a);
    else
        attn_forward_kernel<T, DP, false><<<blocks, kAttnThreads, 0, stream>>>(a);
}

template <typename T>
hipError_t launch_type(const AttnArgs& a, hipStream_t stream) {
    if (a.D <= 32)
        launch<T, 32>(a, stream);
    else if (a.D <= 64)
        launch<T, 64>(a, stream);
    else if (a.D <= 96)
        launch<T, 96>(a, stream);
    else
        launch<T, 128>(a, stream);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.splits == 1) return e;
    int threads = 8;
    while (threads < kAttnThreads && threads < a.splits * (a.D / 4)) threads *= 2;
    const int64_t rows = (int64_t)a.B * a.Hk * a.rows, per = kAttnThreads / threads;
    attn_join_kernel<T><<<(uint32_t)((rows + per - 1) / per), kAttnThreads, 0, stream>>>(a, threads);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_attn_forward(const AttnArgs& a, hipStream_t stream) {
    if (a.dtype == DA_BF16) return launch_type<__bf16>(a, stream);
    if (a.dtype == DA_F16) return launch_type<_Float16>(a, stream);
    return launch_type<float>(a, stream);
}

}  // namespace da
