// Attention, forward.  Contract and formulas: include/attention.h; tiles and products:
// attn_device.h.
//
// Columns are rows of queries, keys and values are streamed.  One pass with a running maximum:
// of a tile's scores s (keys by queries) a column keeps its maximum m and
// sum l, its weights are 2^(s scale / log 2 - m), and the result, [numbers, queries], is scaled
// again only when a maximum grows by more than 2^8, which is rare after the first tiles and
// costs no digits in binary32.  Where m is so large that its own rounding would count in the
// weights, scores are taken less the largest one before they are scaled (kFar, below).
//
// Many rows: four waves of 32 columns and tiles of 64 keys, the next tile on its way while one is
// used; two workgroups to a compute unit, so that one wave's exponentials run beside another's
// products.  Bound by the matrix instructions: 2 x 4096 rows on 8192 keys, 16 heads of 128, bfloat16,
// 507 us, 1085 Tflop/s, where a product of 8192^3 runs at 1363; the clock falls to about 1.75 GHz
// under this load (on another card further: 544).
#include <float.h>
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

// Maxima from here on, in base 2, are far: m, rounded to binary32, is off by up to 2^-4 there and
// by 2^7 at 2^32, where weights would be infinite or 0.  A wave that meets one takes its scores less
// their column's largest from then on, which is exact where it matters; the others pay a
// comparison when a maximum grows and a branch for each tile (one token on 1500 keys 9.8 -> 10.1
// us, 2 x 4096 rows on 8192 keys 503 -> 507).
constexpr float kFar = 0x1p20f;

// A column's running maximum and sum, and what exponents are less by.
struct Running {
    float top = -kInf, shift = 0.0f, sum = 0.0f;
    bool far = false;    // of the wave; shift is then -kLiftLog2 alone
    // Scores of NB blocks become weights, 2^(s scale2 - shift), far ones 2^((s - top) scale2 - shift),
    // after the results so far are scaled to a new maximum where one has grown.
    template <typename T, int NB, int ND>
    __device__ __forceinline__ void weigh(f32x16 (&s)[NB], f32x16 (&acc)[ND], float scale2, float growth) {
        float big = -kInf;
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int i = 0; i < 16; ++i) big = fmaxf(big, s[n][i]);
        big = column_max(big);
        // (a unit of a far maximum's last place may be more than `growth`)
        if (__any(big > top + (far ? 0.0f : growth))) {
            const float now = fmaxf(top, big);
            float to = now == -kInf ? 0.0f : fmaf(now, scale2, -kLiftLog2<T>), less = shift - to;
            if (__builtin_expect(far || __any(fabsf(to) >= kFar), false)) {
                less = far ? (top - now) * scale2 : kLiftLog2<T> - fmaf(now, scale2, -shift);
                to = now == -kInf ? 0.0f : -kLiftLog2<T>;
                far = true;
            }
            const float change = top == -kInf ? 0.0f : __builtin_amdgcn_exp2f(less);
            top = now;
            shift = to;
            sum *= change;
#pragma unroll
            for (int d = 0; d < ND; ++d)
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[d][i] *= change;
        }
        if (__builtin_expect(far, false)) {
            const float base = top == -kInf ? 0.0f : top;
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int i = 0; i < 16; ++i) s[n][i] -= base;
        }
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            float part[2] = {0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                s[n][i] = __builtin_amdgcn_exp2f(fmaf(s[n][i], scale2, -shift));
                part[i % 2] += s[n][i];
            }
            sum += part[0] + part[1];
        }
    }
    // What is kept of a column whose weights add up to `all` and that others' parts join.
    __device__ __forceinline__ float2 part(float all) const {
        if (top == -kInf) return make_float2(-kInf, all);
        return far ? make_float2(top, -all) : make_float2(shift, all);
    }
};

// Parts of a column that meet, each (shift, sum) or, of a far one, (top, -sum): the largest of what
// they are less by, or, if one is far, their largest score, and what each counts for.
template <typename T>
struct Meet {
    float most = -kInf;
    bool far = false;
    // `at(n)` is the n-th part of `count`
    template <class At>
    __device__ __forceinline__ Meet(int count, At at, float scale2) {
        float least = 0.0f;
#pragma unroll
        for (int n = 0; n < count; ++n) {
            most = fmaxf(most, at(n).x);
            least = fminf(least, at(n).y);
        }
        if (__builtin_expect(least < 0.0f, false)) {
            far = true;
            most = -kInf;
            for (int n = 0; n < count; ++n) {
                const float2 p = at(n);
                const float score = p.y < 0.0f || p.x == -kInf ? p.x : (p.x + kLiftLog2<T>) / scale2;
                most = fmaxf(most, p.y < 0.0f ? score : fminf(score, FLT_MAX));
            }
        }
        most = most == -kInf ? 0.0f : most;
    }
    __device__ __forceinline__ float share(float2 p, float scale2) const {
        if (p.x == -kInf) return 0.0f;
        float e = p.x - most;
        if (__builtin_expect(far, false)) e = p.y < 0.0f ? e * scale2 : kLiftLog2<T> - fmaf(most, scale2, -p.x);
        return __builtin_amdgcn_exp2f(e);
    }
    __device__ __forceinline__ float lse(float sum, float scale2) const {
        return sum == 0.0f ? -kInf : fmaf(far ? fmaf(most, scale2, -kLiftLog2<T>) : most, kLn2, logf(sum));
    }
};

template <int ND>
__device__ __forceinline__ void clear(f32x16 (&acc)[ND]) {
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[d][i] = 0.0f;
}

// Waves to a SIMD that the registers leave room for.
template <typename T>
constexpr int kForwardWaves = sizeof(T) == 4 ? 1 : 2;

template <typename T, int DP, bool MASK>
__global__ __launch_bounds__(kAttnThreads, kForwardWaves<T>) void attn_forward_kernel(AttnArgs a) {
    constexpr int TILE = kAttnTile, NB = TILE / 32, ND = DP / 32;
    using Tl = Tile<T, DP, TILE>;
    // arrays of their own: the compiler then sees that what is filled is not what is read
    __shared__ u32x4 k0[Tl::kPieces], v0[Tl::kPieces], k1[Tl::kPieces], v1[Tl::kPieces];
    const Spot spot = spot_of(a, blockIdx.x, gridDim.x);
    if (!spot.there) return;
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int col = lane % 32, half = lane / 32;
    const int b = spot.unit / a.Hk, hk = spot.unit % a.Hk;
    const int first = spot.split * a.split_keys;
    const int keys = min(keys_of(a, b) - first, a.split_keys);   // of this split; may be none
    const int tiles = keys > 0 ? (keys + TILE - 1) / TILE : 0;

    const int r = spot.tile * kAttnWide + wave * 32 + col;
    const int query = (uint32_t)r / (uint32_t)a.group, head = hk * a.group + (uint32_t)r % (uint32_t)a.group;
    const bool there = r < a.rows;
    u32x4 qc[Tl::kSteps];
    load_column<T, DP>(static_cast<const char*>(a.q) + b * a.q_batch + query * a.q_token + head * a.q_head,
                       there, a.D, half, qc);

    const char* kp = static_cast<const char*>(a.k) + b * a.k_batch + hk * a.k_head + first * a.k_token;
    const char* vp = static_cast<const char*>(a.v) + b * a.v_batch + hk * a.v_head + first * a.v_token;
    const uint8_t* mask = MASK ? a.mask + (int64_t)b * a.Nk + first : nullptr;
    const Places<T, DP> at(lane);
    const Filler<Tl> filler(threadIdx.x, a.D * (int)sizeof(T));
    uint32_t byte = 1;   // of the tile that is fetched next

    u32x4 *const kt[2] = {k0, k1}, *const vt[2] = {v0, v1};
    Visible visible_keys[2];
    int tile = 0;
    // Fetches the next tile, or zeros past the last, and reads the mask of the one after it.
    const auto fetch = [&](auto i) {
        const int rows = min(keys - tile * TILE, TILE);
        const Visible vis = visible(byte, rows, lane);
        if constexpr (MASK) byte = mask_byte(mask + (int64_t)(tile + 1) * TILE, keys - (tile + 1) * TILE, lane);
        filler.template run<MASK>(kp + (int64_t)tile * TILE * a.k_token, rows, (uint32_t)a.k_token, kt[i], wave, vis);
        filler.template run<MASK>(vp + (int64_t)tile * TILE * a.v_token, rows, (uint32_t)a.v_token, vt[i], wave, vis);
        visible_keys[i] = vis;
        ++tile;
    };

    f32x16 acc[ND];
    clear(acc);
    Running run;
    const float growth = fminf(kGrowth / a.scale2, FLT_MAX);   // finite: added to -infinity
    const auto step = [&](auto buffer) {
        const LdsBytes ks = (LdsBytes)kt[buffer], vs = (LdsBytes)vt[buffer];
        const Visible vis = visible_keys[buffer];
        f32x16 s[NB];
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            s[n] = mul_columns<T, DP>(at, ks, n, qc);
            hide(s[n], vis.block(n), -kInf);
        }
        run.weigh<T>(s, acc, a.scale2, growth);
#pragma unroll
        for (int n = 0; n < NB; ++n)
            mul_rows<T, DP, false>(at, vs, n, Weights<T, false>(s[n]), acc);
    };

    if constexpr (MASK) byte = mask_byte(mask, keys, lane);
    walk(tiles, fetch, step, [](auto) {});

    const float sum = column_sum(run.sum);
    if (!there) return;
    if (a.splits > 1) {
        const int64_t line = ((int64_t)spot.split * a.B * a.Hk + spot.unit) * a.rows + r;
        if (half == 0) a.part_stat[line] = run.part(sum);
        store_column<float, ND>(a.part + line * a.D, a.D, half, acc, 1.0f);
        return;
    }
    char* out = static_cast<char*>(a.out) + b * a.o_batch + query * a.o_token + head * a.o_head;
    store_column<T, ND>(reinterpret_cast<T*>(out), a.D, half, acc, sum == 0.0f ? 0.0f : 1.0f / sum);
    if (a.lse && half == 0) {
        const float less = run.far ? fmaf(run.top, a.scale2, -kLiftLog2<T>) : run.shift;
        a.lse[((int64_t)b * a.H + head) * a.Nq + query] = sum == 0.0f ? -kInf : fmaf(less, kLn2, logf(sum));
    }
}

// ---- few rows ----------------------------------------------------------------------------
//
// All waves have the same 32 rows, and every so many blocks of 32 keys are a wave's, in tiles of its
// own, so that no wave waits for another until their results meet at the end.  Bound by the
// states' way from memory on long caches (16 entries of one token, 32 heads of 128 on 8 with up to
// 16384 keys, bfloat16: 152 us, 4.8 TB/s, where a copy runs at 5.1), by latency on short ones (8 heads
// of 64 on 1500 keys: 11 us).  One step of all waves together, with barriers, took 182 and 17.
template <typename T, int DP>
__global__ __launch_bounds__(64 * attn_few_waves(DP * (int)sizeof(T)))
void attn_few_kernel(AttnArgs a) {
    constexpr int WAVES = attn_few_waves(DP * (int)sizeof(T)), ND = DP / 32;
    constexpr bool LOW = sizeof(T) == 2;
    using Tl = Tile<T, DP, 32, 64>;
    constexpr bool TWICE = WAVES * Tl::kPieces * 16 * 4 <= 128 * 1024;   // room for the next tile
    constexpr int kMore = TWICE ? WAVES * Tl::kPieces : 1;
    __shared__ u32x4 k0[WAVES * Tl::kPieces], v0[WAVES * Tl::kPieces], k1[kMore], v1[kMore];
    __shared__ float2 stat[WAVES * 32];
    const Spot spot = spot_of(a, blockIdx.x, gridDim.x);
    if (!spot.there) return;
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int col = lane % 32, half = lane / 32;
    const int b = spot.unit / a.Hk, hk = spot.unit % a.Hk;
    const int first = spot.split * a.split_keys + wave * 32;
    const int keys = min(keys_of(a, b), (spot.split + 1) * a.split_keys) - first;   // from the wave's first
    const int tiles = keys > 0 ? (keys + WAVES * 32 - 1) / (WAVES * 32) : 0;

    const int r0 = spot.tile * kAttnFew, r = r0 + col;
    const bool there = r < a.rows;
    u32x4 qc[Tl::kSteps];
    {
        const int query = (uint32_t)r / (uint32_t)a.group;
        const int head = hk * a.group + (uint32_t)r % (uint32_t)a.group;
        load_column<T, DP>(static_cast<const char*>(a.q) + b * a.q_batch + query * a.q_token +
                               head * a.q_head,
                           there, a.D, half, qc);
    }
    const char* kp = static_cast<const char*>(a.k) + b * a.k_batch + hk * a.k_head + first * a.k_token;
    const char* vp = static_cast<const char*>(a.v) + b * a.v_batch + hk * a.v_head + first * a.v_token;
    const uint8_t* mask = a.mask ? a.mask + (int64_t)b * a.Nk + first : nullptr;
    const Places<T, DP> at(lane);
    const Filler<Tl> filler(lane, a.D * (int)sizeof(T));
    uint32_t byte = 1;

    const auto left = [&](int j) { return min(keys - j * WAVES * 32, 32); };
    const auto fetch = [&](int j, const Visible& vis, u32x4* ks, u32x4* vs) {
        const int64_t row = (int64_t)j * WAVES * 32;
        if (mask) {
            filler.template run<true>(kp + row * a.k_token, left(j), (uint32_t)a.k_token, ks, 0, vis);
            filler.template run<true>(vp + row * a.v_token, left(j), (uint32_t)a.v_token, vs, 0, vis);
        } else {
            filler.template run<false>(kp + row * a.k_token, left(j), (uint32_t)a.k_token, ks, 0, vis);
            filler.template run<false>(vp + row * a.v_token, left(j), (uint32_t)a.v_token, vs, 0, vis);
        }
    };
    const auto ahead = [&](int j) {
        if (mask) byte = mask_byte(mask + (int64_t)j * WAVES * 32, left(j), lane);
    };

    f32x16 acc[ND];
    clear(acc);
    Running run;
    const float growth = fminf(kGrowth / a.scale2, FLT_MAX);   // finite: added to -infinity
    const auto step = [&](LdsBytes ks, LdsBytes vs, const Visible& vis) {
        f32x16 s[1] = {mul_columns<T, DP>(at, ks, 0, qc)};
        hide(s[0], vis.block(0), -kInf);
        run.weigh<T>(s, acc, a.scale2, growth);
        mul_rows<T, DP, LOW>(at, vs, 0, Weights<T, LOW>(s[0]), acc);
    };

    if (tiles > 0) {
        u32x4 *ka = k0 + wave * Tl::kPieces, *va = v0 + wave * Tl::kPieces;
        u32x4 *kb = TWICE ? k1 + wave * Tl::kPieces : ka, *vb = TWICE ? v1 + wave * Tl::kPieces : va;
        ahead(0);
        Visible here = visible(byte, left(0), lane);
        if (tiles > 1) ahead(1);
        fetch(0, here, ka, va);
        own_fills();
        int j = 0;
        const auto turn = [&](u32x4* ks, u32x4* vs, u32x4* kn, u32x4* vn) {
            Visible next = here;
            if (j + 1 < tiles) {
                next = visible(byte, left(j + 1), lane);
                if (j + 2 < tiles) ahead(j + 2);
                if constexpr (TWICE) fetch(j + 1, next, kn, vn);
            }
            step((LdsBytes)ks, (LdsBytes)vs, here);
            if constexpr (!TWICE) {
                own_fills();   // and its reads: the tile is filled again
                if (j + 1 < tiles) fetch(j + 1, next, kn, vn);
            }
            own_fills();
            here = next;
            return ++j < tiles;
        };
        while (turn(ka, va, kb, vb) && turn(kb, vb, ka, va)) {}
    }

    // The waves' parts meet.  A wave's place has DP numbers to a column, in
    // fours, turned by the column so that 32 columns' equal fours spread over the banks.
    const float part = column_sum(run.sum);
    __syncthreads();
    if (half == 0) stat[wave * 32 + col] = run.part(part);
    constexpr int kFours = DP / 4, kPlace = 32 * kFours;   // of 16 bytes
    constexpr int kHere = WAVES * Tl::kPieces / kPlace;    // waves that k0 has room for
    static_assert(2 * kHere >= WAVES, "k0 and v0 hold every wave's part");
    const auto place = [&](int w) {
        return reinterpret_cast<f32x4*>(w < kHere ? k0 : v0) + (w < kHere ? w : w - kHere) * kPlace;
    };
    if (there) {
        f32x4* to = place(wave) + col * kFours;
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                to[(d * 8 + j * 2 + half) ^ (col & 7)] =
                    f32x4{acc[d][4 * j], acc[d][4 * j + 1], acc[d][4 * j + 2], acc[d][4 * j + 3]};
    }
    __syncthreads();
    const int rows = min(a.rows - r0, kAttnFew), vectors = a.D / 4;
    for (int n = threadIdx.x; n < rows * vectors; n += 64 * WAVES) {
        const int c = n / vectors, v = n % vectors;
        const Meet<T> meet(WAVES, [&](int w) { return stat[w * 32 + c]; }, a.scale2);
        float sum = 0.0f;
        f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            const float2 s = stat[w * 32 + c];
            const float f = meet.share(s, a.scale2);
            sum = fmaf(fabsf(s.y), f, sum);
            x += place(w)[c * kFours + (v ^ (c & 7))] * f;
        }
        const int row = r0 + c;
        if (a.splits > 1) {
            const int64_t line = ((int64_t)spot.split * a.B * a.Hk + spot.unit) * a.rows + row;
            if (v == 0) a.part_stat[line] = make_float2(meet.most, meet.far ? -sum : sum);
            *reinterpret_cast<f32x4*>(a.part + line * a.D + v * 4) = x;
            continue;
        }
        const int query = (uint32_t)row / (uint32_t)a.group;
        const int head = hk * a.group + (uint32_t)row % (uint32_t)a.group;
        const float inverse = sum == 0.0f ? 0.0f : 1.0f / sum;
        const float result[4] = {x[0] * inverse, x[1] * inverse, x[2] * inverse, x[3] * inverse};
        char* out = static_cast<char*>(a.out) + b * a.o_batch + query * a.o_token + head * a.o_head;
        store_as(reinterpret_cast<T*>(out) + v * 4, result);
        if (a.lse && v == 0) a.lse[((int64_t)b * a.H + head) * a.Nq + query] = meet.lse(sum, a.scale2);
    }
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
    __shared__ f32x4 fours[kAttnThreads];
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
    const Meet<T> meet(splits, [&](int s) { return stat[base + s]; }, a.scale2);
    const auto share = [&](int s) { return meet.share(stat[base + s], a.scale2); };
    float sum = 0.0f;
    for (int s = 0; s < splits; ++s) sum = fmaf(fabsf(stat[base + s].y), share(s), sum);
    if (t < abreast * vectors) {
#pragma unroll 8
        for (int s = t / vectors; s < splits; s += abreast) {
            const f32x4 p = *reinterpret_cast<const f32x4*>(a.part + (s * lines + line) * a.D + at);
            v += p * share(s);
        }
    }
    fours[threadIdx.x] = v;
    __syncthreads();
    if (!there || t >= vectors) return;
    for (int i = 1; i < abreast; ++i) v += fours[threadIdx.x + i * vectors];
    const float inverse = sum == 0.0f ? 0.0f : 1.0f / sum;
    const float result[4] = {v[0] * inverse, v[1] * inverse, v[2] * inverse, v[3] * inverse};
    const int query = (uint32_t)r / (uint32_t)a.group, head = hk * a.group + (uint32_t)r % (uint32_t)a.group;
    char* out = static_cast<char*>(a.out) + b * a.o_batch + query * a.o_token + head * a.o_head;
    store_as(reinterpret_cast<T*>(out) + at, result);
    if (a.lse && at == 0)
        a.lse[((int64_t)b * a.H + head) * a.Nq + query] = meet.lse(sum, a.scale2);
}

template <typename T, int DP>
void launch(const AttnArgs& a, hipStream_t stream) {
    const uint32_t blocks = (uint32_t)(a.blocks + 7) / 8 * 8;
    if (a.few)
        attn_few_kernel<T, DP>
            <<<blocks, 64 * attn_few_waves(DP * (int)sizeof(T)), 0, stream>>>(a);
    else if (a.mask)
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
