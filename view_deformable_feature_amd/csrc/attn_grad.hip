// Attention's gradients.  Contract and formulas: include/attention.h; tiles and products:
// attn_device.h.
//
// Two kinds of workgroups, both in one launch, so that the one's fill the compute units that the
// other's leave (6 x 900 queries on up to 1201 keys, 8 heads of 64, binary16: 42 and 42 us apart, 78
// in one; with three waves to a SIMD, which heads of 64 numbers have room for, 62).
//
// The queries' gradients: as in the forward, columns are rows of queries and keys and values are
// streamed; a column's lse and delta are a register each.  Three products to a tile: scores, dP, and
// keys times dS.
//
// The keys' and values': columns are keys, and the queries and gradients of every head that reads
// them are streamed, so that the heads' sum forms in the accumulators.  Four products to a tile:
// scores, dP, the gradients times p, and the queries times dS.  An invisible key's column runs
// along and is written as zeros.
//
// Two waves to a SIMD, and the loops have no branches of their own: with branches the accumulators
// moved between registers at each of them, and heads of 128 numbers had room for one wave
// (1 x 4096 on 4096, 16 heads of 128 on 4, bfloat16: 694 us, 475 so, 450 to 463 now by the card).
// Bound by the matrix instructions, at 743 to 763 Tflop/s of five products' worth, with the scores'
// and dP's products formed twice, once by either kind: at 1040 to 1070 of the seven that run.  What the scores' exponentials and the
// roundings of p and dS cost lies in their shadow only in part.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "attn_device.h"

namespace da {
namespace {

// In binary16 p lies at 2^15, the largest power that its range holds, where it multiplies the
// gradients.
template <typename T>
constexpr float kLiftLog2 = std::is_same<T, _Float16>::value ? 15.0f : 0.0f;

template <typename T, int DP>
constexpr int kGradWaves = sizeof(T) * DP > 256   ? 1   // to a SIMD, whose registers they share
                           : sizeof(T) * DP > 128 ? 2
                           : sizeof(T) * DP > 64  ? 3
                                                  : 4;

// In 16-bit types dP's product begins with -delta, which saves a subtraction for each score; its
// roundings, of delta's size too then, are far below those of dS (4 x 2048 on 2048, 16 heads of 64,
// bfloat16: 266 us, 255 so).  In binary32 they would not be, and for the keys of wide heads the
// registers do not reach.
template <typename T, int DP>
constexpr bool kKeysFromDelta = sizeof(T) == 2 && DP <= 96;

constexpr int TILE = kAttnTile, NB = TILE / 32;

// A lane's 16 of a tile's statistics, by the rows of a block's results, in fours.
__device__ __forceinline__ f32x4 stats_at(const float* stat, int block, int four, int half) {
    return *reinterpret_cast<const f32x4*>(stat + block * 32 + 8 * four + 4 * half);
}
__device__ __forceinline__ f32x16 stats_of(const float* stat, int block, int half) {
    f32x16 x;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const f32x4 four = stats_at(stat, block, j, half);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[4 * j + e] = four[e];
    }
    return x;
}

// A workgroup's part of LDS, by the buffer: tiles of two tensors, and of the second one's rows what
// exponents are more by, and -delta.
struct Shared {
    u32x4 *a[2], *b[2];
    float* stat[2];
};

template <typename T, int DP, bool MASK>
__device__ __forceinline__ void grad_q(const AttnArgs& a, int block, int blocks, const Shared& t) {
    constexpr int ND = DP / 32;
    using Tl = Tile<T, DP, TILE>;
    const Spot spot = spot_of(a, block, blocks);
    if (!spot.there) return;
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int col = lane % 32, half = lane / 32;
    const int b = spot.unit / a.Hk, hk = spot.unit % a.Hk;
    const int first = spot.split * a.split_keys * TILE;
    const int keys = min(keys_of(a, b) - first, a.split_keys * TILE);   // of this split; may be none
    const int tiles = keys > 0 ? (keys + TILE - 1) / TILE : 0;

    const int r = spot.tile * kAttnWide + wave * 32 + col;
    const int query = (uint32_t)r / (uint32_t)a.group, head = hk * a.group + (uint32_t)r % (uint32_t)a.group;
    const bool there = r < a.rows;
    const int64_t line = ((int64_t)b * a.Nq + query) * a.H + head;
    u32x4 qc[Tl::kSteps], gc[Tl::kSteps];
    load_column<T, DP>(static_cast<const char*>(a.q) + b * a.q_batch + query * a.q_token + head * a.q_head,
                       there, a.D, half, qc);
    load_column<T, DP>(static_cast<const char*>(a.grad_out) + b * a.g_batch + query * a.g_token +
                           head * a.g_head,
                       there, a.D, half, gc);
    const int64_t stat = ((int64_t)b * a.H + head) * a.Nq + query;
    const float lse2 = there ? a.lse2[stat] : kInf, delta = there ? a.delta[stat] : 0.0f;

    const char* kp = static_cast<const char*>(a.k) + b * a.k_batch + hk * a.k_head + first * a.k_token;
    const char* vp = static_cast<const char*>(a.v) + b * a.v_batch + hk * a.v_head + first * a.v_token;
    const uint8_t* mask = MASK ? a.mask + (int64_t)b * a.Nk + first : nullptr;
    const Places<T, DP> at(lane);
    const Filler<Tl> filler(threadIdx.x, a.D * (int)sizeof(T));
    uint32_t byte = 1;   // of the tile that is fetched next

    // Fetches the next tile, or zeros past the last, and reads the mask of the one after it.
    Visible visible_keys[2];
    int tile = 0;
    const auto fetch = [&](auto i) {
        const int rows = min(keys - tile * TILE, TILE);
        const Visible vis = visible(byte, rows, lane);
        if constexpr (MASK) byte = mask_byte(mask + (int64_t)(tile + 1) * TILE, keys - (tile + 1) * TILE, lane);
        filler.template run<MASK>(kp + (int64_t)tile * TILE * a.k_token, rows, (uint32_t)a.k_token, t.a[i], wave, vis);
        filler.template run<MASK>(vp + (int64_t)tile * TILE * a.v_token, rows, (uint32_t)a.v_token, t.b[i], wave, vis);
        visible_keys[i] = vis;
        ++tile;
    };

    f32x16 acc[ND];
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[d][i] = 0.0f;
    Lift<T, ND> lift;

    const auto step = [&](auto buffer) {
        const LdsBytes ks = (LdsBytes)t.a[buffer], vs = (LdsBytes)t.b[buffer];
        const Visible vis = visible_keys[buffer];
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            f32x16 s = mul_columns<T, DP>(at, ks, n, qc);
            f32x16 dp;
            if constexpr (sizeof(T) == 2) {
                dp = mul_columns<T, DP>(at, vs, n, gc, all_equal(-delta));
            } else {
                dp = mul_columns<T, DP>(at, vs, n, gc);
#pragma unroll
                for (int i = 0; i < 16; ++i) dp[i] -= delta;
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) s[i] = __builtin_amdgcn_exp2f(fmaf(s[i], a.scale2, -lse2)) * dp[i];
            hide(s, vis.block(n), 0.0f);
            lift.apply(s, acc);
            mul_rows<T, DP, false>(at, ks, n, Weights<T, false>(s), acc);
        }
    };

    if constexpr (MASK) byte = mask_byte(mask, keys, lane);
    walk(tiles, fetch, step, [](auto) {});

    if (!there) return;
    const float factor = a.scale * lift.down();
    if (a.splits > 1)
        store_column<float, ND>(a.part + (spot.split * (int64_t)a.B * a.Nq * a.H + line) * a.D, a.D, half,
                                acc, factor);
    else
        store_column<T, ND>(static_cast<T*>(a.grad_q) + line * a.D, a.D, half, acc, factor);
}

template <typename T, int DP>
__device__ __forceinline__ void grad_kv(const AttnArgs& a, int block, int blocks, const Shared& t) {
    constexpr int ND = DP / 32;
    using Tl = Tile<T, DP, TILE>;
    const Spot spot = spot_of(a, block, blocks);
    if (!spot.there) return;
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int col = lane % 32, half = lane / 32;
    const int b = spot.unit / a.Hk, hk = spot.unit % a.Hk;
    const int keys = keys_of(a, b);
    const int first = spot.tile * kAttnWide;
    const int per_head = (a.Nq + TILE - 1) / TILE, from = spot.split * a.split_keys;
    const int tiles = first < keys ? min(per_head * a.group - from, a.split_keys) : 0;

    const int key = first + wave * 32 + col;
    const bool there = key < a.Nk;
    bool seen = key < keys;
    if (a.mask && seen) seen = a.mask[(int64_t)b * a.Nk + key] != 0;
    u32x4 kc[Tl::kSteps], vc[Tl::kSteps];
    load_column<T, DP>(static_cast<const char*>(a.k) + b * a.k_batch + key * a.k_token + hk * a.k_head,
                       seen, a.D, half, kc);
    load_column<T, DP>(static_cast<const char*>(a.v) + b * a.v_batch + key * a.v_token + hk * a.v_head,
                       seen, a.D, half, vc);

    const char* qp = static_cast<const char*>(a.q) + b * a.q_batch + (int64_t)hk * a.group * a.q_head;
    const char* gp = static_cast<const char*>(a.grad_out) + b * a.g_batch +
                     (int64_t)hk * a.group * a.g_head;
    const int64_t stats = ((int64_t)b * a.H + hk * a.group) * a.Nq;
    const Places<T, DP> at(lane);
    const Filler<Tl> filler(threadIdx.x, a.D * (int)sizeof(T));

    // of the tile that is fetched next
    int head = a.Nq ? from / per_head : 0, row = a.Nq ? from % per_head * TILE : 0;
    float mine = 0.0f;       // a thread's part of its statistics
    const Visible none = {0};
    // Fetches the next tile, or zeros past the last.
    const auto fetch = [&](auto i) {
        const int rows = head < a.group ? min(a.Nq - row, TILE) : 0;
        const int at_row = threadIdx.x % TILE;
        // past the last row p is 0
        mine = threadIdx.x < TILE ? kInf : 0.0f;
        if (threadIdx.x < 2 * TILE && at_row < rows)
            mine = (threadIdx.x < TILE ? a.lse2 : a.delta)[stats + (int64_t)head * a.Nq + row + at_row];
        filler.template run<false>(qp + head * a.q_head + row * a.q_token, rows, (uint32_t)a.q_token, t.a[i], wave, none);
        filler.template run<false>(gp + head * a.g_head + row * a.g_token, rows, (uint32_t)a.g_token, t.b[i], wave, none);
        row += TILE;
        if (row >= a.Nq) {
            row = 0;
            ++head;
        }
    };
    // At the end of a step, when they have arrived: what is done with them waits for the fills too.
    const auto keep = [&](auto i) {
        if (threadIdx.x < 2 * TILE) t.stat[i][threadIdx.x] = (threadIdx.x < TILE ? kLiftLog2<T> : 0.0f) - mine;
    };

    f32x16 dk[ND], dv[ND];
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) dk[d][i] = dv[d][i] = 0.0f;
    Lift<T, ND> lift;

    const auto step = [&](auto buffer) {
        const LdsBytes qs = (LdsBytes)t.a[buffer], gs = (LdsBytes)t.b[buffer];
        const float* stat = t.stat[buffer];
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            f32x16 p = mul_columns<T, DP>(at, qs, n, kc);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const f32x4 more = stats_at(stat, n, j, half);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    p[4 * j + e] = __builtin_amdgcn_exp2f(fmaf(p[4 * j + e], a.scale2, more[e]));
            }
            mul_rows<T, DP, false>(at, gs, n, Weights<T, false>(p), dv);
            f32x16 ds;
            if constexpr (kKeysFromDelta<T, DP>) {
                ds = mul_columns<T, DP>(at, gs, n, vc, stats_of(stat + TILE, n, half));
#pragma unroll
                for (int i = 0; i < 16; ++i) ds[i] *= p[i];
            } else {
                ds = mul_columns<T, DP>(at, gs, n, vc);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const f32x4 less = stats_at(stat + TILE, n, j, half);
#pragma unroll
                    for (int e = 0; e < 4; ++e) ds[4 * j + e] = p[4 * j + e] * (ds[4 * j + e] + less[e]);
                }
            }
            lift.apply(ds, dk);
            mul_rows<T, DP, false>(at, qs, n, Weights<T, false>(ds), dk);
        }
    };

    walk(tiles, fetch, step, keep);

    const float back = std::is_same<T, _Float16>::value ? 1.0f / 32768.0f : 1.0f;
    const float fk = a.scale * lift.down() * back, fv = back;
    if (!there) return;
    if (!seen) {
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i) dk[d][i] = dv[d][i] = 0.0f;
    }
    const int64_t line = ((int64_t)b * a.Nk + key) * a.Hk + hk;
    if (a.splits > 1) {
        const int64_t at_line = (spot.split * (int64_t)a.B * a.Nk * a.Hk + line) * a.D;
        store_column<float, ND>(a.part_k + at_line, a.D, half, dk, fk);
        store_column<float, ND>(a.part_v + at_line, a.D, half, dv, fv);
        return;
    }
    store_column<T, ND>(static_cast<T*>(a.grad_k) + line * a.D, a.D, half, dk, fk);
    store_column<T, ND>(static_cast<T*>(a.grad_v) + line * a.D, a.D, half, dv, fv);
}

template <typename T, int DP, bool MASK>
__global__ __launch_bounds__(kAttnThreads)
__attribute__((amdgpu_waves_per_eu(kGradWaves<T, DP>, kGradWaves<T, DP>)))
void attn_grad_kernel(AttnArgs of_q, AttnArgs of_kv, int q_blocks) {
    using Tl = Tile<T, DP, TILE>;
    // arrays of their own: the compiler then sees that what is filled is not what is read
    __shared__ u32x4 a0[Tl::kPieces], b0[Tl::kPieces], a1[Tl::kPieces], b1[Tl::kPieces];
    __shared__ __align__(16) float stat0[2 * TILE], stat1[2 * TILE];
    const Shared t = {{a0, a1}, {b0, b1}, {stat0, stat1}};
    if ((int)blockIdx.x < q_blocks)
        grad_q<T, DP, MASK>(of_q, blockIdx.x, q_blocks, t);
    else
        grad_kv<T, DP>(of_kv, blockIdx.x - q_blocks, gridDim.x - q_blocks, t);
}

// ---- lse in base 2, and delta ------------------------------------------------------------
//
// Eight lanes to a row of out and grad_out, a run of 16-byte pieces in turn to each.  Workgroups walk
// over the rows where there are more than a launch has threads for.
//
// On its way from the scores lse is rounded three times, here the last one, by u = 2^-24 of itself
// each, so that a p that is 1 comes out as 2^(+-3 u |lse2|).  From 2^22 on that could pass what
// binary16 holds, and later be infinite: there lse2 is raised by 4 u of itself (one more for this
// rounding), and no p passes 1.
constexpr float kFarLse = 0x1p22f;

template <typename T>
__global__ __launch_bounds__(kAttnThreads) void attn_delta_kernel(AttnArgs a) {
    constexpr int V = 16 / (int)sizeof(T), kRows = kAttnThreads / 8;
    const int part = threadIdx.x % 8;
    const int64_t lines = (int64_t)a.B * a.Nq * a.H;
    for (int64_t line = (int64_t)blockIdx.x * kRows + threadIdx.x / 8; line < lines;
         line += (int64_t)gridDim.x * kRows) {
        const int64_t bq = line / a.H, b = bq / a.Nq, query = bq % a.Nq;
        const int head = (int)(line % a.H);
        const T* o = reinterpret_cast<const T*>(static_cast<const char*>(a.out) + b * a.o_batch +
                                                query * a.o_token + head * a.o_head);
        const T* g = reinterpret_cast<const T*>(static_cast<const char*>(a.grad_out) + b * a.g_batch +
                                                query * a.g_token + head * a.g_head);
        float sum = 0.0f;
        for (int at = part * V; at < a.D; at += 8 * V) {
            float x[V], y[V];
            load_as(o + at, x);
            load_as(g + at, y);
#pragma unroll
            for (int e = 0; e < V; ++e) sum = fmaf(x[e], y[e], sum);
        }
#pragma unroll
        for (int m = 1; m < 8; m *= 2) sum += __shfl_xor(sum, m);
        if (part != 0) continue;
        const int64_t stat = (b * a.H + head) * a.Nq + query;
        const float lse = a.lse[stat];
        float lse2 = lse / kLn2;
        if (fabsf(lse2) >= kFarLse) lse2 += fabsf(lse2) * 0x1p-22f;
        a.lse2[stat] = lse == -kInf ? kInf : lse2;
        a.delta[stat] = sum;
    }
}

// ---- splits' gradients added up ----------------------------------------------------------
//
// Eight numbers of grad_q, grad_k and grad_v in turn to `threads` threads, a power of two up to
// 32, which have every so many splits each and meet in the wave: with one thread to all of 50
// splits the launch was bound by its reads' latency.
struct JoinSide {
    const float* part;
    void* out;
    int64_t numbers;   // of one split; a multiple of 8
    int32_t splits;
};
struct JoinArgs {
    JoinSide side[3];
};

template <typename T>
__global__ __launch_bounds__(kAttnThreads) void attn_grad_join_kernel(JoinArgs a, int threads) {
    int64_t at = ((int64_t)blockIdx.x * kAttnThreads + threadIdx.x) / threads * 8;
    const int first = threadIdx.x % threads;
    int i = 0;
    while (i < 2 && at >= a.side[i].numbers) at -= a.side[i++].numbers;
    const JoinSide& t = a.side[i];
    if (at >= t.numbers) return;
    float sum[8] = {};
#pragma unroll 4
    for (int s = first; s < t.splits; s += threads) {
        float v[8];
        load_as(t.part + s * t.numbers + at, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[e] += v[e];
    }
    for (int m = 1; m < threads; m *= 2)
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[e] += __shfl_xor(sum[e], m);
    if (first == 0) store_as(static_cast<T*>(t.out) + at, sum);
}

template <typename T, int DP>
void launch(const AttnArgs& of_q, const AttnArgs& of_kv, hipStream_t stream) {
    const int q = (of_q.blocks + 7) / 8 * 8, kv = (of_kv.blocks + 7) / 8 * 8;
    if (of_q.mask)
        attn_grad_kernel<T, DP, true><<<(uint32_t)(q + kv), kAttnThreads, 0, stream>>>(of_q, of_kv, q);
    else
        attn_grad_kernel<T, DP, false><<<(uint32_t)(q + kv), kAttnThreads, 0, stream>>>(of_q, of_kv, q);
}

template <typename T>
hipError_t launch_type(const AttnArgs& of_q, const AttnArgs& of_kv, hipStream_t stream) {
    if (of_q.D <= 32)
        launch<T, 32>(of_q, of_kv, stream);
    else if (of_q.D <= 64)
        launch<T, 64>(of_q, of_kv, stream);
    else if (of_q.D <= 96)
        launch<T, 96>(of_q, of_kv, stream);
    else
        launch<T, 128>(of_q, of_kv, stream);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_attn_grad(const AttnArgs& of_q, const AttnArgs& of_kv, hipStream_t stream) {
    if (of_q.dtype == DA_BF16) return launch_type<__bf16>(of_q, of_kv, stream);
    if (of_q.dtype == DA_F16) return launch_type<_Float16>(of_q, of_kv, stream);
    return launch_type<float>(of_q, of_kv, stream);
}

hipError_t launch_attn_grad_join(const AttnArgs& of_q, const AttnArgs& of_kv, hipStream_t stream) {
    JoinArgs a = {};
    if (of_q.blocks && of_q.splits > 1)
        a.side[0] = {of_q.part, of_q.grad_q, (int64_t)of_q.B * of_q.Nq * of_q.H * of_q.D, of_q.splits};
    if (of_kv.blocks && of_kv.splits > 1) {
        const int64_t n = (int64_t)of_kv.B * of_kv.Nk * of_kv.Hk * of_kv.D;
        a.side[1] = {of_kv.part_k, of_kv.grad_k, n, of_kv.splits};
        a.side[2] = {of_kv.part_v, of_kv.grad_v, n, of_kv.splits};
    }
    const int64_t eights = (a.side[0].numbers + a.side[1].numbers + a.side[2].numbers) / 8;
    if (eights == 0) return hipSuccess;
    const int most = std::max(a.side[0].numbers ? a.side[0].splits : 1, a.side[1].numbers ? a.side[1].splits : 1);
    int threads = 1;
    while (threads < 32 && threads * 4 < most) threads *= 2;
    const uint32_t blocks = (uint32_t)((eights * threads + kAttnThreads - 1) / kAttnThreads);
    if (of_q.dtype == DA_BF16)
        attn_grad_join_kernel<__bf16><<<blocks, kAttnThreads, 0, stream>>>(a, threads);
    else if (of_q.dtype == DA_F16)
        attn_grad_join_kernel<_Float16><<<blocks, kAttnThreads, 0, stream>>>(a, threads);
    else
        attn_grad_join_kernel<float><<<blocks, kAttnThreads, 0, stream>>>(a, threads);
    return hipGetLastError();
}

hipError_t launch_attn_delta(const AttnArgs& a, hipStream_t stream) {
    const int64_t threads = (int64_t)a.B * a.Nq * a.H * 8;
    const uint32_t blocks = (uint32_t)std::min<int64_t>((threads + kAttnThreads - 1) / kAttnThreads, 1 << 22);
    if (a.dtype == DA_BF16)
        attn_delta_kernel<__bf16><<<blocks, kAttnThreads, 0, stream>>>(a);
    else if (a.dtype == DA_F16)
        attn_delta_kernel<_Float16><<<blocks, kAttnThreads, 0, stream>>>(a);
    else
        attn_delta_kernel<float><<<blocks, kAttnThreads, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace da
