// Attention's gradients to the queries, and the sums that the other gradients need as well.  Contract
// and formulas: include/attention.h; tiles and products: attn_device.h.
//
// As in the forward, columns are rows of queries and keys and values are streamed; a column's
// lse and delta are a register each.  Three products to a tile: scores, dP, and keys times dS.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "attn_device.h"

namespace da {
namespace {

template <typename T, int DP>
constexpr int kGradQWaves = sizeof(T) == 4 ? 1 : 2;

template <typename T, int DP, bool MASK>
__global__ __launch_bounds__(kAttnThreads, (kGradQWaves<T, DP>))
void attn_grad_q_kernel(AttnArgs a) {
    constexpr int TILE = kAttnTile, NB = TILE / 32, ND = DP / 32;
    using Tl = Tile<T, DP, TILE>;
    __shared__ u32x4 k0[Tl::kPieces], v0[Tl::kPieces], k1[Tl::kPieces], v1[Tl::kPieces];
    const Spot spot = spot_of(a);
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
    float lse2 = kInf, delta = 0.0f;
    {
        u32x4 oc[Tl::kSteps];
        load_column<T, DP>(static_cast<const char*>(a.out) + b * a.o_batch + query * a.o_token +
                               head * a.o_head,
                           there, a.D, half, oc);
#pragma unroll
        for (int t = 0; t < Tl::kSteps; ++t) delta = dot_pieces<T>(oc[t], gc[t], delta);
        delta = column_sum(delta);
        const int64_t stat = ((int64_t)b * a.H + head) * a.Nq + query;
        if (there) {
            const float lse = a.lse[stat];
            lse2 = lse == -kInf ? kInf : lse / kLn2;
            if (spot.split == 0 && half == 0) {   // for the other gradients
                a.lse2[stat] = lse2;
                a.delta[stat] = delta;
            }
        }
    }

    const char* kp = static_cast<const char*>(a.k) + b * a.k_batch + hk * a.k_head + first * a.k_token;
    const char* vp = static_cast<const char*>(a.v) + b * a.v_batch + hk * a.v_head + first * a.v_token;
    const uint8_t* mask = MASK ? a.mask + (int64_t)b * a.Nk + first : nullptr;
    const Places<T, DP> at(lane);
    const Filler<Tl> filler(threadIdx.x, a.D * (int)sizeof(T));
    uint32_t byte = 1;   // of the tile that is fetched next

    // Fetches tile j, or zeros past the last, and reads the mask of the one after it.
    const auto fetch = [&](int j, u32x4* ks, u32x4* vs) {
        const int rows = min(keys - j * TILE, TILE);
        const Visible vis = visible(byte, rows, lane);
        filler.template run<MASK>(kp + (int64_t)j * TILE * a.k_token, rows, (uint32_t)a.k_token, ks, wave, vis);
        filler.template run<MASK>(vp + (int64_t)j * TILE * a.v_token, rows, (uint32_t)a.v_token, vs, wave, vis);
        if constexpr (MASK) byte = mask_byte(mask + (int64_t)(j + 1) * TILE, keys - (j + 1) * TILE, lane);
        return vis;
    };

    f32x16 acc[ND];
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[d][i] = 0.0f;
    Lift<T, ND> lift;

    const auto step = [&](LdsBytes ks, LdsBytes vs, const Visible& vis) {
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            f32x16 s = mul_columns<T, DP>(at, ks, n, qc);
            const f32x16 dp = mul_columns<T, DP>(at, vs, n, gc);
#pragma unroll
            for (int i = 0; i < 16; ++i)
                s[i] = __builtin_amdgcn_exp2f(fmaf(s[i], a.scale2, -lse2)) * (dp[i] - delta);
            hide(s, vis.block(n), half, 0.0f);
            lift.apply(s, acc);
            mul_rows<T, DP, false>(at, ks, n, Weights<T, false>(s), acc);
        }
    };

    // A tile is worked on while the next one fills the other half of LDS.  The loop has no branches of
    // its own, so that the results stay in their registers.
    if (tiles > 0) {
        if constexpr (MASK) byte = mask_byte(mask, keys, lane);
        Visible here = fetch(0, k0, v0);
        tile_barrier();
        for (int j = 0; j + 1 < tiles; j += 2) {
            Visible next = fetch(j + 1, k1, v1);
            step((LdsBytes)k0, (LdsBytes)v0, here);
            tile_barrier();
            here = fetch(j + 2, k0, v0);
            step((LdsBytes)k1, (LdsBytes)v1, next);
            tile_barrier();
        }
        if (tiles % 2) step((LdsBytes)k0, (LdsBytes)v0, here);
    }

    if (!there) return;
    const float factor = a.scale * lift.down();
    if (a.splits > 1)
        store_column<float, ND>(a.part + (spot.split * (int64_t)a.B * a.Nq * a.H + line) * a.D, a.D, half,
                                acc, factor);
    else
        store_column<T, ND>(static_cast<T*>(a.grad_q) + line * a.D, a.D, half, acc, factor);
}

// ---- lse in base 2, and delta, where the queries' gradients are not wanted ---------------
//
// Eight lanes to a row of out and grad_out, a run of 16-byte pieces in turn to each.
template <typename T>
__global__ __launch_bounds__(kAttnThreads) void attn_delta_kernel(AttnArgs a) {
    constexpr int V = 16 / (int)sizeof(T);
    const int64_t line = ((int64_t)blockIdx.x * kAttnThreads + threadIdx.x) / 8;
    const int part = threadIdx.x % 8;
    if (line >= (int64_t)a.B * a.Nq * a.H) return;
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
    if (part != 0) return;
    const int64_t stat = (b * a.H + head) * a.Nq + query;
    const float lse = a.lse[stat];
    a.lse2[stat] = lse == -kInf ? kInf : lse / kLn2;
    a.delta[stat] = sum;
}

// ---- splits' gradients added up ----------------------------------------------------------
//
// Eight numbers to a thread, of grad_q, grad_k and grad_v in turn.
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
__global__ __launch_bounds__(kAttnThreads) void attn_grad_join_kernel(JoinArgs a) {
    int64_t at = ((int64_t)blockIdx.x * kAttnThreads + threadIdx.x) * 8;
    int i = 0;
    while (i < 2 && at >= a.side[i].numbers) at -= a.side[i++].numbers;
    const JoinSide& t = a.side[i];
    if (at >= t.numbers) return;
    float sum[8];
    load_as(t.part + at, sum);
#pragma unroll 4
    for (int s = 1; s < t.splits; ++s) {
        float v[8];
        load_as(t.part + s * t.numbers + at, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[e] += v[e];
    }
    store_as(static_cast<T*>(t.out) + at, sum);
}

template <typename T, int DP>
void launch(const AttnArgs& a, hipStream_t stream) {
    const uint32_t blocks = (uint32_t)(a.blocks + 7) / 8 * 8;
    if (a.mask)
        attn_grad_q_kernel<T, DP, true><<<blocks, kAttnThreads, 0, stream>>>(a);
    else
        attn_grad_q_kernel<T, DP, false><<<blocks, kAttnThreads, 0, stream>>>(a);
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
    return hipGetLastError();
}

}  // namespace

hipError_t launch_attn_grad_q(const AttnArgs& a, hipStream_t stream) {
    if (a.dtype == DA_BF16) return launch_type<__bf16>(a, stream);
    if (a.dtype == DA_F16) return launch_type<_Float16>(a, stream);
    return launch_type<float>(a, stream);
}

hipError_t launch_attn_grad_join(const AttnArgs& of_q, const AttnArgs& of_kv, hipStream_t stream) {
    JoinArgs a = {};
    if (of_q.grad_q && of_q.splits > 1)
        a.side[0] = {of_q.part, of_q.grad_q, (int64_t)of_q.B * of_q.Nq * of_q.H * of_q.D, of_q.splits};
    if (of_kv.grad_k && of_kv.splits > 1) {
        const int64_t n = (int64_t)of_kv.B * of_kv.Nk * of_kv.Hk * of_kv.D;
        a.side[1] = {of_kv.part_k, of_kv.grad_k, n, of_kv.splits};
        a.side[2] = {of_kv.part_v, of_kv.grad_v, n, of_kv.splits};
    }
    const int64_t threads = (a.side[0].numbers + a.side[1].numbers + a.side[2].numbers) / 8;
    if (threads == 0) return hipSuccess;
    const uint32_t blocks = (uint32_t)((threads + kAttnThreads - 1) / kAttnThreads);
    if (of_q.dtype == DA_BF16)
        attn_grad_join_kernel<__bf16><<<blocks, kAttnThreads, 0, stream>>>(a);
    else if (of_q.dtype == DA_F16)
        attn_grad_join_kernel<_Float16><<<blocks, kAttnThreads, 0, stream>>>(a);
    else
        attn_grad_join_kernel<float><<<blocks, kAttnThreads, 0, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_attn_delta(const AttnArgs& a, hipStream_t stream) {
    const int64_t threads = (int64_t)a.B * a.Nq * a.H * 8;
    const uint32_t blocks = (uint32_t)((threads + kAttnThreads - 1) / kAttnThreads);
    if (a.dtype == DA_BF16)
        attn_delta_kernel<__bf16><<<blocks, kAttnThreads, 0, stream>>>(a);
    else if (a.dtype == DA_F16)
        attn_delta_kernel<_Float16><<<blocks, kAttnThreads, 0, stream>>>(a);
    else
        attn_delta_kernel<float><<<blocks, kAttnThreads, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace da
