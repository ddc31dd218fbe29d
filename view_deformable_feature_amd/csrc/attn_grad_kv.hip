// Attention's gradients to keys and values.  Contract and formulas: include/attention.h; tiles
// and products: attn_device.h.
//
// Columns are keys, and the queries and gradients of every head that reads them are streamed, so
// that the heads' sum forms in the accumulators.  Four products to a tile: scores, dP, the gradients
// times p, and the queries times dS.  An invisible key's column runs along and is written as
// zeros.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "attn_device.h"

namespace da {
namespace {

// In binary16 p lies at 2^15, the largest power that its range holds.
template <typename T>
constexpr float kLiftLog2 = std::is_same<T, _Float16>::value ? 15.0f : 0.0f;

template <typename T, int DP>
constexpr int kGradKvWaves = sizeof(T) == 4 ? 1 : 2;

template <typename T, int DP>
__global__ __launch_bounds__(kAttnThreads) __attribute__((amdgpu_waves_per_eu(kGradKvWaves<T, DP>, kGradKvWaves<T, DP>)))
void attn_grad_kv_kernel(AttnArgs a) {
    constexpr int TILE = kAttnTile, NB = TILE / 32, ND = DP / 32;
    using Tl = Tile<T, DP, TILE>;
    __shared__ u32x4 q0[Tl::kPieces], g0[Tl::kPieces], q1[Tl::kPieces], g1[Tl::kPieces];
    __shared__ __align__(16) float stat0[2 * TILE], stat1[2 * TILE];   // lse2, delta of a tile
    const Spot spot = spot_of(a);
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
    const auto fetch = [&](u32x4* qs, u32x4* gs) {
        const int rows = head < a.group ? min(a.Nq - row, TILE) : 0;
        filler.template run<false>(qp + head * a.q_head + row * a.q_token, rows, (uint32_t)a.q_token, qs, wave, none);
        filler.template run<false>(gp + head * a.g_head + row * a.g_token, rows, (uint32_t)a.g_token, gs, wave, none);
        const int t = threadIdx.x % TILE;
        // past the last row p is 0
        mine = threadIdx.x < TILE ? kInf : 0.0f;
        if (threadIdx.x < 2 * TILE && t < rows)
            mine = (threadIdx.x < TILE ? a.lse2 : a.delta)[stats + (int64_t)head * a.Nq + row + t];
        row += TILE;
        if (row >= a.Nq) {
            row = 0;
            ++head;
        }
    };
    const auto keep = [&](float* stat) {
        if (threadIdx.x < 2 * TILE) stat[threadIdx.x] = mine;
    };

    f32x16 dk[ND], dv[ND];
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) dk[d][i] = dv[d][i] = 0.0f;
    Lift<T, ND> lift;

    const auto step = [&](LdsBytes qs, LdsBytes gs, const float* stat) {
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            f32x16 p = mul_columns<T, DP>(at, qs, n, kc);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const f32x4 lse2 = *reinterpret_cast<const f32x4*>(stat + n * 32 + 8 * j + 4 * half);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    p[4 * j + e] = __builtin_amdgcn_exp2f(
                        fmaf(p[4 * j + e], a.scale2, kLiftLog2<T> - lse2[e]));
            }
            mul_rows<T, DP, false>(at, gs, n, Weights<T, false>(p), dv);
            f32x16 ds = mul_columns<T, DP>(at, gs, n, vc);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const f32x4 delta =
                    *reinterpret_cast<const f32x4*>(stat + TILE + n * 32 + 8 * j + 4 * half);
#pragma unroll
                for (int e = 0; e < 4; ++e) ds[4 * j + e] = p[4 * j + e] * (ds[4 * j + e] - delta[e]);
            }
            lift.apply(ds, dk);
            mul_rows<T, DP, false>(at, qs, n, Weights<T, false>(ds), dk);
        }
    };

    // A tile is worked on while the next one fills the other half of LDS.  The loop has no branches of
    // its own, so that the results stay in their registers.
    if (tiles > 0) {
        fetch(q0, g0);
        keep(stat0);
        tile_barrier();
        for (int j = 0; j + 1 < tiles; j += 2) {
            fetch(q1, g1);
            step((LdsBytes)q0, (LdsBytes)g0, stat0);
            keep(stat1);
            tile_barrier();
            fetch(q0, g0);
            step((LdsBytes)q1, (LdsBytes)g1, stat1);
            keep(stat0);
            tile_barrier();
        }
        if (tiles % 2) step((LdsBytes)q0, (LdsBytes)g0, stat0);
    }
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

template <typename T, int DP>
void launch(const AttnArgs& a, hipStream_t stream) {
    const uint32_t blocks = (uint32_t)(a.blocks + 7) / 8 * 8;
    attn_grad_kv_kernel<T, DP><<<blocks, kAttnThreads, 0, stream>>>(a);
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

hipError_t launch_attn_grad_kv(const AttnArgs& a, hipStream_t stream) {
    if (a.dtype == DA_BF16) return launch_type<__bf16>(a, stream);
    if (a.dtype == DA_F16) return launch_type<_Float16>(a, stream);
    return launch_type<float>(a, stream);
}

}  // namespace da
