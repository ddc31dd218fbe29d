// Internal launch description of the attention kernels (attn_forward.hip, attn_grad.hip), filled by
// the host API (attn_api.cpp).  Not part of the public ABI.
//
// Rows are the queries of the heads that share a key head: row r of a (batch entry, key head)
// is query r / group of its head r % group.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#include "attention.h"

namespace da {

constexpr int kAttnThreads = 256;   // four waves
// A workgroup has 32 columns (rows of the forward and of grad_q, keys of grad_k and grad_v) to each
// wave.  Where that leaves the forward too few workgroups, one has 32 rows in all and its waves
// share the keys, 32 at a time to each.
constexpr int kAttnWide = 128, kAttnFew = 32;
constexpr int kAttnTile = 64;      // rows or keys streamed at a time, kAttnFew to each wave of the other
constexpr int kAttnMostSplits = 256;   // of a forward's keys: a thread of the join to each

struct AttnArgs {
    const void *q, *k, *v;
    const int32_t* lens;      // [B] or NULL
    const uint8_t* mask;      // [B, Nk] or NULL
    void* out;                // [B, Nq, H, D], strided
    float* lse;               // [B, H, Nq] or NULL in the forward
    const void* grad_out;
    void *grad_q, *grad_k, *grad_v;   // dense
    float* part;              // forward: [splits, B Hk, rows, D] results of a split's keys, not
                              // divided by their sums
    float2* part_stat;        // forward: [splits, B Hk, rows] (logarithm of base 2 that the
                              // result is scaled by, sum), or (largest score, -sum) of far ones
    float *part_k, *part_v;   // backward: [splits, B, Nk, Hk, D] (and part, [splits, B, Nq, H, D])
                              // gradients from a split's rows (keys)
    float* lse2;              // backward: [B, H, Nq] lse in base 2, +infinity for an empty row
    float* delta;             // backward: [B, H, Nq]
    int64_t q_batch, q_token, q_head;   // strides in bytes
    int64_t k_batch, k_token, k_head;
    int64_t v_batch, v_token, v_head;
    int64_t o_batch, o_token, o_head;
    int64_t g_batch, g_token, g_head;   // of grad_out
    int32_t B, Nq, Nk, H, Hk, D;
    int32_t group, rows;      // H / Hk; Nq * group
    int32_t col_tiles;        // tiles of columns
    int32_t splits;           // of what is streamed
    int32_t split_keys;       // keys of a split (forward), or tiles of it (backward)
    int32_t blocks;           // workgroups with work; a launch has a multiple of 8 of each kind
    float scale, scale2;      // scale2: scale / log 2
    int32_t dtype;
    bool few;
};

// Waves of a workgroup with few rows.  They have tiles of their own, two of 32 keys and values each
// where 128 KB hold them; eight where that leaves room for them, else four.
constexpr int attn_few_waves(int head_bytes) { return head_bytes <= 128 ? 8 : 4; }
inline int attn_few_waves(const AttnArgs& a) {
    const int wide = a.D <= 32 ? 32 : a.D <= 64 ? 64 : 128;
    return attn_few_waves(wide * (a.dtype == DA_F32 ? 4 : 2));
}

hipError_t launch_attn_forward(const AttnArgs& a, hipStream_t stream);
hipError_t launch_attn_delta(const AttnArgs& a, hipStream_t stream);
// Both kinds of gradients, after delta; one without blocks is left out.
hipError_t launch_attn_grad(const AttnArgs& of_q, const AttnArgs& of_kv, hipStream_t stream);
// Splits' gradients added up: of_q's, of_kv's, where they have more than one.
hipError_t launch_attn_grad_join(const AttnArgs& of_q, const AttnArgs& of_kv, hipStream_t stream);

}  // namespace da
