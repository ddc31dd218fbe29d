// Host side of the attention: argument checks, the form a problem takes, dispatch.  Every check
// runs before anything is enqueued.  Contract: include/attention.h.
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>
#include <utility>

#include "attention.h"
#include "attn_internal.h"
#include "host_errors.h"
#include "host_strides.h"

namespace {

using da::extent_bytes;
using da::may_meet;
using da::ranges_clash;
using da::report_error;

typedef da::wide_t wide;
constexpr int64_t k2to31 = int64_t(1) << 31;

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }
int elem_bytes(int32_t t) { return t == DA_F32 ? 4 : 2; }
uint64_t part_bytes(uint64_t n) { return (n + 255) & ~uint64_t(255); }

da_status check_strides(const char* name, const int64_t (&stride)[3], int64_t batch, int64_t tokens,
                        int64_t heads, int64_t D, int e) {
    for (int64_t s : stride) {
        if (s < 0) return report_error(DA_ERR_INVALID_ARG, "a stride of %s is negative", name);
        if (s > (int64_t(1) << 56) || s * e % 16 != 0)
            return report_error(DA_ERR_INVALID_ARG, "a stride of %s is not a multiple of 16 bytes", name);
    }
    if (stride[1] * e >= (1 << 24))
        return report_error(DA_ERR_UNSUPPORTED, "a token of %s takes 2^24 bytes or more", name);
    if (extent_bytes(stride, batch, tokens, heads, D, e) >= ((wide)1 << 62))
        return report_error(DA_ERR_UNSUPPORTED, "%s spans 2^62 bytes or more", name);
    return DA_OK;
}

da_status check_problem(const attn_problem* p) {
    if (!p) return report_error(DA_ERR_INVALID_ARG, "problem is NULL");
    if (p->flags != 0 || p->reserved != 0)
        return report_error(DA_ERR_INVALID_ARG, "problem.flags and problem.reserved must be 0");
    if (p->batch < 0 || p->queries < 0 || p->keys < 0)
        return report_error(DA_ERR_INVALID_ARG, "batch, queries and keys must be >= 0");
    if (p->heads < 1 || p->key_heads < 1 || p->head_dim < 1)
        return report_error(DA_ERR_INVALID_ARG, "heads, key_heads and head_dim must be >= 1");
    if (p->heads % p->key_heads != 0)
        return report_error(DA_ERR_INVALID_ARG, "heads (%lld) is not a multiple of key_heads (%lld)",
                            (long long)p->heads, (long long)p->key_heads);
    if (p->dtype != DA_F32 && p->dtype != DA_BF16 && p->dtype != DA_F16)
        return report_error(DA_ERR_INVALID_ARG, "dtype %d is not a da_dtype", (int)p->dtype);
    if (!(p->scale > 0.0f) || !(p->scale <= 0x1p126f))   // times 1 / log 2 it is finite
        return report_error(DA_ERR_INVALID_ARG, "scale must be > 0 and at most 2^126");
    if (p->head_dim % 8 != 0 || p->head_dim > 128)
        return report_error(DA_ERR_UNSUPPORTED, "head_dim is not a multiple of 8 up to 128");
    const int e = elem_bytes(p->dtype);
    if (p->batch >= k2to31 || p->queries >= k2to31 || p->keys >= (int64_t(1) << 30) || p->heads >= k2to31 ||
        (wide)p->queries * (p->heads / p->key_heads) >= k2to31 - 256 ||
        (wide)p->batch * p->key_heads >= k2to31 || (wide)p->heads * p->head_dim * e >= (1 << 24))
        return report_error(DA_ERR_UNSUPPORTED,
                            "2^31 rows or key heads, 2^30 keys, or heads of 2^24 bytes a token");
    if ((wide)p->batch * p->queries * p->heads >= (wide)1 << 45 ||
        (wide)p->batch * p->keys * p->key_heads >= (wide)1 << 45)
        return report_error(DA_ERR_UNSUPPORTED, "2^45 rows or keys");
    da_status st = check_strides("q", p->q_stride, p->batch, p->queries, p->heads, p->head_dim, e);
    if (st == DA_OK) st = check_strides("k", p->k_stride, p->batch, p->keys, p->key_heads, p->head_dim, e);
    if (st == DA_OK) st = check_strides("v", p->v_stride, p->batch, p->keys, p->key_heads, p->head_dim, e);
    if (st == DA_OK)
        st = check_strides("out", p->out_stride, p->batch, p->queries, p->heads, p->head_dim, e);
    return st;
}

void describe(const attn_problem* p, da::AttnArgs& a) {
    memset(&a, 0, sizeof a);
    const int64_t e = elem_bytes(p->dtype);
    a.q_batch = p->q_stride[0] * e, a.q_token = p->q_stride[1] * e, a.q_head = p->q_stride[2] * e;
    a.k_batch = p->k_stride[0] * e, a.k_token = p->k_stride[1] * e, a.k_head = p->k_stride[2] * e;
    a.v_batch = p->v_stride[0] * e, a.v_token = p->v_stride[1] * e, a.v_head = p->v_stride[2] * e;
    a.o_batch = p->out_stride[0] * e, a.o_token = p->out_stride[1] * e, a.o_head = p->out_stride[2] * e;
    a.g_batch = p->grad_stride[0] * e, a.g_token = p->grad_stride[1] * e, a.g_head = p->grad_stride[2] * e;
    a.B = (int32_t)p->batch;
    a.Nq = (int32_t)p->queries;
    a.Nk = (int32_t)p->keys;
    a.H = (int32_t)p->heads;
    a.Hk = (int32_t)p->key_heads;
    a.D = (int32_t)p->head_dim;
    a.group = a.H / a.Hk;
    a.rows = a.Nq * a.group;
    a.splits = 1;
    a.split_keys = std::max(a.Nk, 1);
    a.scale = p->scale;
    a.scale2 = (float)((double)p->scale * 1.4426950408889634);
    a.dtype = p->dtype;
}

// The forward's form and the splits of its keys: of a few candidates the one whose time this counts
// least, in microseconds.  A workgroup takes so long for a tile of 64 keys (wide) or for its waves'
// 32 keys each (few rows), longer where several have to share a compute unit (16 heads of 48 on
// 3 x 1329 rows, binary16: wide 44, by 32 rows 73); splits cost a launch that joins them, and their
// results' way.  Measured, 8 heads of 64 numbers, bfloat16:
// 128 rows on 8192 keys wide in 1, 8 and 32 splits 89, 22 and 20 us, by 32 rows 35, 16 and 28; 300
// rows on 4096 keys wide in 1, 4, 8 and 16 splits 48, 21, 19 and 23, by 32 rows in 1, 3 and 8 21, 17
// and 26; 16 x 875 rows of two entries on 684 keys wide 14, by 32 rows 29; one row on 1500 keys in
// 1 and 6 splits 11.4 and 10.7 on the GPU, 11 and 15 with the second launch's host time.
void choose_forward(da::AttnArgs& a) {
    const int64_t units = (int64_t)a.B * a.Hk;
    const int D = a.D <= 32 ? 32 : a.D <= 64 ? 64 : a.D <= 96 ? 96 : 128, waves = da::attn_few_waves(a);
    const bool f32 = a.dtype == DA_F32;
    const double step_time[2] = {f32 ? 0.35 + 0.058 * D : 0.45 + 0.004 * D,
                                 f32 ? 0.009 * D * waves : 0.7 + 0.0036 * D};
    double best = 1e30;
    for (int few = a.rows <= da::kAttnFew; few < 2; ++few) {
        const int64_t width = few ? da::kAttnFew : da::kAttnWide;
        const int64_t tiles = (a.rows + width - 1) / width, blocks = std::max<int64_t>(units * tiles, 1);
        const int64_t keys = few ? (int64_t)da::kAttnFew * waves : da::kAttnTile;   // of a step
        const int64_t steps = std::max<int64_t>((a.Nk + keys - 1) / keys, 1);
        for (int64_t most : {int64_t(1), 256 / blocks, 512 / blocks}) {
            const int64_t splits = std::min({most, steps, (int64_t)da::kAttnMostSplits});
            if (splits < 1) continue;
            const int64_t per = (steps + splits - 1) / splits, made = (steps + per - 1) / per;
            // 32 rows to a workgroup: one to a compute unit, and four times the states' way
            const int64_t all = blocks * made, rounds = (all + 255) / 256;
            const double load = !few ? std::max(1.0, (double)all / 256)
                                     : rounds == 1 ? 1.0 : (double)rounds * (f32 ? 1.2 : 1.8);
            double time = load * (double)per * step_time[few];
            if (made > 1) time += 6.0 + 2e-6 * (double)(made * units * a.rows) * a.D;
            if (time >= best) continue;
            best = time;
            a.few = few;
            a.col_tiles = (int32_t)tiles;
            a.splits = (int32_t)made;
            a.split_keys = (int32_t)(made > 1 ? per * keys : std::max(a.Nk, 1));
        }
    }
    // long shares are halved, so that entries of different lengths spread over the compute units
    const int64_t keys = a.few ? (int64_t)da::kAttnFew * waves : da::kAttnTile, per = a.split_keys / keys;
    if (a.splits > 1 && per >= 32 && a.splits * 2 <= da::kAttnMostSplits) {
        a.split_keys = (int32_t)((per + 1) / 2 * keys);
        a.splits = (int32_t)((a.Nk + (int64_t)a.split_keys - 1) / a.split_keys);
    }
}

// The splits of what is streamed to so many columns of a key head: up to 128 workgroups in all, 256
// where each keeps 8 tiles, 512 where it keeps 32.  Measured, 64 numbers, bfloat16, both kinds
// together: 900 queries on 600 keys of 8 heads (64 and 40 workgroups of 10 and 15 tiles) without
// splits, up to 128, 256 and 512 workgroups 37, 28, 31 and 33 us; 2048 on 2048 of 8 heads (128 of 32)
// 70, 70, 62 and 60; 293 on 6304 of 2 heads (6 of 99, 100 of 5) 86, 24, 45 and 50.
void choose_backward(da::AttnArgs& a, int64_t columns, int64_t tiles) {
    a.col_tiles = (int32_t)((columns + da::kAttnWide - 1) / da::kAttnWide);
    const int64_t blocks = std::max<int64_t>((int64_t)a.B * a.Hk * a.col_tiles, 1);
    tiles = std::max<int64_t>(tiles, 1);
    int64_t per = tiles;
    for (const auto& t : {std::pair<int, int>{128, 1}, {256, 8}, {512, 32}}) {
        const int64_t splits = std::min(tiles, t.first / blocks);
        if (splits < 1) continue;
        const int64_t share = (tiles + splits - 1) / splits;
        if (share >= t.second) per = share;
    }
    a.split_keys = (int32_t)per;
    a.splits = (int32_t)((tiles + per - 1) / per);
}
void choose_grad_q(da::AttnArgs& a) {
    choose_backward(a, a.rows, ((int64_t)a.Nk + da::kAttnTile - 1) / da::kAttnTile);
}
void choose_grad_kv(da::AttnArgs& a) {
    choose_backward(a, a.Nk, ((int64_t)a.Nq + da::kAttnTile - 1) / da::kAttnTile * a.group);
}

// Counts the workgroups; a launch has fewer than 2^32 threads.
da_status count_blocks(da::AttnArgs& a) {
    const wide blocks = (wide)a.B * a.Hk * a.col_tiles * a.splits;
    const int threads = a.few ? 64 * da::attn_few_waves(a) : da::kAttnThreads;
    if (blocks + 8 >= (wide(1) << 32) / threads)
        return report_error(DA_ERR_UNSUPPORTED, "2^32 threads of workgroups or more");
    a.blocks = (int32_t)blocks;
    return DA_OK;
}

// Both kinds of gradients' splits and workgroups, of one launch.  What their joins and delta's launch
// take sets no limit of its own: sides that are split have at most 256 workgroups' columns, and
// delta's workgroups walk over the rows.
da_status plan_backward(da::AttnArgs& of_q, da::AttnArgs& of_kv) {
    choose_grad_q(of_q);
    choose_grad_kv(of_kv);
    da_status st = count_blocks(of_q);
    if (st == DA_OK) st = count_blocks(of_kv);
    if (st == DA_OK && (wide)of_q.blocks + of_kv.blocks + 16 >= (wide(1) << 32) / da::kAttnThreads)
        st = report_error(DA_ERR_UNSUPPORTED, "2^32 threads of workgroups or more");
    return st;
}

uint64_t stat_bytes(const da::AttnArgs& a) {
    return part_bytes((uint64_t)a.splits * a.B * a.Hk * a.rows * sizeof(float2));
}
uint64_t need_forward(const da::AttnArgs& a) {
    if (a.splits == 1) return 0;
    return stat_bytes(a) + part_bytes((uint64_t)a.splits * a.B * a.Hk * a.rows * a.D * sizeof(float));
}
uint64_t part_q_bytes(const da::AttnArgs& q) {
    return q.splits == 1 ? 0 : part_bytes((uint64_t)q.splits * q.B * q.Nq * q.H * q.D * sizeof(float));
}
uint64_t part_k_bytes(const da::AttnArgs& kv) {
    return kv.splits == 1 ? 0 : part_bytes((uint64_t)kv.splits * kv.B * kv.Nk * kv.Hk * kv.D * sizeof(float));
}
uint64_t row_bytes(const da::AttnArgs& a) { return part_bytes((uint64_t)a.B * a.H * a.Nq * sizeof(float)); }

da_status check_workspace(uint64_t need, const void* workspace, size_t workspace_bytes) {
    if (!need) return DA_OK;
    if (!workspace) return report_error(DA_ERR_INVALID_ARG, "workspace is NULL");
    if (!aligned(workspace, 256))
        return report_error(DA_ERR_INVALID_ARG, "workspace is not 256-byte aligned");
    if (workspace_bytes < need)
        return report_error(DA_ERR_INVALID_ARG, "workspace has %zu bytes, %llu needed",
                            workspace_bytes, (unsigned long long)need);
    return DA_OK;
}

struct Sizes {
    wide q, k, v, out, grad, dense_q, dense_k;
};
Sizes sizes_of(const attn_problem* p) {
    const int e = elem_bytes(p->dtype);
    return {extent_bytes(p->q_stride, p->batch, p->queries, p->heads, p->head_dim, e),
            extent_bytes(p->k_stride, p->batch, p->keys, p->key_heads, p->head_dim, e),
            extent_bytes(p->v_stride, p->batch, p->keys, p->key_heads, p->head_dim, e),
            extent_bytes(p->out_stride, p->batch, p->queries, p->heads, p->head_dim, e),
            extent_bytes(p->grad_stride, p->batch, p->queries, p->heads, p->head_dim, e),
            (wide)p->batch * p->queries * p->heads * p->head_dim * e,
            (wide)p->batch * p->keys * p->key_heads * p->head_dim * e};
}

da_status check_inputs(const attn_problem* p, const void* q, const void* k, const void* v,
                       const int32_t* kv_lens) {
    if ((p->queries > 0 && !q) || (p->keys > 0 && (!k || !v)))
        return report_error(DA_ERR_INVALID_ARG, "q / k / v is NULL");
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16))
        return report_error(DA_ERR_INVALID_ARG, "q / k / v is not 16-byte aligned");
    if (!aligned(kv_lens, 4)) return report_error(DA_ERR_INVALID_ARG, "kv_lens is not 4-byte aligned");
    return DA_OK;
}

}  // namespace

extern "C" {

da_status attn_forward_workspace_size(const attn_problem* p, size_t* bytes) {
    if (!bytes) return report_error(DA_ERR_INVALID_ARG, "bytes is NULL");
    da_status st = check_problem(p);
    if (st != DA_OK) return st;
    da::AttnArgs a;
    describe(p, a);
    choose_forward(a);
    *bytes = 0;
    if (p->batch == 0 || p->queries == 0) return DA_OK;
    st = count_blocks(a);
    if (st != DA_OK) return st;
    *bytes = (size_t)need_forward(a);
    return DA_OK;
}

da_status attn_forward(const attn_problem* p, const void* q, const void* k, const void* v,
                       const int32_t* kv_lens, const uint8_t* key_mask, void* out, float* lse,
                       void* workspace, size_t workspace_bytes, void* stream) {
    da_status st = check_problem(p);
    if (st != DA_OK) return st;
    if (p->batch == 0 || p->queries == 0) return DA_OK;
    st = check_inputs(p, q, k, v, kv_lens);
    if (st != DA_OK) return st;
    if (!out) return report_error(DA_ERR_INVALID_ARG, "out is NULL");
    if (!aligned(out, 16) || !aligned(lse, 4))
        return report_error(DA_ERR_INVALID_ARG, "out is not 16-byte aligned, or lse not 4-byte");
    const Sizes n = sizes_of(p);
    const wide lse_bytes = (wide)p->batch * p->heads * p->queries * 4;
    const int e = elem_bytes(p->dtype);
    const da::Heads to = {out, {p->batch, p->queries, p->heads}, p->out_stride, p->head_dim, e};
    if (may_meet(to, {q, {p->batch, p->queries, p->heads}, p->q_stride, p->head_dim, e}) ||
        may_meet(to, {k, {p->batch, p->keys, p->key_heads}, p->k_stride, p->head_dim, e}) ||
        may_meet(to, {v, {p->batch, p->keys, p->key_heads}, p->v_stride, p->head_dim, e}) ||
        ranges_clash(out, n.out, lse, lse_bytes) || ranges_clash(lse, lse_bytes, q, n.q) ||
        ranges_clash(lse, lse_bytes, k, n.k) || ranges_clash(lse, lse_bytes, v, n.v))
        return report_error(DA_ERR_INVALID_ARG, "out or lse overlaps an input, or the other");
    if (da::overlaps_itself(p->out_stride, p->batch, p->queries, p->heads, p->head_dim))
        return report_error(DA_ERR_INVALID_ARG, "places of out overlap");
    da::AttnArgs a;
    describe(p, a);
    choose_forward(a);
    st = count_blocks(a);
    if (st == DA_OK) st = check_workspace(need_forward(a), workspace, workspace_bytes);
    if (st != DA_OK) return st;
    a.q = q, a.k = k, a.v = v;
    a.lens = kv_lens;
    a.mask = key_mask;
    a.out = out;
    a.lse = lse;
    if (a.splits > 1) {
        a.part_stat = static_cast<float2*>(workspace);
        a.part = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + stat_bytes(a));
    }
    return da::report_hip(da::launch_attn_forward(a, static_cast<hipStream_t>(stream)),
                          "attention forward launch");
}

da_status attn_backward_workspace_size(const attn_problem* p, size_t* bytes) {
    if (!bytes) return report_error(DA_ERR_INVALID_ARG, "bytes is NULL");
    da_status st = check_problem(p);
    if (st != DA_OK) return st;
    da::AttnArgs a;
    describe(p, a);
    da::AttnArgs of_kv = a;
    st = plan_backward(a, of_kv);
    if (st != DA_OK) return st;
    *bytes = (size_t)(2 * row_bytes(a) + part_q_bytes(a) + 2 * part_k_bytes(of_kv));
    return DA_OK;
}

da_status attn_backward(const attn_problem* p, const void* q, const void* k, const void* v,
                        const void* out, const float* lse, const void* grad_out,
                        const int32_t* kv_lens, const uint8_t* key_mask, void* grad_q, void* grad_k,
                        void* grad_v, void* workspace, size_t workspace_bytes, void* stream) {
    da_status st = check_problem(p);
    if (st != DA_OK) return st;
    st = check_strides("grad_out", p->grad_stride, p->batch, p->queries, p->heads, p->head_dim,
                       elem_bytes(p->dtype));
    if (st != DA_OK) return st;
    if (p->batch == 0) return DA_OK;
    st = check_inputs(p, q, k, v, kv_lens);
    if (st != DA_OK) return st;
    if (p->queries > 0 && (!out || !lse || !grad_out))
        return report_error(DA_ERR_INVALID_ARG, "out / lse / grad_out is NULL");
    if (p->keys > 0 && !grad_k != !grad_v)
        return report_error(DA_ERR_INVALID_ARG, "one of grad_k and grad_v is NULL");
    if (!aligned(out, 16) || !aligned(grad_out, 16) || !aligned(grad_q, 16) || !aligned(grad_k, 16) ||
        !aligned(grad_v, 16) || !aligned(lse, 4))
        return report_error(DA_ERR_INVALID_ARG,
                            "out or a gradient is not 16-byte aligned, or lse not 4-byte");
    const Sizes n = sizes_of(p);
    const struct {
        const void* at;
        wide bytes;
    } results[] = {{grad_q, n.dense_q}, {grad_k, n.dense_k}, {grad_v, n.dense_k}},
      inputs[] = {{q, n.q}, {k, n.k}, {v, n.v}, {out, n.out}, {grad_out, n.grad},
                  {lse, (wide)p->batch * p->heads * p->queries * 4}};
    for (int i = 0; i < 3; ++i) {
        for (const auto& x : inputs)
            if (ranges_clash(results[i].at, results[i].bytes, x.at, x.bytes))
                return report_error(DA_ERR_INVALID_ARG, "a gradient overlaps an input");
        for (int j = 0; j < i; ++j)
            if (ranges_clash(results[i].at, results[i].bytes, results[j].at, results[j].bytes))
                return report_error(DA_ERR_INVALID_ARG, "two gradients overlap");
    }
    da::AttnArgs of_q;
    describe(p, of_q);
    of_q.q = q, of_q.k = k, of_q.v = v;
    of_q.lens = kv_lens;
    of_q.mask = key_mask;
    of_q.out = const_cast<void*>(out);
    of_q.lse = const_cast<float*>(lse);
    of_q.grad_out = grad_out;
    of_q.grad_q = grad_q, of_q.grad_k = grad_k, of_q.grad_v = grad_v;
    unsigned char* base = static_cast<unsigned char*>(workspace);
    of_q.lse2 = reinterpret_cast<float*>(base);
    of_q.delta = reinterpret_cast<float*>(base + row_bytes(of_q));
    da::AttnArgs of_kv = of_q;
    st = plan_backward(of_q, of_kv);
    if (st != DA_OK) return st;
    const uint64_t need = 2 * row_bytes(of_q) + part_q_bytes(of_q) + 2 * part_k_bytes(of_kv);
    st = check_workspace(need, workspace, workspace_bytes);
    if (st != DA_OK) return st;
    of_q.part = reinterpret_cast<float*>(base + 2 * row_bytes(of_q));
    of_kv.part_k = reinterpret_cast<float*>(base + 2 * row_bytes(of_q) + part_q_bytes(of_q));
    of_kv.part_v = of_kv.part_k + part_k_bytes(of_kv) / sizeof(float);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    hipError_t e = hipSuccess;
    if (p->queries == 0 || !grad_q) of_q.blocks = 0;
    if (p->keys == 0 || !grad_k) of_kv.blocks = 0;
    if (of_q.blocks == 0 && of_kv.blocks == 0) return DA_OK;
    if (p->queries > 0) e = da::launch_attn_delta(of_q, s);
    if (e == hipSuccess) e = da::launch_attn_grad(of_q, of_kv, s);
    if (e == hipSuccess) e = da::launch_attn_grad_join(of_q, of_kv, s);
    return da::report_hip(e, "attention backward launch");
}

}  // extern "C"
