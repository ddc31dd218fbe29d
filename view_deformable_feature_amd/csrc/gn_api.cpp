// Host side of the group norm: argument checks, slab and chunk layout, dispatch.
// Every check runs before anything is enqueued.  Contract: include/group_norm.h.
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>
#include <numeric>

#include "gn_internal.h"
#include "group_norm.h"
#include "host_errors.h"

namespace {

using da::report_error;

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }
bool valid_dtype(int32_t t) { return t == DA_F32 || t == DA_BF16 || t == DA_F16; }
int elem_bytes(int32_t t) { return t == DA_F32 ? 4 : 2; }

// [a, a + na) and [b, b + nb) share a byte, or are one tensor seen as two types
bool clash(const void* a, int64_t na, const void* b, int64_t nb, bool may_be_same) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    if (x == y && may_be_same) return false;
    return x < y + (uintptr_t)nb && y < x + (uintptr_t)na;
}

da_status check_problem(const gn_problem* p) {
    if (!p) return report_error(DA_ERR_INVALID_ARG, "problem is NULL");
    if (p->flags != 0 || p->reserved != 0)
        return report_error(DA_ERR_INVALID_ARG, "problem.flags and problem.reserved must be 0");
    if (p->batch < 0) return report_error(DA_ERR_INVALID_ARG, "batch must be >= 0");
    if (p->rows < 1 || p->channels < 1 || p->groups < 1)
        return report_error(DA_ERR_INVALID_ARG, "rows, channels and groups must be >= 1");
    if (p->channels % p->groups != 0)
        return report_error(DA_ERR_INVALID_ARG, "channels (%lld) is not a multiple of groups (%lld)",
                            (long long)p->channels, (long long)p->groups);
    if (!valid_dtype(p->x_dtype) || !valid_dtype(p->out_dtype))
        return report_error(DA_ERR_INVALID_ARG, "x_dtype %d / out_dtype %d is not a da_dtype",
                            (int)p->x_dtype, (int)p->out_dtype);
    if (p->activation < DA_ACT_NONE || p->activation > DA_ACT_GELU)
        return report_error(DA_ERR_INVALID_ARG, "activation %d is not a da_activation",
                            (int)p->activation);
    if (!isfinite(p->eps) || p->eps < 0.0f)
        return report_error(DA_ERR_INVALID_ARG, "eps must be finite and >= 0");
    if (p->channels > (1 << 16)) return report_error(DA_ERR_UNSUPPORTED, "channels > 2^16");
    if (p->batch >= (int64_t(1) << 31) || p->rows >= (int64_t(1) << 31) ||
        (p->batch > 0 && p->rows > (int64_t(1) << 45) / p->batch))
        return report_error(DA_ERR_UNSUPPORTED, "2^31 images or rows of an image, or 2^45 rows");
    return DA_OK;
}

// Workspace parts in bytes, 256-byte aligned.
uint64_t part_bytes(uint64_t n) { return (n + 255) & ~uint64_t(255); }

// The layout of an image's slab in one workgroup of up to `threads` threads, `most` vectors
// to a thread; false where none fits.  Of the widths that fit, the widest that leaves a
// workgroup for every compute unit, else the narrowest of at least 64 bytes of a row.  Measured
// (us in a captured graph, whole slabs and by chunks): 64 x 784 x 256 bfloat16 forward 17 and
// 27, backward 33 and 43; 6 x 176 x 256 binary32 6.3 and 10.6, 8.6 and 10.6; 1 x 196 x 512
// binary16 6.0 and 12.4, 9.0 and 14.8.  Small maps of few rows may go by 16 and 32 bytes, for
// more workgroups: 2 x 784 x 256 bfloat16 takes 6.8 so and 9.4 by 64 bytes; but each row is a
// line fetched for a piece of it, and 2 x 4096 x 64 bfloat16 takes 11.8 (chunks 11.8), 2 x 8192
// x 64 17.1 (12.0); backward, with half the threads, 2 x 2048 x 64 12.8 (13.6) and 2 x 4096 x 64
// 16.8 (13.7).
bool lay_out_whole(const gn_problem* p, int vec, int threads, int most, da::GnArgs& a) {
    const int64_t C = p->channels, elem = elem_bytes(p->x_dtype);
    const int64_t base = std::lcm(C / p->groups, (int64_t)vec);
    const bool small = p->batch * p->rows * C * elem <= (4 << 20) && p->rows <= 4 * threads;
    const auto vectors = [&](int64_t width, int t) {
        const int64_t R = t / (width / vec);
        return R ? (p->rows + R - 1) / R : INT64_MAX;
    };
    int64_t width = 0;
    for (int64_t w = base; w <= C && (w == base || w * elem <= 256); w *= 2) {
        if (vectors(w, threads) > most || w / (C / p->groups) > da::kGnUnits) break;
        if (w < C && w * elem < 64 && !small) continue;
        if (width && p->batch * ((C + w - 1) / w) < 256) break;
        width = w;
    }
    if (!width) return false;
    a.threads = 256;
    while (a.threads < threads && vectors(width, a.threads) > 4) a.threads *= 2;
    a.vecs = (int32_t)vectors(width, a.threads);
    a.slab_ch = (int32_t)width;
    a.upg = 1;
    a.cpu = a.cpg;
    a.slabs = (int32_t)((C + width - 1) / width);
    a.units = a.G;
    a.rows_per_chunk = a.S;
    a.chunks = 1;
    return true;
}

// What a pass can keep of a whole image's slab (threads 0: it goes by chunks).
struct Keeps {
    int threads, vecs;
};
constexpr Keeps kForward = {da::kGnWholeThreads, da::kGnWholeVecs};
// A grad_out of another type than x goes by chunks: 64 x 784 x 256 bfloat16 with a binary32
// gradient takes 44 us (115 MB), 33 with its own type (77 MB).
Keeps backward_keeps(const gn_problem* p) {
    return p->x_dtype == p->out_dtype ? Keeps{da::kGnWholeBwdThreads, da::kGnWholeBwdVecs}
                                      : Keeps{0, 0};
}

// The layout for vectors of `vec` channels (1, or 16 bytes' worth).
void lay_out(const gn_problem* p, int vec, Keeps keeps, da::GnArgs& a) {
    memset(&a, 0, sizeof a);
    const int64_t C = p->channels, cpg = C / p->groups, most = (int64_t)da::kGnThreads * vec;
    a.S = p->rows;
    a.N = (int32_t)p->batch;
    a.C = (int32_t)C;
    a.G = (int32_t)p->groups;
    a.cpg = (int32_t)cpg;
    a.share = 1.0 / ((double)a.S * (double)cpg);
    a.act = p->activation;
    a.x_dtype = p->x_dtype;
    a.out_dtype = p->out_dtype;
    a.eps = p->eps;
    if (keeps.threads && lay_out_whole(p, vec, keeps.threads, keeps.vecs, a)) return;
    const int64_t base = std::lcm(cpg, (int64_t)vec);
    if (base <= most) {
        // whole groups and whole vectors; 256 bytes of a row where that many fit
        const int64_t want = 256 / elem_bytes(p->x_dtype);
        a.slab_ch = (int32_t)std::min<int64_t>(
            std::min(most / base, std::max<int64_t>(1, want / base)) * base, C);
        a.upg = 1;
        a.cpu = (int32_t)cpg;
        a.slabs = (int32_t)((C + a.slab_ch - 1) / a.slab_ch);
        a.units = a.G;
    } else {
        a.cpu = a.slab_ch = (int32_t)std::min(most, cpg);
        a.upg = (int32_t)((cpg + a.cpu - 1) / a.cpu);
        a.slabs = a.units = a.G * a.upg;
    }
    // row chunks: 16 rows to a thread, fewer where that leaves less than two workgroups to a
    // compute unit.  More chunks than that cost more in every workgroup's join than they bring:
    // with eight to a compute unit 64 x 3136 x 128 bfloat16 takes 154 us backward (72), 1 x
    // 40000 x 256 67 forward (35).
    const int64_t R = std::max<int64_t>(1, da::kGnThreads / (a.slab_ch / vec));
    int64_t per_thread = 16;
    while (per_thread > 4 &&
           (int64_t)a.N * a.slabs * ((a.S + R * per_thread - 1) / (R * per_thread)) < 512)
        per_thread /= 2;
    int64_t rows = R * per_thread;
    constexpr int64_t kMaxChunks = 1024;   // read again by every workgroup of the image
    rows = std::max(rows, (a.S + kMaxChunks - 1) / kMaxChunks);
    a.rows_per_chunk = rows;
    a.chunks = (int32_t)((a.S + rows - 1) / rows);
}

// Whether vectors fit the problem (the pointers have their say as well).
bool vectors_fit(const gn_problem* p) {
    const int64_t vec = 16 / elem_bytes(p->x_dtype), C = p->channels, cpg = C / p->groups;
    if (C % vec) return false;
    return std::lcm(cpg, vec) <= da::kGnThreads * vec || cpg % vec == 0;
}

uint64_t stat_part_bytes(const da::GnArgs& a) {
    return part_bytes((uint64_t)a.N * a.chunks * a.units * sizeof(double2));
}
uint64_t unit_part_bytes(const da::GnArgs& a) {
    return part_bytes((uint64_t)a.N * a.chunks * a.units * sizeof(float2));
}
uint64_t chan_part_bytes(const da::GnArgs& a) {
    return part_bytes((uint64_t)a.N * a.chunks * a.C * sizeof(float2));
}

uint64_t group_bytes(const gn_problem* p) { return part_bytes((uint64_t)p->batch * p->groups * 4); }

// Workspace: forward, the chunks' statistics (and mean and rstd, for a caller that reads them
// from there); backward, the chunks' sums.  The larger of both layouts' needs, since the size
// is asked for before the pointers are known.
uint64_t need_forward(const gn_problem* p, bool stats_kept) {
    uint64_t need = 0;
    for (int vec : {1, 16 / elem_bytes(p->x_dtype)}) {
        if (vec > 1 && !vectors_fit(p)) continue;
        da::GnArgs a;
        lay_out(p, vec, kForward, a);
        need = std::max(need, (stats_kept ? 2 * group_bytes(p) : 0) +
                                  (a.threads ? 0 : group_bytes(p) + stat_part_bytes(a)));
    }
    return need;
}
uint64_t need_backward(const gn_problem* p) {
    uint64_t need = 0;
    for (int vec : {1, 16 / elem_bytes(p->x_dtype)}) {
        if (vec > 1 && !vectors_fit(p)) continue;
        da::GnArgs a;
        lay_out(p, vec, backward_keeps(p), a);
        need = std::max(need, chan_part_bytes(a) + (a.threads ? 0 : unit_part_bytes(a)));
    }
    return need;
}

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

// A launch has fewer than 2^32 threads (256 groups' joins take 64 workgroups).
da_status check_grid(const da::GnArgs& a) {
    const int64_t threads = a.threads ? a.threads : da::kGnThreads;
    if (((int64_t)a.N * a.chunks * a.slabs + a.C) * threads >= (int64_t(1) << 32) ||
        (int64_t)a.N * ((a.G + 3) / 4) * da::kGnThreads >= (int64_t(1) << 32))
        return report_error(DA_ERR_UNSUPPORTED, "2^32 threads of workgroups or more");
    return DA_OK;
}

}  // namespace

namespace da {

da_status gn_stats_bytes(const gn_problem* p, uint64_t& bytes) {
    const da_status st = check_problem(p);
    if (st != DA_OK) return st;
    for (int vec : {1, 16 / elem_bytes(p->x_dtype)}) {
        if (vec > 1 && !vectors_fit(p)) continue;
        GnArgs a;
        lay_out(p, vec, kForward, a);
        const da_status grid = check_grid(a);
        if (grid != DA_OK) return grid;
    }
    bytes = need_forward(p, true);
    return DA_OK;
}

hipError_t enqueue_gn_stats(const gn_problem* p, const void* x, void* workspace, GnArgs& a,
                            hipStream_t stream) {
    const bool vec = vectors_fit(p) && aligned(x, 16);
    lay_out(p, vec ? 16 / elem_bytes(p->x_dtype) : 1, kForward, a);
    unsigned char* base = static_cast<unsigned char*>(workspace);
    a.x = x;
    a.mean = reinterpret_cast<float*>(base);
    a.rstd = reinterpret_cast<float*>(base + group_bytes(p));
    a.origins = reinterpret_cast<float*>(base + 2 * group_bytes(p));
    a.stat_part = reinterpret_cast<double2*>(base + 3 * group_bytes(p));
    return launch_gn_stats(a, vec, stream);
}

}  // namespace da

extern "C" {

da_status gn_forward_workspace_size(const gn_problem* p, size_t* bytes) {
    if (!bytes) return report_error(DA_ERR_INVALID_ARG, "bytes is NULL");
    const da_status st = check_problem(p);
    if (st != DA_OK) return st;
    *bytes = (size_t)need_forward(p, false);
    return DA_OK;
}

da_status gn_forward(const gn_problem* p, const void* x, const float* weight, const float* bias,
                     void* out, float* mean, float* rstd, void* workspace, size_t workspace_bytes,
                     void* stream) {
    da_status st = check_problem(p);
    if (st != DA_OK) return st;
    if (p->batch == 0) return DA_OK;
    if (!x || !out) return report_error(DA_ERR_INVALID_ARG, "x / out is NULL");
    const int xb = elem_bytes(p->x_dtype), ob = elem_bytes(p->out_dtype);
    if (!aligned(x, xb) || !aligned(out, ob) || !aligned(weight, 4) || !aligned(bias, 4) ||
        !aligned(mean, 4) || !aligned(rstd, 4))
        return report_error(DA_ERR_INVALID_ARG, "a tensor is not element aligned");
    const int64_t n = p->batch * p->rows * p->channels;
    if (clash(x, n * xb, out, n * ob, p->x_dtype == p->out_dtype))
        return report_error(DA_ERR_INVALID_ARG, "out overlaps x without being x");
    const int wide = 16 / xb;
    const bool vec = vectors_fit(p) && aligned(x, 16) && aligned(out, std::min(16, wide * ob));
    da::GnArgs a;
    lay_out(p, vec ? wide : 1, kForward, a);
    st = check_grid(a);
    if (st != DA_OK) return st;
    st = check_workspace(need_forward(p, false), workspace, workspace_bytes);
    if (st != DA_OK) return st;
    a.x = x;
    a.weight = weight;
    a.bias = bias;
    a.out = out;
    a.mean = mean;
    a.rstd = rstd;
    a.origins = static_cast<float*>(workspace);
    if (!a.threads)
        a.stat_part = reinterpret_cast<double2*>(static_cast<unsigned char*>(workspace) + group_bytes(p));
    return da::report_hip(da::launch_gn_forward(a, vec, static_cast<hipStream_t>(stream)),
                          "group norm forward launch");
}

da_status gn_backward_workspace_size(const gn_problem* p, size_t* bytes) {
    if (!bytes) return report_error(DA_ERR_INVALID_ARG, "bytes is NULL");
    const da_status st = check_problem(p);
    if (st != DA_OK) return st;
    *bytes = (size_t)need_backward(p);
    return DA_OK;
}

da_status gn_backward(const gn_problem* p, const void* x, const void* grad_out, const float* mean,
                      const float* rstd, const float* weight, const float* bias, void* grad_x,
                      float* grad_weight, float* grad_bias, void* workspace,
                      size_t workspace_bytes, void* stream) {
    da_status st = check_problem(p);
    if (st != DA_OK) return st;
    const int xb = elem_bytes(p->x_dtype), ob = elem_bytes(p->out_dtype);
    if (p->batch > 0 && (!x || !grad_out || !mean || !rstd))
        return report_error(DA_ERR_INVALID_ARG, "x / grad_out / mean / rstd is NULL");
    if (!aligned(x, xb) || !aligned(grad_out, ob) || !aligned(grad_x, xb) || !aligned(weight, 4) ||
        !aligned(bias, 4) || !aligned(mean, 4) || !aligned(rstd, 4) || !aligned(grad_weight, 4) ||
        !aligned(grad_bias, 4))
        return report_error(DA_ERR_INVALID_ARG, "a tensor is not element aligned");
    const int64_t n = p->batch * p->rows * p->channels;
    if (grad_x && (clash(grad_x, n * xb, x, n * xb, false) ||
                   clash(grad_x, n * xb, grad_out, n * ob, p->x_dtype == p->out_dtype)))
        return report_error(DA_ERR_INVALID_ARG,
                            "grad_x overlaps x, or grad_out without being grad_out");
    const int wide = 16 / xb;
    const bool vec = vectors_fit(p) && aligned(x, 16) && aligned(grad_x, 16) &&
                     aligned(grad_out, std::min(16, wide * ob));
    da::GnArgs a;
    lay_out(p, vec ? wide : 1, backward_keeps(p), a);
    st = check_grid(a);
    if (st != DA_OK) return st;
    st = check_workspace(need_backward(p), workspace, workspace_bytes);
    if (st != DA_OK) return st;
    a.x = x;
    a.grad_out = grad_out;
    a.weight = weight;
    a.bias = bias;
    a.mean = const_cast<float*>(mean);
    a.rstd = const_cast<float*>(rstd);
    a.grad_x = grad_x;
    a.grad_weight = grad_weight;
    a.grad_bias = grad_bias;
    unsigned char* base = static_cast<unsigned char*>(workspace);
    a.chan_part = reinterpret_cast<float2*>(base);
    if (!a.threads) a.unit_part = reinterpret_cast<float2*>(base + chan_part_bytes(a));
    return da::report_hip(da::launch_gn_backward(a, vec, static_cast<hipStream_t>(stream)),
                          "group norm backward launch");
}

}  // extern "C"
