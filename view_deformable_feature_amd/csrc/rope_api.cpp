// Host side of the rotation and the head norm: argument checks, vectors and lanes of a head,
// dispatch.  Every check runs before anything is enqueued.  Contract: include/rotary.h.
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>

#include "host_errors.h"
#include "host_strides.h"
#include "rope_internal.h"
#include "rotary.h"

namespace {

using da::ranges_clash;
using da::report_error;

typedef da::wide_t wide;
constexpr int64_t k2to31 = int64_t(1) << 31;
constexpr int kMostDim = 512;

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }
int elem_bytes(int32_t t) { return t == DA_F32 ? 4 : 2; }
uint64_t part_bytes(uint64_t n) { return (n + 255) & ~uint64_t(255); }

wide extent(const int64_t (&stride)[3], const rope_tensor* t, int64_t D, int e) {
    return da::extent_bytes(stride, t->batch, t->tokens, t->heads, D, e);
}

da_status check_problem(const rope_problem* p, bool norm) {
    if (!p) return report_error(DA_ERR_INVALID_ARG, "problem is NULL");
    if ((p->flags & ~(norm ? 0 : ROPE_FLAG_INVERSE)) != 0 || p->reserved != 0)
        return report_error(DA_ERR_INVALID_ARG, "problem.flags has unknown bits, or reserved is not 0");
    if (p->head_dim < 1) return report_error(DA_ERR_INVALID_ARG, "head_dim must be >= 1");
    if (p->rotated < 0 || p->rotated > p->head_dim || p->rotated % 2 != 0)
        return report_error(DA_ERR_INVALID_ARG, "rotated (%lld) is not even and within head_dim (%lld)",
                            (long long)p->rotated, (long long)p->head_dim);
    if (p->dtype != DA_F32 && p->dtype != DA_BF16 && p->dtype != DA_F16)
        return report_error(DA_ERR_INVALID_ARG, "dtype %d is not a da_dtype", (int)p->dtype);
    if (p->layout != ROPE_LAYOUT_HALF && p->layout != ROPE_LAYOUT_INTERLEAVED)
        return report_error(DA_ERR_INVALID_ARG, "layout %d is not a rope_layout", (int)p->layout);
    if (!isfinite(p->magnitude)) return report_error(DA_ERR_INVALID_ARG, "magnitude must be finite");
    if (norm && (!isfinite(p->eps) || p->eps < 0.0f))
        return report_error(DA_ERR_INVALID_ARG, "eps must be finite and >= 0");
    if (p->head_dim > kMostDim) return report_error(DA_ERR_UNSUPPORTED, "head_dim > %d", kMostDim);
    return DA_OK;
}

da_status check_tensor(const rope_problem* p, const rope_tensor* t) {
    if (t->reserved != 0) return report_error(DA_ERR_INVALID_ARG, "tensor.reserved must be 0");
    if (t->batch < 0 || t->tokens < 0) return report_error(DA_ERR_INVALID_ARG, "batch and tokens must be >= 0");
    if (t->heads < 1) return report_error(DA_ERR_INVALID_ARG, "heads must be >= 1");
    if (t->pos_type < ROPE_POS_INDEX || t->pos_type > ROPE_POS_F32)
        return report_error(DA_ERR_INVALID_ARG, "pos_type %d is not a rope_pos_type", (int)t->pos_type);
    for (int i = 0; i < 3; ++i)
        if (t->x_stride[i] < 0 || t->y_stride[i] < 0 || t->x_stride[i] > (int64_t(1) << 56) ||
            t->y_stride[i] > (int64_t(1) << 56))
            return report_error(DA_ERR_INVALID_ARG, "a stride is negative or past 2^56");
    if (t->pos_stride < 0 || t->pos_stride > (int64_t(1) << 40))
        return report_error(DA_ERR_INVALID_ARG, "pos_stride is negative or past 2^40");
    if (t->batch >= k2to31 || t->tokens >= k2to31 || t->heads >= k2to31 ||
        (wide)t->batch * t->tokens >= k2to31 - 1024)
        return report_error(DA_ERR_UNSUPPORTED, "2^31 tokens of all batch entries, or heads");
    if ((wide)t->batch * t->tokens * t->heads * p->head_dim >= (wide)1 << 56)
        return report_error(DA_ERR_UNSUPPORTED, "2^56 numbers");
    const int e = elem_bytes(p->dtype);
    if (extent(t->x_stride, t, p->head_dim, e) >= (wide)1 << 62 ||
        extent(t->y_stride, t, p->head_dim, e) >= (wide)1 << 62)
        return report_error(DA_ERR_UNSUPPORTED, "a tensor spans 2^62 bytes or more");
    return DA_OK;
}

int pos_bytes(int32_t t) { return t == ROPE_POS_I64 ? 8 : 4; }

constexpr int64_t kWantedBlocks = 512;      // workgroups that each tensor of a launch should have
constexpr int64_t kBackwardBlocks = 512;    // that each of a backward launch has at most

bool empty(const rope_tensor* t) { return !t || t->batch == 0 || t->tokens == 0; }

// The largest vector, at most 16 bytes, that the sizes, strides and addresses allow.
struct Vectors {
    int vec;
    explicit Vectors(const rope_problem* p) : vec(16 / elem_bytes(p->dtype)) {
        fit(p->head_dim);
        if (p->layout == ROPE_LAYOUT_HALF) fit(p->rotated / 2);
    }
    void fit(int64_t n) {
        while (n % vec != 0) vec /= 2;
    }
    void fit(const rope_problem* p, const rope_tensor* t, const int64_t (&stride)[3], const void* at) {
        if (t->batch > 1) fit(stride[0]);
        if (t->tokens > 1) fit(stride[1]);
        if (t->heads > 1) fit(stride[2]);
        while (!aligned(at, vec * elem_bytes(p->dtype))) vec /= 2;
    }
};

// Lanes and units of a head.
int lay_out(const rope_problem* p, int vec, da::RopeArgs& a) {
    a.D = (int32_t)p->head_dim;
    a.R = (int32_t)p->rotated;
    a.eps = p->eps;
    a.magnitude = p->magnitude;
    a.sign = p->flags & ROPE_FLAG_INVERSE ? -1.0f : 1.0f;
    a.layout = p->layout;
    a.dtype = p->dtype;
    const int32_t turned = p->layout == ROPE_LAYOUT_HALF ? a.R / (2 * vec) : 0;
    a.units = turned + (a.D - turned * 2 * vec + 2 * vec - 1) / (2 * vec);
    a.lanes = 1;
    while (a.lanes < a.units && a.lanes < 64) a.lanes *= 2;
    const int per_lane = (a.units + a.lanes - 1) / a.lanes;
    return per_lane <= 1 ? 1 : per_lane <= 2 ? 2 : 4;
}

// A side's tensor and its workgroups: heads abreast so that a group of lanes has four or more of a
// token's to walk over, but up to all of them side by side where that leaves fewer than `want`
// workgroups.  A launch has fewer than 2^32 threads; the backward's workgroups walk over the tokens.
da_status share_out(const rope_tensor* t, const da::RopeArgs& a, bool backward, da::RopeSide& s) {
    s.tokens = t->batch * t->tokens;
    s.N = (int32_t)t->tokens;
    s.H = (int32_t)t->heads;
    s.pos_type = t->pos_type;
    s.pos_batch = t->pos_stride;
    s.x_batch = t->x_stride[0], s.x_token = t->x_stride[1], s.x_head = t->x_stride[2];
    s.y_batch = t->y_stride[0], s.y_token = t->y_stride[1], s.y_head = t->y_stride[2];
    const int64_t groups = da::kRopeThreads / a.lanes;
    s.abreast = 1;
    const auto blocks = [&] {
        const int64_t tokens = groups / s.abreast;
        return (s.tokens + tokens - 1) / tokens;
    };
    while (s.abreast * 2 <= std::min(groups, t->heads) &&
           (s.abreast * 8 <= t->heads || blocks() < kWantedBlocks))
        s.abreast *= 2;
    const int64_t n = blocks();
    if (!backward && n >= (int64_t(1) << 32) / da::kRopeThreads / 2)
        return report_error(DA_ERR_UNSUPPORTED, "2^31 threads of workgroups or more");
    s.blocks = (int32_t)(backward ? std::min(n, kBackwardBlocks) : n);
    return DA_OK;
}

// One tensor of a call.
struct Given {
    const char* name;
    const rope_tensor* t;
    const void *x, *positions;
    const float* weight;
    const void* y;        // the result; in the backward grad_y
    void* dx;
    float* grad_weight;
};

da::Heads of(const rope_problem* p, const rope_tensor* t, const void* at, const int64_t (&stride)[3]) {
    return {at, {t->batch, t->tokens, t->heads}, stride, p->head_dim, elem_bytes(p->dtype)};
}

da_status check_given(const rope_problem* p, const Given& g, const double* freqs, bool backward) {
    const int e = elem_bytes(p->dtype);
    if (!g.x || !g.y) return report_error(DA_ERR_INVALID_ARG, "%s or its other tensor is NULL", g.name);
    if (p->rotated > 0 && !freqs) return report_error(DA_ERR_INVALID_ARG, "freqs is NULL");
    if (g.t->pos_type != ROPE_POS_INDEX && p->rotated > 0 && !g.positions)
        return report_error(DA_ERR_INVALID_ARG, "positions of %s is NULL", g.name);
    if (!aligned(g.x, e) || !aligned(g.y, e) || !aligned(g.dx, e) || !aligned(g.weight, 4) ||
        !aligned(g.grad_weight, 4) || !aligned(freqs, 8) ||
        (g.t->pos_type != ROPE_POS_INDEX && !aligned(g.positions, pos_bytes(g.t->pos_type))))
        return report_error(DA_ERR_INVALID_ARG, "a tensor of %s is not element aligned", g.name);
    const wide nx = extent(g.t->x_stride, g.t, p->head_dim, e), ny = extent(g.t->y_stride, g.t, p->head_dim, e);
    if (!backward) {
        if (da::overlaps_itself(g.t->y_stride, g.t->batch, g.t->tokens, g.t->heads, p->head_dim))
            return report_error(DA_ERR_INVALID_ARG, "places of the result of %s overlap", g.name);
        const bool same = g.x == g.y && !memcmp(g.t->x_stride, g.t->y_stride, sizeof g.t->x_stride);
        if (!same && da::may_meet(of(p, g.t, g.x, g.t->x_stride), of(p, g.t, g.y, g.t->y_stride)))
            return report_error(DA_ERR_INVALID_ARG, "the result of %s overlaps it without being it", g.name);
        return DA_OK;
    }
    const wide nd = (wide)g.t->batch * g.t->tokens * g.t->heads * p->head_dim * e;
    const bool dense = g.t->y_stride[2] == p->head_dim && g.t->y_stride[1] == p->head_dim * g.t->heads &&
                       g.t->y_stride[0] == p->head_dim * g.t->heads * g.t->tokens;
    if (ranges_clash(g.dx, nd, g.x, nx) || (!(g.dx == g.y && dense) && ranges_clash(g.dx, nd, g.y, ny)))
        return report_error(DA_ERR_INVALID_ARG, "the gradient of %s overlaps an input", g.name);
    return DA_OK;
}

// Checks all of a call and fills in a launch; sides that have nothing to do are left out, but for
// weights' gradients, which are zeros then.
da_status set_up(const rope_problem* p, const Given (&given)[2], const double* freqs, bool norm,
                 bool backward, da::RopeArgs& a, int& vec, int& per_lane) {
    memset(&a, 0, sizeof a);
    da_status st = check_problem(p, norm);
    if (st != DA_OK) return st;
    Vectors v(p);
    for (const Given& g : given) {
        if (!g.t) continue;
        st = check_tensor(p, g.t);
        if (st != DA_OK) return st;
        const bool none = empty(g.t);
        if (none && !(backward && g.grad_weight)) continue;
        if (!none) {
            st = check_given(p, g, freqs, backward);
            if (st != DA_OK) return st;
            v.fit(p, g.t, g.t->x_stride, g.x);
            v.fit(p, g.t, g.t->y_stride, g.y);
            while (g.dx && !aligned(g.dx, v.vec * elem_bytes(p->dtype))) v.vec /= 2;
        }
        da::RopeSide& s = a.side[a.sides++];
        s.x = g.x;
        s.y = const_cast<void*>(g.y);
        s.dx = g.dx;
        s.positions = g.positions;
        s.weight = g.weight;
        s.grad_weight = g.grad_weight;
    }
    // results of one side over what the other reads or writes
    if (!empty(given[0].t) && !empty(given[1].t)) {
        const int e = elem_bytes(p->dtype);
        for (int i = 0; i < 2; ++i) {
            const Given &g = given[i], &o = given[1 - i];
            const auto bytes = [&](const Given& x) { return (wide)x.t->batch * x.t->tokens * x.t->heads * p->head_dim * e; };
            // a forward result may lie between the other's heads; the backward's are dense
            const auto meets = [&](const int64_t (&stride)[3], const void* at) {
                const da::Heads other = of(p, o.t, at, stride);
                return backward ? ranges_clash(g.dx, bytes(g), at, other.bytes())
                                : da::may_meet(of(p, g.t, g.y, g.t->y_stride), other);
            };
            if (meets(o.t->x_stride, o.x) || meets(o.t->y_stride, o.y) ||
                (backward && ranges_clash(g.dx, bytes(g), o.dx, bytes(o))))
                return report_error(DA_ERR_INVALID_ARG, "a result of %s overlaps a tensor of %s", g.name, o.name);
        }
    }
    vec = v.vec;
    per_lane = lay_out(p, vec, a);
    a.freqs = freqs;
    int at = 0;
    for (const Given& g : given) {
        if (!g.t || (empty(g.t) && !(backward && g.grad_weight))) continue;
        const da_status shared = share_out(g.t, a, backward, a.side[at++]);
        if (shared != DA_OK) return shared;
    }
    return DA_OK;
}

// Workgroups' sums of one side: as many as there may be, since the vectors are not known yet.
uint64_t need_of(const rope_problem* p, const rope_tensor* t) {
    return t ? part_bytes((uint64_t)kBackwardBlocks * p->head_dim * sizeof(float)) : 0;
}

}  // namespace

extern "C" {

da_status rope_forward(const rope_problem* p, const rope_tensor* t, const void* x, const void* positions,
                       const double* freqs, void* y, void* stream) {
    if (!t) return report_error(DA_ERR_INVALID_ARG, "tensor is NULL");
    const Given given[2] = {{"x", t, x, positions, nullptr, y, nullptr, nullptr}, {}};
    da::RopeArgs a;
    int vec, per_lane;
    const da_status st = set_up(p, given, freqs, false, false, a, vec, per_lane);
    if (st != DA_OK || a.sides == 0) return st;
    return da::report_hip(da::launch_rope(a, false, vec, per_lane, static_cast<hipStream_t>(stream)),
                          "rotation launch");
}

da_status rope_norm_forward(const rope_problem* p, const rope_tensor* qt, const void* q,
                            const void* q_positions, const float* q_weight, void* q_out,
                            const rope_tensor* kt, const void* k, const void* k_positions,
                            const float* k_weight, void* k_out, const double* freqs, void* stream) {
    const Given given[2] = {{"q", qt, q, q_positions, q_weight, q_out, nullptr, nullptr},
                            {"k", kt, k, k_positions, k_weight, k_out, nullptr, nullptr}};
    da::RopeArgs a;
    int vec, per_lane;
    const da_status st = set_up(p, given, freqs, true, false, a, vec, per_lane);
    if (st != DA_OK || a.sides == 0) return st;
    return da::report_hip(da::launch_rope(a, true, vec, per_lane, static_cast<hipStream_t>(stream)),
                          "head norm launch");
}

da_status rope_norm_backward_workspace_size(const rope_problem* p, const rope_tensor* qt,
                                            const rope_tensor* kt, size_t* bytes) {
    if (!bytes) return report_error(DA_ERR_INVALID_ARG, "bytes is NULL");
    da_status st = check_problem(p, true);
    for (const rope_tensor* t : {qt, kt})
        if (st == DA_OK && t) st = check_tensor(p, t);
    if (st != DA_OK) return st;
    *bytes = (size_t)(need_of(p, qt) + need_of(p, kt));
    return DA_OK;
}

da_status rope_norm_backward(const rope_problem* p, const rope_tensor* qt, const void* q,
                             const void* q_positions, const float* q_weight, const void* grad_q_out,
                             void* grad_q, float* grad_q_weight, const rope_tensor* kt, const void* k,
                             const void* k_positions, const float* k_weight, const void* grad_k_out,
                             void* grad_k, float* grad_k_weight, const double* freqs, void* workspace,
                             size_t workspace_bytes, void* stream) {
    const Given given[2] = {
        {"q", qt, q, q_positions, q_weight, grad_q_out, grad_q, grad_q_weight},
        {"k", kt, k, k_positions, k_weight, grad_k_out, grad_k, grad_k_weight}};
    da::RopeArgs a;
    int vec, per_lane;
    const da_status st = set_up(p, given, freqs, true, true, a, vec, per_lane);
    if (st != DA_OK || a.sides == 0) return st;
    uint64_t need = need_of(p, qt) + need_of(p, kt);
    if (!grad_q_weight && !grad_k_weight) need = 0;
    if (need) {
        if (!workspace) return report_error(DA_ERR_INVALID_ARG, "workspace is NULL");
        if (!aligned(workspace, 256))
            return report_error(DA_ERR_INVALID_ARG, "workspace is not 256-byte aligned");
        if (workspace_bytes < need)
            return report_error(DA_ERR_INVALID_ARG, "workspace has %zu bytes, %llu needed",
                                workspace_bytes, (unsigned long long)need);
        unsigned char* base = static_cast<unsigned char*>(workspace);
        for (int i = 0; i < a.sides; ++i) {
            a.side[i].part = reinterpret_cast<float*>(base);
            base += part_bytes((uint64_t)kBackwardBlocks * p->head_dim * sizeof(float));
        }
    }
    return da::report_hip(da::launch_rope_norm_backward(a, vec, per_lane, static_cast<hipStream_t>(stream)),
                          "head norm gradient launch");
}

}  // extern "C"
