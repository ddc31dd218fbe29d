// Host side of the 8-bit products: argument checks, workspace layout, dispatch.  Every
// check runs before anything is enqueued.  Contract: include/int8.h.
#include <stdint.h>
#include <string.h>

#include "gn_internal.h"
#include "host_errors.h"
#include "i8_internal.h"
#include "int8.h"

namespace {

using da::report_error;

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }
bool valid_dtype(int32_t t) { return t == DA_F32 || t == DA_BF16 || t == DA_F16; }
int elem_bytes(int32_t t) { return t == DA_F32 ? 4 : 2; }
uint64_t part_bytes(uint64_t n) { return (n + 255) & ~uint64_t(255); }

constexpr int64_t kMostK = 131071;   // 2^14 (two -128) times this stays below 2^31

da_status check_sizes(int64_t M, int64_t K, int64_t N) {
    if (M < 0) return report_error(DA_ERR_INVALID_ARG, "rows must be >= 0");
    if (K < 1 || N < 1)
        return report_error(DA_ERR_INVALID_ARG, "in_channels and out_channels must be >= 1");
    if (K > kMostK)
        return report_error(DA_ERR_UNSUPPORTED, "in_channels > %lld", (long long)kMostK);
    if (M >= (int64_t(1) << 31) || N >= (int64_t(1) << 31))
        return report_error(DA_ERR_UNSUPPORTED, "2^31 rows or output channels or more");
    // a launch has fewer than 2^32 threads: 256 to 64 x 64 results, 512 to 16 output channels of
    // up to 256 rows in groups of 64, 64 or fewer to a row that is quantised
    const int64_t lanes = K <= 64 ? 8 : K <= 128 ? 16 : K <= 256 ? 32 : 64;
    if ((M + 63) / 64 * ((N + 63) / 64) >= (int64_t(1) << 24) || N >= (int64_t(1) << 24) ||
        M * lanes >= (int64_t(1) << 32) - 256)
        return report_error(DA_ERR_UNSUPPORTED,
                            "2^32 threads of workgroups or more (or 2^24 output channels)");
    return DA_OK;
}

da_status check_problem(const i8_problem* p, bool codes) {
    if (!p) return report_error(DA_ERR_INVALID_ARG, "problem is NULL");
    if (p->flags != 0) return report_error(DA_ERR_INVALID_ARG, "problem.flags must be 0");
    const da_status st = check_sizes(p->rows, p->in_channels, p->out_channels);
    if (st != DA_OK) return st;
    if (!valid_dtype(p->x_dtype) || !valid_dtype(p->out_dtype))
        return report_error(DA_ERR_INVALID_ARG, "x_dtype %d / out_dtype %d is not a da_dtype",
                            (int)p->x_dtype, (int)p->out_dtype);
    if (codes && p->x_dtype != 0)
        return report_error(DA_ERR_INVALID_ARG, "x_dtype must be 0 for codes");
    if (p->activation < DA_ACT_NONE || p->activation > DA_ACT_GELU)
        return report_error(DA_ERR_INVALID_ARG, "activation %d is not a da_activation",
                            (int)p->activation);
    return DA_OK;
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

// Paths whose product reads codes that were written to memory first.
bool through_memory(da::I8Path path) {
    return path == da::I8Path::kTiles || path == da::I8Path::kSkinnyCodes;
}

// Codes and scales of a quantised [M, K].
uint64_t codes_bytes(int64_t M, int64_t K) { return part_bytes((uint64_t)M * K); }
uint64_t quantised_bytes(int64_t M, int64_t K) { return codes_bytes(M, K) + part_bytes(M * 4); }

da::I8Args args_of(int64_t M, int64_t K, int64_t N, int32_t act, int32_t x_dtype, int32_t out_dtype) {
    da::I8Args a;
    memset(&a, 0, sizeof a);
    a.M = M;
    a.K = (int32_t)K;
    a.N = (int32_t)N;
    a.act = act;
    a.x_dtype = x_dtype;
    a.out_dtype = out_dtype;
    return a;
}

// out [M, N] shares a byte with an operand of so many bytes
da_status check_apart(const void* out, uint64_t out_bytes, const void* in, uint64_t in_bytes,
                      const char* name) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(out), y = reinterpret_cast<uintptr_t>(in);
    if (x < y + in_bytes && y < x + out_bytes)
        return report_error(DA_ERR_INVALID_ARG, "the result overlaps %s", name);
    return DA_OK;
}
da_status check_apart(int64_t M, int64_t K, int64_t N, const void* out, int32_t out_dtype,
                      const void* x, int x_bytes, const void* w) {
    const uint64_t bytes = (uint64_t)M * N * elem_bytes(out_dtype);
    const da_status st = check_apart(out, bytes, x, (uint64_t)M * K * x_bytes, "x");
    return st != DA_OK ? st : check_apart(out, bytes, w, (uint64_t)N * K, "w");
}

}  // namespace

extern "C" {

da_status i8_quantize_rows(int64_t rows, int64_t channels, int32_t x_dtype, const void* x,
                           int8_t* codes, float* scale, void* stream) {
    da_status st = check_sizes(rows, channels, 1);
    if (st != DA_OK) return st;
    if (!valid_dtype(x_dtype))
        return report_error(DA_ERR_INVALID_ARG, "x_dtype %d is not a da_dtype", (int)x_dtype);
    if (rows == 0) return DA_OK;
    if (!x || !codes || !scale)
        return report_error(DA_ERR_INVALID_ARG, "x / codes / scale is NULL");
    if (!aligned(x, elem_bytes(x_dtype)) || !aligned(scale, 4))
        return report_error(DA_ERR_INVALID_ARG, "x / scale is not element aligned");
    st = check_apart(codes, (uint64_t)rows * channels, x, (uint64_t)rows * channels * elem_bytes(x_dtype),
                     "x");
    if (st != DA_OK) return st;
    da::I8Args a = args_of(rows, channels, 1, DA_ACT_NONE, x_dtype, DA_F32);
    a.x = x;
    a.a = codes;
    a.a_scale = scale;
    return da::report_hip(da::launch_i8_quantize(a, nullptr, static_cast<hipStream_t>(stream)),
                          "row quantisation launch");
}

da_status i8_matmul_workspace_size(const i8_problem* p, size_t* bytes) {
    if (!bytes) return report_error(DA_ERR_INVALID_ARG, "bytes is NULL");
    const da_status st = check_problem(p, true);
    if (st != DA_OK) return st;
    *bytes = 0;
    return DA_OK;
}

da_status i8_matmul(const i8_problem* p, const int8_t* a_codes, const float* a_scale,
                    const int8_t* w, const float* w_scale, const float* bias, void* out,
                    void* workspace, size_t workspace_bytes, void* stream) {
    da_status st = check_problem(p, true);
    if (st != DA_OK) return st;
    if (p->rows == 0) return DA_OK;
    if (!a_codes || !a_scale || !w || !w_scale || !out)
        return report_error(DA_ERR_INVALID_ARG, "a / a_scale / w / w_scale / out is NULL");
    if (!aligned(a_scale, 4) || !aligned(w_scale, 4) || !aligned(bias, 4) ||
        !aligned(out, elem_bytes(p->out_dtype)))
        return report_error(DA_ERR_INVALID_ARG, "a tensor is not element aligned");
    st = check_apart(p->rows, p->in_channels, p->out_channels, out, p->out_dtype, a_codes, 1, w);
    if (st != DA_OK) return st;
    da::I8Args a = args_of(p->rows, p->in_channels, p->out_channels, p->activation, p->x_dtype,
                           p->out_dtype);
    a.a = const_cast<int8_t*>(a_codes);
    a.a_scale = const_cast<float*>(a_scale);
    a.w = w;
    a.w_scale = w_scale;
    a.bias = bias;
    a.out = out;
    const da::I8Path path = da::i8_path(a.M, a.K, a.N, true, false);
    return da::report_hip(
        da::launch_i8_product(a, path, true, nullptr, static_cast<hipStream_t>(stream)),
        "8-bit product launch");
}

da_status i8_linear_workspace_size(const i8_problem* p, size_t* bytes) {
    if (!bytes) return report_error(DA_ERR_INVALID_ARG, "bytes is NULL");
    const da_status st = check_problem(p, false);
    if (st != DA_OK) return st;
    const da::I8Path path = da::i8_path(p->rows, p->in_channels, p->out_channels, false, false);
    *bytes = through_memory(path) ? (size_t)quantised_bytes(p->rows, p->in_channels) : 0;
    return DA_OK;
}

da_status i8_linear(const i8_problem* p, const void* x, const int8_t* w, const float* w_scale,
                    const float* bias, void* out, void* workspace, size_t workspace_bytes,
                    void* stream) {
    size_t need = 0;
    da_status st = i8_linear_workspace_size(p, &need);
    if (st != DA_OK) return st;
    if (p->rows == 0) return DA_OK;
    if (!x || !w || !w_scale || !out)
        return report_error(DA_ERR_INVALID_ARG, "x / w / w_scale / out is NULL");
    if (!aligned(x, elem_bytes(p->x_dtype)) || !aligned(w_scale, 4) || !aligned(bias, 4) ||
        !aligned(out, elem_bytes(p->out_dtype)))
        return report_error(DA_ERR_INVALID_ARG, "a tensor is not element aligned");
    st = check_workspace(need, workspace, workspace_bytes);
    if (st != DA_OK) return st;
    st = check_apart(p->rows, p->in_channels, p->out_channels, out, p->out_dtype, x,
                     elem_bytes(p->x_dtype), w);
    if (st != DA_OK) return st;
    da::I8Args a = args_of(p->rows, p->in_channels, p->out_channels, p->activation, p->x_dtype,
                           p->out_dtype);
    a.x = x;
    a.w = w;
    a.w_scale = w_scale;
    a.bias = bias;
    a.out = out;
    const da::I8Path path = da::i8_path(a.M, a.K, a.N, false, false);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    hipError_t e = hipSuccess;
    if (through_memory(path)) {
        unsigned char* base = static_cast<unsigned char*>(workspace);
        a.a = reinterpret_cast<int8_t*>(base);
        a.a_scale = reinterpret_cast<float*>(base + codes_bytes(a.M, a.K));
        e = da::launch_i8_quantize(a, nullptr, s);
    }
    if (e == hipSuccess) e = da::launch_i8_product(a, path, false, nullptr, s);
    return da::report_hip(e, "8-bit linear launch");
}

da_status i8_norm_linear_workspace_size(const gn_problem* p, int64_t out_channels, size_t* bytes) {
    if (!bytes) return report_error(DA_ERR_INVALID_ARG, "bytes is NULL");
    uint64_t need = 0;
    da_status st = da::gn_stats_bytes(p, need);
    if (st != DA_OK) return st;
    const int64_t M = p->batch * p->rows;
    st = check_sizes(M, p->channels, out_channels);
    if (st != DA_OK) return st;
    // 512 threads or more to an image and a slice of the weights (224 output channels or more)
    if (p->batch * ((out_channels + 223) / 224) >= (int64_t(1) << 22))
        return report_error(DA_ERR_UNSUPPORTED,
                            "2^22 images times runs of 224 output channels, or more");
    if (through_memory(da::i8_path(M, p->channels, out_channels, false, true)))
        need += quantised_bytes(M, p->channels);
    *bytes = p->batch ? (size_t)need : 0;
    return DA_OK;
}

da_status i8_norm_linear(const gn_problem* p, int64_t out_channels, const void* x,
                         const float* norm_weight, const float* norm_bias, const int8_t* w,
                         const float* w_scale, const float* bias, void* out, void* workspace,
                         size_t workspace_bytes, void* stream) {
    size_t need = 0;
    da_status st = i8_norm_linear_workspace_size(p, out_channels, &need);
    if (st != DA_OK) return st;
    if (p->batch == 0) return DA_OK;
    if (!x || !w || !w_scale || !out)
        return report_error(DA_ERR_INVALID_ARG, "x / w / w_scale / out is NULL");
    if (!aligned(x, elem_bytes(p->x_dtype)) || !aligned(norm_weight, 4) || !aligned(norm_bias, 4) ||
        !aligned(w_scale, 4) || !aligned(bias, 4) || !aligned(out, elem_bytes(p->out_dtype)))
        return report_error(DA_ERR_INVALID_ARG, "a tensor is not element aligned");
    st = check_workspace(need, workspace, workspace_bytes);
    if (st != DA_OK) return st;
    const int64_t M = p->batch * p->rows;
    st = check_apart(M, p->channels, out_channels, out, p->out_dtype, x, elem_bytes(p->x_dtype), w);
    if (st != DA_OK) return st;
    da::I8Args a = args_of(M, p->channels, out_channels, DA_ACT_NONE, p->x_dtype, p->out_dtype);
    a.x = x;
    a.w = w;
    a.w_scale = w_scale;
    a.bias = bias;
    a.out = out;
    a.norm_weight = norm_weight;
    a.norm_bias = norm_bias;
    const da::I8Path path = da::i8_path(a.M, a.K, a.N, false, true);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    unsigned char* base = static_cast<unsigned char*>(workspace);
    if (through_memory(path)) {
        a.a = reinterpret_cast<int8_t*>(base);
        base += codes_bytes(a.M, a.K);
        a.a_scale = reinterpret_cast<float*>(base);
        base += part_bytes(a.M * 4);
    }
    da::GnArgs g;
    hipError_t e = da::enqueue_gn_stats(p, x, base, g, s);
    if (e == hipSuccess && through_memory(path)) e = da::launch_i8_quantize(a, &g, s);
    if (e == hipSuccess)
        e = da::launch_i8_product(a, path, false, through_memory(path) ? nullptr : &g, s);
    return da::report_hip(e, "normalised 8-bit linear launch");
}

}  // extern "C"
