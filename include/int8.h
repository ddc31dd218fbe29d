/*
 * int8.h -- matrix products of 8-bit integers with scales for each row and output
 * channel, in libdeformagg: the linear layers around the aggregation and the deformable
 * convolution (the layer that makes offset_mask, the one that makes the sampling
 * weights, 1x1 projections) as a model is served.
 *
 * Codes.  A row of K numbers x is held as whole numbers q in [-127, 127] and one binary32
 * scale, q * scale standing for x:
 *
 *   big = max |x|,  scale = big / 127,  q = nearest whole number of x * (127 / big)
 *
 * where both quotients and the product are binary32 numbers, rounded once each, and ties
 * of the nearest whole number go to the even one.  A row whose big is below 2^-100 (127 /
 * big would leave binary32 soon after) has scale 0 and codes 0.  A row that holds a NaN or
 * an infinity has scale NaN and codes 0, so that everything computed from it is NaN.
 * Weights [N, K] are held the same way, a scale per output channel.
 *
 * Products.  With a [M, K] and w [N, K] of codes (any 8-bit value, -128 too):
 *
 *   out[m, n] = act((sum_k a[m, k] * w[n, k]) * a_scale[m] * w_scale[n] + bias[n])
 *
 * the sum exact in 32-bit integers (K <= 131071), converted to binary32, then binary32
 * arithmetic, a 16-bit result rounded once to nearest even.
 *
 * Conventions of the library (see deformagg.h): the caller owns every buffer, calls
 * are asynchronous on `stream` and may be captured into a HIP graph, every check runs
 * on the host before anything is enqueued, da_last_error() names a failed check.  No
 * atomics on results: every result is the same bit for bit from run to run.
 */
#ifndef INT8_H
#define INT8_H

#include "deformagg.h"
#include "group_norm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Problem description.  rows may be 0 (nothing to do); in_channels in [1, 131071],
 * out_channels in [1, 2^24).  A launch has fewer than 2^32 threads, which bounds rows to
 * 2^26 with more than 256 input channels (2^27 to 2^29 with fewer) and rows times
 * out_channels to 2^36.  out must not overlap an input; x (the codes) and w are checked. */
typedef struct {
    int64_t rows;         /* M                                             */
    int64_t in_channels;  /* K                                             */
    int64_t out_channels; /* N                                             */
    int32_t activation;   /* da_activation of the result                   */
    int32_t x_dtype;      /* da_dtype of x (i8_matmul: must be 0)          */
    int32_t out_dtype;    /* da_dtype of out                               */
    int32_t flags;        /* must be 0                                     */
} i8_problem;

/*
 * i8_quantize_rows -- codes and scales of each row of x [rows, channels].
 *   x      device [rows, channels] of x_dtype, element aligned.
 *   codes  device int8 [rows, channels], fully overwritten; must not overlap x.
 *   scale  device float [rows], fully overwritten.
 */
DA_API da_status i8_quantize_rows(int64_t rows, int64_t channels, int32_t x_dtype, const void* x,
                                  int8_t* codes, float* scale, void* stream);

/* i8_matmul_workspace_size -- bytes of device workspace i8_matmul needs (0 for every
 * problem at present). */
DA_API da_status i8_matmul_workspace_size(const i8_problem* problem, size_t* bytes);

/*
 * i8_matmul -- out from codes, which may begin at any byte (large products are faster where a
 * and w are 16-byte aligned).
 *   a          device int8 [M, K].
 *   a_scale    device float [M].
 *   w          device int8 [N, K].
 *   w_scale    device float [N].
 *   bias       device float [N], or NULL.
 *   out        device [M, N] of out_dtype, element aligned, fully overwritten.
 *   workspace  device scratch of i8_matmul_workspace_size() bytes, 256-byte aligned (may
 *              be NULL when that is 0); contents on entry do not matter.
 * Errors: DA_ERR_INVALID_ARG, DA_ERR_UNSUPPORTED (more than 131071 input channels, rows or
 * output channels past the limits above), DA_ERR_HIP.
 */
DA_API da_status i8_matmul(const i8_problem* problem, const int8_t* a, const float* a_scale,
                           const int8_t* w, const float* w_scale, const float* bias, void* out,
                           void* workspace, size_t workspace_bytes, void* stream);

/* i8_linear_workspace_size -- bytes of device workspace i8_linear needs. */
DA_API da_status i8_linear_workspace_size(const i8_problem* problem, size_t* bytes);

/*
 * i8_linear -- i8_quantize_rows of x, then i8_matmul, as one call: the same numbers.
 *   x  device [M, K] of x_dtype, element aligned.  The rest as in i8_matmul.
 */
DA_API da_status i8_linear(const i8_problem* problem, const void* x, const int8_t* w,
                           const float* w_scale, const float* bias, void* out, void* workspace,
                           size_t workspace_bytes, void* stream);

/* i8_norm_linear_workspace_size -- bytes of device workspace i8_norm_linear needs. */
DA_API da_status i8_norm_linear_workspace_size(const gn_problem* problem, int64_t out_channels,
                                               size_t* bytes);

/*
 * i8_norm_linear -- group norm with its activation (group_norm.h), each normalised row
 * quantised from its binary32 values, then the product: out[n, s, :] of [N, S,
 * out_channels].  problem describes x, the groups, eps and the activation between norm and
 * product; problem->out_dtype is the type of out.  Fewer than 2^22 images
 * times runs of 224 output channels.
 *   x                         device [N, S, C] of x_dtype, element aligned.
 *   norm_weight, norm_bias    device float [C], or NULL, as in gn_forward.
 *   w, w_scale, bias          the projection's codes [out_channels, C], scales and bias
 *                             (or NULL), as in i8_matmul.
 *   out                       device [N, S, out_channels] of out_dtype, element aligned.
 *   workspace                 as above.
 */
DA_API da_status i8_norm_linear(const gn_problem* problem, int64_t out_channels, const void* x,
                                const float* norm_weight, const float* norm_bias, const int8_t* w,
                                const float* w_scale, const float* bias, void* out,
                                void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}  /* extern "C" */
#endif

#endif /* INT8_H */
