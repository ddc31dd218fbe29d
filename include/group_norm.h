/*
 * group_norm.h -- group norm with an activation on channels-last maps, in libdeformagg.
 *
 * x [N, S, C] holds N images of S rows (pixels, in any order) of C channels; the C
 * channels form G groups of C / G consecutive ones.  For image n and group g
 *
 *   mean = the average of x over the S rows and the group's channels,
 *   var  = the average of (x - mean)^2 over the same values (their number, not one less),
 *   rstd = 1 / sqrt(var + eps),
 *   z    = (x - mean) * rstd * weight[c] + bias[c],
 *   out  = act(z),   act one of: z, max(z, 0), z / (1 + exp(-z)), z * Phi(z)
 *
 * with Phi the standard normal distribution function.  It is the norm that follows a
 * (deformable) convolution whose output is channels last, as dcn_forward's is: its
 * [N, H, W, C] is [N, H*W, C] here.  Means and variances are formed by averaging
 * deviations (never as a difference of large sums) and combined in binary64, as are the
 * gradients' sums over images and chunks; all other arithmetic is binary32, and a 16-bit
 * result is rounded once to nearest even.  A NaN, an infinity or a deviation whose square
 * overflows binary32 makes its whole (image, group) NaN, rstd among it, and deviations past
 * 2^46 may, by the sum of their squares; other groups are untouched by it.
 *
 * Conventions of the library (see deformagg.h): the caller owns every buffer, calls
 * are asynchronous on `stream` and may be captured into a HIP graph, every check runs
 * on the host before anything is enqueued, da_last_error() names a failed check.  No
 * atomics: every result is the same bit for bit from run to run.
 */
#ifndef GROUP_NORM_H
#define GROUP_NORM_H

#include "deformagg.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    DA_ACT_NONE = 0, /* z                                     */
    DA_ACT_RELU = 1, /* max(z, 0); derivative 0 at 0          */
    DA_ACT_SILU = 2, /* z / (1 + exp(-z))                     */
    DA_ACT_GELU = 3  /* z * Phi(z); Phi as computed is off by at most
                        (24 + 2 z^2) 2^-24 of itself                 */
} da_activation;

/* Problem description.  batch may be 0 (nothing to normalise); rows, channels and
 * groups >= 1; channels % groups == 0; eps finite and >= 0. */
typedef struct {
    int64_t batch;      /* N                                              */
    int64_t rows;       /* S: pixels of one image                         */
    int64_t channels;   /* C, at most 2^16                                */
    int64_t groups;     /* G                                              */
    float eps;
    int32_t activation; /* da_activation                                  */
    int32_t x_dtype;    /* da_dtype of x and grad_x                       */
    int32_t out_dtype;  /* da_dtype of out and grad_out                   */
    int32_t flags;      /* must be 0                                      */
    int32_t reserved;   /* must be 0                                      */
} gn_problem;

/* gn_forward_workspace_size -- bytes of device workspace gn_forward needs (0 where one
 * workgroup holds its share of an image on chip).  Host only. */
DA_API da_status gn_forward_workspace_size(const gn_problem* problem, size_t* bytes);

/*
 * gn_forward -- the formulas above.
 *   x          device [N, S, C] of x_dtype, element aligned.
 *   weight     device float [C], or NULL for ones.
 *   bias       device float [C], or NULL for zeros.
 *   out        device [N, S, C] of out_dtype, fully overwritten.  It may be x itself
 *              where the types agree; it must not overlap x otherwise.
 *   mean, rstd device float [N, G], fully overwritten, for gn_backward; either may be
 *              NULL.
 *   workspace  device scratch of gn_forward_workspace_size() bytes, 256-byte aligned (may
 *              be NULL when that is 0); contents on entry do not matter.
 * Errors: DA_ERR_INVALID_ARG, DA_ERR_UNSUPPORTED (more than 2^16 channels, a launch of 2^32
 * threads or more: about 2^24 images), DA_ERR_HIP.
 */
DA_API da_status gn_forward(const gn_problem* problem, const void* x, const float* weight,
                            const float* bias, void* out, float* mean, float* rstd,
                            void* workspace, size_t workspace_bytes, void* stream);

/* gn_backward_workspace_size -- bytes of device workspace gn_backward needs. */
DA_API da_status gn_backward_workspace_size(const gn_problem* problem, size_t* bytes);

/*
 * gn_backward -- with xhat = (x - mean) * rstd and dz = grad_out * act'(z):
 *
 *   grad_weight[c] = sum of dz * xhat over images and rows,
 *   grad_bias[c]   = sum of dz over images and rows,
 *   grad_x         = rstd * (weight[c] * dz - m1 - xhat * m2),
 *
 * m1 and m2 the averages over (rows, the group's channels) of weight[c] * dz and of
 * weight[c] * dz * xhat.
 *   grad_out     device [N, S, C] of out_dtype, element aligned.
 *   mean, rstd   device float [N, G], as gn_forward wrote them.
 *   weight, bias as in gn_forward.
 *   grad_x       device [N, S, C] of x_dtype, fully overwritten, or NULL.  It may be
 *                grad_out itself where the types agree, and must not overlap x or grad_out
 *                otherwise.
 *   grad_weight, grad_bias  device float [C], fully overwritten (zeros for batch 0), or
 *                NULL.
 *   workspace    device scratch of gn_backward_workspace_size() bytes, 256-byte aligned (may
 *                be NULL when that is 0); contents on entry do not matter.
 * Errors as gn_forward.
 */
DA_API da_status gn_backward(const gn_problem* problem, const void* x, const void* grad_out,
                             const float* mean, const float* rstd, const float* weight,
                             const float* bias, void* grad_x, float* grad_weight,
                             float* grad_bias, void* workspace, size_t workspace_bytes,
                             void* stream);

#ifdef __cplusplus
}  /* extern "C" */
#endif

#endif /* GROUP_NORM_H */
