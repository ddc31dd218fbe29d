/*
 * rotary.h -- rotation of heads by the angles of their positions, and the head norm in the
 * same pass, in libdeformagg.
 *
 * x [B, N, H, D] are the heads of N tokens (queries or keys before an attention).  The first R
 * numbers of a head form R / 2 pairs: numbers i and i + R / 2 (half layout) or 2 i and 2 i + 1
 * (interleaved).  Token n of batch entry b has a position t, and pair i turns by the angle
 * t * freqs[i]:
 *
 *   c = magnitude * cos(t freqs[i]),  s = magnitude * sin(t freqs[i]),
 *   y_a = x_a c - x_b s,   y_b = x_b c + x_a s.
 *
 * Numbers from R on stay as they are.  With ROPE_FLAG_INVERSE the sign of s changes: the
 * rotation's transpose, which is its gradient.  Frequencies are binary64, and so are the
 * angles up to their place within a turn, so that far positions keep their digits; a position
 * is any number (an index, or a coordinate).  An angle of 2^52 and more, or none at all, makes its
 * pairs NaN.
 *
 * The head norm comes before the rotation: with
 *
 *   r = 1 / sqrt(average of x^2 over the D numbers + eps),   n = x r weight[d],
 *
 * n takes x's place.  Sums and numbers under way, x^2 among them, are binary32, a 16-bit result is
 * rounded once to nearest even.
 *
 * Conventions of the library (see deformagg.h): the caller owns every buffer, calls
 * are asynchronous on `stream` and may be captured into a HIP graph, every check runs
 * on the host before anything is enqueued, da_last_error() names a failed check.  No
 * atomics: every result is the same bit for bit from run to run.
 */
#ifndef ROTARY_H
#define ROTARY_H

#include "deformagg.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    ROPE_LAYOUT_HALF = 0,        /* pairs (i, i + R / 2)  */
    ROPE_LAYOUT_INTERLEAVED = 1  /* pairs (2 i, 2 i + 1)  */
} rope_layout;

typedef enum {
    ROPE_POS_INDEX = 0, /* token n has position n; positions NULL */
    ROPE_POS_I32 = 1,
    ROPE_POS_I64 = 2,   /* exact up to 2^53                       */
    ROPE_POS_F32 = 3
} rope_pos_type;

#define ROPE_FLAG_INVERSE 1

/* What queries and keys of one call share.  head_dim 1 to 512; rotated even, 0 to head_dim; eps
 * finite and >= 0; magnitude finite. */
typedef struct {
    int64_t head_dim;  /* D                                                     */
    int64_t rotated;   /* R                                                     */
    float eps;         /* head norm only                                        */
    float magnitude;
    int32_t layout;    /* rope_layout                                           */
    int32_t dtype;     /* da_dtype of x, y and their gradients                  */
    int32_t flags;     /* ROPE_FLAG_INVERSE (rope_forward only)                 */
    int32_t reserved;  /* must be 0                                             */
} rope_problem;

/* One tensor of heads.  batch and tokens may be 0; heads >= 1.  Strides count elements, of a
 * batch entry, a token and a head, and are >= 0; a head's numbers are consecutive. */
typedef struct {
    int64_t batch;       /* B                                                   */
    int64_t tokens;      /* N                                                   */
    int64_t heads;       /* H                                                   */
    int64_t x_stride[3]; /* of the input                                        */
    int64_t y_stride[3]; /* of the result; in rope_norm_backward, of grad_y     */
    int64_t pos_stride;  /* positions from one batch entry to the next, or 0    */
    int32_t pos_type;    /* rope_pos_type                                       */
    int32_t reserved;    /* must be 0                                           */
} rope_tensor;

/*
 * rope_forward -- the rotation of one tensor.
 *   x, positions (as pos_type says), y   device, element aligned.  y may be x itself with the
 *                                        same strides, or lie between x's heads in one packed
 *                                        buffer; it must not overlap x otherwise.
 *   freqs                                device double [R / 2] (may be NULL when R is 0).
 * Errors: DA_ERR_INVALID_ARG, DA_ERR_UNSUPPORTED (head_dim, 2^31 tokens or heads, a launch of 2^31
 * threads or more), DA_ERR_HIP.
 */
DA_API da_status rope_forward(const rope_problem* problem, const rope_tensor* tensor, const void* x,
                              const void* positions, const double* freqs, void* y, void* stream);

/*
 * rope_norm_forward -- head norm and rotation of queries and keys, in one launch.  Either tensor
 * may be left out (tensor NULL).
 *   weight    device float [D], or NULL for ones.
 *   others    as in rope_forward.
 */
DA_API da_status rope_norm_forward(const rope_problem* problem, const rope_tensor* q_tensor,
                                   const void* q, const void* q_positions, const float* q_weight,
                                   void* q_out, const rope_tensor* k_tensor, const void* k,
                                   const void* k_positions, const float* k_weight, void* k_out,
                                   const double* freqs, void* stream);

/* rope_norm_backward_workspace_size -- bytes of device workspace rope_norm_backward needs. */
DA_API da_status rope_norm_backward_workspace_size(const rope_problem* problem,
                                                   const rope_tensor* q_tensor,
                                                   const rope_tensor* k_tensor, size_t* bytes);

/*
 * rope_norm_backward -- with dn the inverse rotation of grad_y and xhat = x r:
 *
 *   grad_weight[d] = sum of dn[d] xhat[d] over batch entries, tokens and heads,
 *   grad_x[d]      = r (dn[d] weight[d] - xhat[d] * average over d of dn weight xhat).
 *
 *   q, k               the inputs of rope_norm_forward, with x_stride.
 *   grad_q_out, ..     device, with y_stride.
 *   grad_q, grad_k     device [B, N, H, D], dense, element aligned, fully overwritten, or NULL.
 *                      They may be the gradients that come in, where those are dense, and must
 *                      not overlap an input, from its first number to its last, otherwise.
 *   grad_q_weight, ..  device float [D], fully overwritten, or NULL; sums join in binary64.
 *   workspace          device scratch of rope_norm_backward_workspace_size() bytes, 256-byte
 *                      aligned (may be NULL when that is 0); contents on entry do not matter.
 */
DA_API da_status rope_norm_backward(const rope_problem* problem, const rope_tensor* q_tensor,
                                    const void* q, const void* q_positions, const float* q_weight,
                                    const void* grad_q_out, void* grad_q, float* grad_q_weight,
                                    const rope_tensor* k_tensor, const void* k,
                                    const void* k_positions, const float* k_weight,
                                    const void* grad_k_out, void* grad_k, float* grad_k_weight,
                                    const double* freqs, void* workspace, size_t workspace_bytes,
                                    void* stream);

#ifdef __cplusplus
}  /* extern "C" */
#endif

#endif /* ROTARY_H */
