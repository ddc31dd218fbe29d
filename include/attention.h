/*
 * attention.h -- attention of queries to keys and values of another length, in libdeformagg.
 *
 * q [B, Nq, H, D] are the queries of H heads, k and v [B, Nk, Hk, D] the states of Hk key
 * heads, H a multiple of Hk: query head h reads key head h / (H / Hk).  Key j of batch entry
 * b is visible if j < kv_lens[b] and key_mask[b, j] is not 0.  For each query i and head
 *
 *   s_j   = scale * sum over d of q[i, d] k[j, d],
 *   lse   = log of the sum over visible j of exp(s_j),
 *   p_j   = exp(s_j - lse),
 *   out_i = sum over visible j of p_j v[j].
 *
 * Without a visible key out is 0 and lse is -infinity.  What stands in invisible keys and
 * values, NaN or infinities too, reaches no result.  It is the attention of anchors to the
 * instances kept from earlier frames, or of a map's tokens to an encoder's, with one query a
 * batch entry as its serving form.
 *
 * Products of 16-bit types are exact and add up in binary32; scores, maxima, sums and results
 * under way are binary32, and a 16-bit result is rounded once to nearest even.  Weights come from
 * the scores' differences, so that large scores (within binary32 before `scale`) give weights as
 * small ones do.  In 16 bits the weights are rounded to q's type (bfloat16, binary16) before they
 * multiply v, and in the gradients so are p and p (dP - delta): a share of at most half a step of
 * each term, the same as the rounding of the result.  With at most 32 rows (queries times heads to
 * a key head) weights are carried in twice the digits.
 *
 * Conventions of the library (see deformagg.h): the caller owns every buffer, calls
 * are asynchronous on `stream` and may be captured into a HIP graph, every check runs
 * on the host before anything is enqueued, da_last_error() names a failed check.  No
 * atomics: every result is the same bit for bit from run to run.  A workspace belongs to one
 * call at a time.
 */
#ifndef ATTENTION_H
#define ATTENTION_H

#include "deformagg.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Problem description.  batch, queries and keys may be 0; heads, key_heads >= 1; heads %
 * key_heads == 0; head_dim a multiple of 8, at most 128; scale > 0, at most 2^126.  Strides count
 * elements, of a batch entry, a token and a head; a head's numbers are consecutive.  They are
 * >= 0 and multiples of 16 bytes (an input's batch stride may be 0: the same states for all). */
typedef struct {
    int64_t batch;       /* B                                             */
    int64_t queries;     /* Nq                                            */
    int64_t keys;        /* Nk                                            */
    int64_t heads;       /* H                                             */
    int64_t key_heads;   /* Hk                                            */
    int64_t head_dim;    /* D                                             */
    int64_t q_stride[3]; /* batch entry, token, head                      */
    int64_t k_stride[3];
    int64_t v_stride[3];
    int64_t out_stride[3];
    int64_t grad_stride[3]; /* of grad_out; not read by attn_forward        */
    float scale;
    int32_t dtype;       /* da_dtype of q, k, v, out and the gradients    */
    int32_t flags;       /* must be 0                                     */
    int32_t reserved;    /* must be 0                                     */
} attn_problem;

/* attn_forward_workspace_size -- bytes of device workspace attn_forward needs (0 where one
 * workgroup sees all keys of its queries).  Host only; refuses the problems that attn_forward
 * does. */
DA_API da_status attn_forward_workspace_size(const attn_problem* problem, size_t* bytes);

/*
 * attn_forward -- the formulas above.
 *   q, k, v    device, 16-byte aligned, with the problem's strides.
 *   kv_lens    device int32 [B], or NULL for Nk; below 0 counts as 0, above Nk as Nk.
 *   key_mask   device, one byte for each of [B, Nk], or NULL for all visible.
 *   out        device [B, Nq, H, D] with out_stride, 16-byte aligned, fully overwritten; its
 *              places must not overlap each other, nor q, k or v (it may lie between their
 *              heads in one packed buffer).
 *   lse        device float [B, H, Nq], dense, fully overwritten, for attn_backward; or NULL.
 *   workspace  device scratch of attn_forward_workspace_size() bytes, 256-byte aligned (may
 *              be NULL when that is 0); contents on entry do not matter.
 * Errors: DA_ERR_INVALID_ARG, DA_ERR_UNSUPPORTED (head_dim, strides of a token of 2^24 bytes or
 * more, 2^31 rows, 2^30 keys, a launch of 2^32 threads or more: 2^24 tiles of 128 rows of a key head,
 * or, with 32 rows or fewer, 2^23 key heads of all batch entries, 2^24 of more than 128 bytes),
 * DA_ERR_HIP.
 */
DA_API da_status attn_forward(const attn_problem* problem, const void* q, const void* k,
                              const void* v, const int32_t* kv_lens, const uint8_t* key_mask,
                              void* out, float* lse, void* workspace, size_t workspace_bytes,
                              void* stream);

/* attn_backward_workspace_size -- bytes of device workspace attn_backward needs.  Refuses the
 * problems that attn_backward does. */
DA_API da_status attn_backward_workspace_size(const attn_problem* problem, size_t* bytes);

/*
 * attn_backward -- with p as above and, for each query and head,
 * delta = sum over d of grad_out[i, d] out[i, d]:
 *
 *   dP_j    = sum over d of grad_out[i, d] v[j, d],
 *   dS_j    = p_j (dP_j - delta),
 *   grad_q  = scale * sum over visible j of dS_j k[j],
 *   grad_k  = scale * sum over i and the heads of the key head of dS_j q[i],
 *   grad_v  = sum over i and the heads of the key head of p_j grad_out[i].
 *
 * Gradients of invisible keys and of queries without a visible key are 0.  p is formed from lse,
 * which has the digits of binary32: it is off by a share of up to |lse| 2^-22, and where |lse|
 * passes 2^21 no more is known of it than that it is at most 1.
 *   out, lse   as attn_forward wrote them.
 *   grad_out   device [B, Nq, H, D] with grad_stride, 16-byte aligned.
 *   grad_q     device [B, Nq, H, D]; grad_k, grad_v device [B, Nk, Hk, D]; dense, 16-byte
 *              aligned, fully overwritten; grad_q may be NULL, grad_k and grad_v both may.  They
 *              must not overlap an input, from its first number to its last, or each other.
 *              With a batch stride of 0 each entry's part is written on its own: their sum is
 *              the gradient of the shared states.
 *   workspace  device scratch of attn_backward_workspace_size() bytes, 256-byte aligned;
 *              contents on entry do not matter.
 * Errors as attn_forward; the launch has a workgroup of 256 threads for each 128 rows, and for each
 * 128 keys, of a batch entry's key head, and for each split of few.
 */
DA_API da_status attn_backward(const attn_problem* problem, const void* q, const void* k,
                               const void* v, const void* out, const float* lse,
                               const void* grad_out, const int32_t* kv_lens,
                               const uint8_t* key_mask, void* grad_q, void* grad_k, void* grad_v,
                               void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}  /* extern "C" */
#endif

#endif /* ATTENTION_H */
