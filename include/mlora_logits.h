/*
 * mlora_logits.h -- C ABI of libmlora.so: what a policy says of given tokens.
 * The log-probability of a token out of a row of logits with the row's entropy,
 * log-sum-exp and largest alternatives; the gradient of all of them in the
 * logits; and the same results for the rows of a transformer handle
 * (mlora_tf.h), whose logits are never stored whole.  The losses need the
 * target's log-probability (Deep Dive - Tinker, "The RL datum shape"); entropy
 * and alternatives are named by no page, so the definitions are the library's:
 *     z = scale * x                          x: a row of V logits
 *     lse = log sum_j exp(z_j),   p_j = exp(z_j - lse)
 *     logprob = z_y - lse                    y: the row's target
 *     entropy = -sum_j p_j log p_j           (p_j = 0 adds nothing)
 *     alternatives: the `top` largest x_j in falling order, of equal ones the
 *         lowest id first (-0 equals 0), each with z_j - lse
 * A logit of -infinity is a token that is not allowed: p_j = 0, its logprob is
 * -infinity, and it is no alternative.  Places without an alternative get id -1
 * and logprob -infinity.
 * A row whose logits are all -infinity has no distribution: lse = logprob =
 * -infinity, entropy 0, no alternatives.  A row with NaN or +infinity gets NaN in
 * all results and ids -1.
 * Sums and statistics are fp32: lse and the logprobs are off by about 2^-21 plus
 * 2^-22 of themselves, the entropy by 2^-21 plus 2^-21 of itself.  scale * x has to
 * lie within fp32's range.  Results repeat bit for bit; a row's do not depend on the other
 * rows' values, but their number and the vocabulary decide how many threads share a row,
 * and so the order of its sums.
 *
 * Conventions are those of mlora.h.  No call allocates or synchronises, so all
 * can be captured into a CUDA graph.
 */
#ifndef MLORA_LOGITS_H
#define MLORA_LOGITS_H

#include "mlora_tf.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Largest number of alternatives, and largest vocabulary. */
#define MLORA_LOGITS_MAX_TOP 32
#define MLORA_LOGITS_MAX_VOCAB (1 << 22)

/* Rows of logits (DEVICE). */
typedef struct {
    const void* logits;        /* n_rows rows of vocab elements of `dtype`, aligned to their elements  */
    const int32_t* targets;    /* [n_rows], or NULL: no targets.  -1: a row without one; any other id   */
                               /* outside 0 .. vocab-1 raises bit 0 of *status and counts as -1         */
    int32_t* status;           /* DEVICE int32 (may be NULL): bits raised by the kernels                */
    int64_t stride;            /* elements between rows, >= vocab                                       */
    int64_t n_rows;            /* >= 0                                                                  */
    int32_t vocab;             /* 1 .. MLORA_LOGITS_MAX_VOCAB                                           */
    int32_t dtype;             /* mlora_dtype                                                           */
    float scale;               /* 2^-20 .. 2^20 (one over the temperature)                              */
    int32_t top;               /* alternatives a row, 0 .. MLORA_LOGITS_MAX_TOP                         */
} mlora_logits;

/* Results (DEVICE, fp32 and int32); any may be NULL.  logprobs of a row without a
 * target is NaN. */
typedef struct {
    float* logprobs;           /* [n_rows]         */
    float* entropy;            /* [n_rows]         */
    float* lse;                /* [n_rows]         */
    int32_t* top_ids;          /* [n_rows x top]   */
    float* top_logprobs;       /* [n_rows x top]   */
} mlora_token_stats;

/* One pass over the logits.  Errors: E_ARG, E_CUDA. */
int mlora_token_logprobs(const mlora_logits* x, const mlora_token_stats* out, void* stream);

/* What the gradient needs (DEVICE): the forward's lse and entropy, and the
 * gradients of a loss in the results; any of these may be NULL (nothing comes
 * from that result), entropy where d_entropy is, top_ids where d_top is. */
typedef struct {
    const float* lse;          /* [n_rows]         */
    const float* entropy;      /* [n_rows]         */
    const int32_t* top_ids;    /* [n_rows x top]   */
    const float* d_logprobs;   /* [n_rows]; not read for a row without a target                  */
    const float* d_entropy;    /* [n_rows]         */
    const float* d_lse;        /* [n_rows]         */
    const float* d_top;        /* [n_rows x top]; not read where the id is -1                    */
} mlora_token_grads;

/* dlogits = the gradient in x, rounded once to x's type:
 *     dx_j = scale ( [j = y] d_logprob + sum_k [j = id_k] d_top_k
 *                    + p_j (d_lse - d_logprob - sum_k d_top_k) - d_entropy p_j (log p_j + entropy) )
 * p_j comes from the rounded lse and carries about 2^-22 (1 + |lse|) of itself.
 * A row whose incoming gradients are all 0, and a row without a distribution (lse =
 * -infinity), gets zeros whatever its logits; the row of an lse that is NaN otherwise NaN.
 * An id outside -1 .. vocab-1 raises bit 0 of *status and counts as -1; an id may
 * occur more than once in a row.  dlogits: rows of vocab elements of x's dtype,
 * out_stride apart; it is x->logits (with its stride) or none of its rows overlaps one of x.
 * Rows that do not lie like the logits' (addresses equal modulo 32 bytes) are read and written
 * an element at a time.
 * Errors: E_ARG, E_CUDA. */
int mlora_token_logprobs_backward(const mlora_logits* x, const mlora_token_grads* g, void* dlogits,
                                  int64_t out_stride, void* stream);

/* The results for the rows of a transformer batch: mlora_tf_forward, with the
 * LM head's logits held as fp32 a few thousand rows at a time in memory that the
 * handle already has.  scale and top as above.  logprobs are those of
 * mlora_tf_forward but for the order of the sums (at scale 1).  A token that
 * mlora_tf_forward flags gets NaN and ids -1.  b->targets may be NULL if
 * out->logprobs is.  Outputs [n_tokens] and [n_tokens x top].
 * Errors: E_ARG, E_CUDA. */
int mlora_tf_forward_stats(mlora_tf_t* h, const mlora_tf_batch* b, float scale, int32_t top,
                           const mlora_token_stats* out, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* MLORA_LOGITS_H */
