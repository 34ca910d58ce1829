/*
 * What stands around the products of a model that answers, on one MI355X
 * (gfx950): a whole mixture-of-experts layer for a few tokens; a linear layer
 * with a low-rank adapter per row; log probabilities of given tokens with entropy
 * and alternatives, and their gradient.
 *
 * Memory: every pointer is a device pointer of the caller's, aligned to its
 * element; outputs must not overlap inputs or one another, except where an
 * entry point says so.  The calls take their scratch memory from the caller
 * (workspace, 16-byte aligned, at least the bytes that the *_workspace_size
 * function of the same parameters returns; contents on entry do not matter);
 * the library allocates nothing and keeps nothing, so the calls may be captured
 * into HIP graphs, and calls with workspaces of their own may run at the same
 * time.  Results are bitwise reproducible: no sum's order depends on timing.
 *
 * Streams, threads, errors: as in gemm.h.  Argument checks come before any HIP
 * call: GEMM_ERR_INVALID_ARG for an unknown type or activation, negative sizes
 * or sizes above 2^30, a leading dimension shorter than its row or above 2^40, a
 * null or misaligned pointer of a non-empty operand, a workspace that is too
 * small, a call whose kernels would need 2^32 threads or more, and the limits named
 * below.  Calls without rows launch nothing.
 */
#ifndef DENSE_GEMM_03_AMD_GEMM_SERVING_H
#define DENSE_GEMM_03_AMD_GEMM_SERVING_H

#include "gemm_linear.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ----------------------------------------------------- mixture of experts --
 *
 * A whole layer for a few tokens, each of which goes to `top` of the experts:
 *
 *     h[t, j] = act(x_t . gate_e) * (x_t . up_e)      e = ids[t, j]    (gated)
 *     h[t, j] = act(x_t . up_e)                                        (not gated)
 *     y_t = sum_j weights[t, j] h[t, j] . down_e + residual_t
 *
 * w_up holds, per expert (stride_up elements apart), hidden x inner values, or
 * with a gate hidden x 2 inner: the gate's columns first.  w_down holds inner x
 * hidden per expert.  transw == GEMM_OP_T: both are stored transposed (2 inner x
 * hidden and hidden x inner).  ids (int32) and weights (fp32) are tokens x top,
 * contiguous, on the device and read by the kernels alone.  An id outside 0 ..
 * experts-1 counts for nothing, whatever its weight holds: padding, or an expert that
 * lives elsewhere; a token without experts gets its residual, or zeros.  Only the
 * weights of experts that a token names are read.
 *
 * Both products are formed as in gemm_linear; h is kept to 16 bits of mantissa
 * (bf16 operands) or as it is (fp32) between them, sums over experts are in fp32,
 * and y is rounded once, to dtype_y.  An expert that a token names twice counts
 * with the sum of the two weights.
 *
 * For a few tokens: at most 512, 32 experts each out of at most 1024, hidden and
 * inner at most 2^22, ldup and lddown at most 2^24.  An expert's weights are read once
 * per 64 tokens that name it: for long batches sort the rows by expert and use
 * gemm_linear.  An infinite value of w_down gives infinities or NaN.
 */
typedef struct {
    int32_t dtype;       /* of x, w_up and w_down: GEMM_DTYPE_F32 or GEMM_DTYPE_BF16 */
    int32_t dtype_y;     /* of y and residual */
    int32_t transw;      /* GEMM_OP_N or GEMM_OP_T */
    int32_t act;         /* gemm_act */
    int32_t gated;       /* 0 or 1 */
    int32_t reserved;    /* 0 */
    int64_t tokens, hidden, inner, experts, top;
    int64_t ldx, ldy, ldr;                 /* x, y, residual */
    int64_t ldup, lddown;                  /* w_up, w_down */
    int64_t stride_up, stride_down;        /* elements between consecutive experts */
} gemm_moe_params;

int64_t gemm_moe_layer_workspace_size(const gemm_moe_params *params);

/* residual may be NULL, or y itself with ldr == ldy. */
int gemm_moe_layer(const gemm_moe_params *params, const void *x, const void *w_up, const void *w_down,
                   const int32_t *ids, const float *weights, const void *residual, void *y,
                   void *workspace, int64_t workspace_bytes, hipStream_t stream);

/* ------------------------------------------------------ low-rank adapters --
 *
 * gemm_linear for the rows of many requests, each with a low-rank adapter of its
 * own beside the shared weights:
 *
 *     z = x . w + bias + scales[i] (x . a_i^T) . b_i^T      i = ids[row]
 *     y = act(z) + residual
 *
 * ids is int32, one per row, on the device and read by the kernels alone, in any
 * order (rows of a request side by side are fastest); an id outside 0 ..
 * adapters-1 leaves its row without an adapter.  a_i is rank x K and b_i N x rank,
 * row-major, stride_a and stride_b elements apart.  Adapters of a lower rank have
 * zeros in the rest.  scales (fp32, one per adapter) may be NULL: 1.  An adapter that
 * holds infinities or NaN makes infinities or NaN of its own rows alone (of a value in
 * b, in its column).
 *
 * Precision as in gemm_linear; x . a^T is formed in fp32 and kept to 16 bits of
 * mantissa (bf16 operands) or as it is (fp32) for the second product.
 *
 * Limits: rank at most 4096, lda at most 2^24.  gemm_linear_force_config holds
 * for these calls, too.
 */
typedef struct {
    int32_t dtype;       /* of x, w, a and b: GEMM_DTYPE_F32 or GEMM_DTYPE_BF16 */
    int32_t dtype_y;     /* of y and residual */
    int32_t dtype_bias;
    int32_t transw;      /* GEMM_OP_N: w is K x N; GEMM_OP_T: w is N x K */
    int32_t act;         /* gemm_act */
    int32_t reserved;    /* 0 */
    int64_t rows, N, K;
    int64_t adapters, rank;
    int64_t ldx, ldw, ldy, ldr;            /* x, w, y, residual */
    int64_t lda, ldb;                      /* a, b */
    int64_t stride_a, stride_b;            /* elements between consecutive adapters */
} gemm_adapter_params;

int64_t gemm_adapter_linear_workspace_size(const gemm_adapter_params *params);

/* bias and residual may be NULL; residual may be y itself with ldr == ldy. */
int gemm_adapter_linear(const gemm_adapter_params *params, const void *x, const void *w, const void *a,
                        const void *b, const int32_t *ids, const float *scales, const void *bias,
                        const void *residual, void *y, void *workspace, int64_t workspace_bytes,
                        hipStream_t stream);

/* ------------------------------------------------------ log probabilities --
 *
 * For each row z of logits (`vocab` values), with m its largest value,
 *
 *     d_j = scale (z_j - m)      L = log sum_j exp(d_j)      p_j = exp(d_j - L)
 *     logprob = d_token - L      entropy = L - sum_j p_j d_j
 *
 * and the `top` largest logits: their places, in falling order (equal logits:
 * the lower place first), and their log probabilities.  The distances are formed
 * before they are scaled, and m and L are kept apart, so that logits of any size
 * lose nothing; sums are in fp32.
 *
 * A token outside 0 .. vocab-1 (padding) has logprob 0 and no gradient through it.
 * -infinity is a forbidden place: p = 0, and it adds 0 to the entropy.  A row of
 * nothing else has logprob and L = -infinity, entropy 0 and gradient 0.  The type's
 * lowest value is a number like any other.  A row that holds NaN or +infinity has
 * NaN for logprob (of a token), entropy, m, L and the log probabilities of its
 * alternatives; NaN ranks with -infinity among the alternatives.
 */
typedef struct {
    int32_t dtype;   /* of the logits: GEMM_DTYPE_F32 or GEMM_DTYPE_BF16 */
    int32_t top;     /* alternatives: 0 .. 64, at most vocab */
    float scale;     /* 1 / temperature: > 0, at most 2^64 */
    int32_t reserved; /* 0 */
    int64_t rows, vocab;   /* vocab >= 1 */
    int64_t ld;      /* of the logits */
} gemm_log_probs_params;

int64_t gemm_log_probs_workspace_size(const gemm_log_probs_params *params);

/*
 * tokens: int32, one per row, or NULL with logprob NULL.  logprob, entropy: fp32,
 * one per row; stats: fp32, rows x 2, m and L; top_ids (int32) and top_logprobs
 * (fp32): rows x top.  Each output may be NULL and is then left out, but not
 * logprob with tokens, nor top_ids with top > 0.
 */
int gemm_log_probs(const gemm_log_probs_params *params, const void *logits, const int32_t *tokens,
                   float *logprob, float *entropy, float *stats, int32_t *top_ids, float *top_logprobs,
                   void *workspace, int64_t workspace_bytes, hipStream_t stream);

/*
 * dlogits = the gradient of sum over rows of dlogprob * logprob + dentropy * entropy:
 *
 *     dz_j = scale (dlogprob (1[j = token] - p_j) - dentropy p_j (log p_j + entropy))
 *
 * rounded once to the logits' type.  stats and entropy are gemm_log_probs' outputs
 * of the same logits and scale (top is not used).  dlogprob (with tokens) or
 * dentropy (with entropy) may be NULL: taken as zero.  dlogits has leading dimension
 * ldd and may be the logits themselves, with ldd == ld.  A row whose two factors
 * are zero has gradient 0 whatever its logits hold.
 */
int gemm_log_probs_grad(const gemm_log_probs_params *params, const void *logits, const int32_t *tokens,
                        const float *stats, const float *entropy, const float *dlogprob,
                        const float *dentropy, void *dlogits, int64_t ldd, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* DENSE_GEMM_03_AMD_GEMM_SERVING_H */
