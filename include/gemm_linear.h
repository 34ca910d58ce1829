/*
 * Linear layers on one MI355X (gfx950): matrix products with bias, activation
 * and residual in their epilogue, dense or grouped by expert with ragged row
 * counts, and their gradients.  The products run on the matrix cores with the
 * precision of gemm.h: fp32 operands in true fp32, bf16 operands exactly, both
 * accumulated in fp32.
 *
 * The layer.  x has `rows` rows of K values, w is K x N (transw ==
 * GEMM_OP_N) or N x K (GEMM_OP_T), row-major with leading dimensions:
 *
 *     z = alpha * x . w + bias        y = act(z) + residual
 *
 * z is formed in fp32 and never rounded on the way to y; y (and z, where it is
 * asked for) are rounded once, to dtype_y.  bias, residual and pre (the stored
 * z) are optional: NULL leaves them out.
 *
 * Grouped by expert.  With groups > 0 the rows are sorted by group: rows
 * offsets[g] .. offsets[g+1]-1 of x, y, residual and pre belong to group g,
 * which has its own weights w + g * stride_w and bias + g * stride_bias.
 * offsets is a device array of groups + 1 int32, non-decreasing, within 0 ..
 * rows; it is read by the kernels alone (no host synchronisation), so the
 * counts may come from a router that still runs on the stream.  A group may be
 * empty.  Rows before offsets[0] and from offsets[groups] on belong to nobody:
 * their values are not used, and they are not written.  Values outside 0 .. rows
 * are clamped into it and a group that ends before it begins is taken as empty,
 * so no access leaves the arrays whatever offsets holds; with offsets that fall,
 * the results of the rows between the smallest and the largest of them are
 * undefined.  With groups == 0 there is one product over all rows, and offsets,
 * stride_w and stride_bias are not used.
 *
 * Gradients, for dy = the gradient of y:
 *
 *     dz = dy * act'(z)      dbias = sum of dz over the (group's) rows
 *     dx = alpha * dz . w^T  dw = alpha * x^T . dz        dresidual = dy
 *
 * gemm_linear_act_grad forms dz and dbias, gemm_linear_weight_grad dw, and dx
 * is gemm_linear on dz with the other transw (K and N exchanged, no
 * activation).  dz is stored in the operands' type, the type in which the two
 * products read it: for bf16 that is one rounding to nearest even; dbias sums
 * the values before it, in fp32.  That rounding adds as much to the error of
 * bf16 dx and dw as their own (0.0017 relative, in the norm, becomes 0.0023); a
 * caller who wants it left out passes dy, x and w as fp32 (dtype_dx and dtype_dw
 * may be bf16 all the same), at the rate of fp32 products.
 *
 * Results are bitwise reproducible: no atomics, fixed order of sums.
 *
 * Memory: every pointer is a device pointer of the caller's, aligned to its
 * element; outputs must not overlap inputs or one another, except that residual
 * may be y itself, and dz of gemm_linear_act_grad may be dy itself, with the same
 * leading dimension (GEMM_ERR_INVALID_ARG otherwise).  The calls take their
 * scratch memory from the caller (workspace, 16-byte aligned, at least the bytes
 * that the *_workspace_size function of the same parameters returns; contents on
 * entry do not matter); the library allocates nothing and keeps nothing, so the
 * calls may be captured into HIP graphs, and calls with workspaces of their own
 * may run at the same time.
 *
 * Streams, threads, errors: as in gemm.h.  Argument checks come before any HIP
 * call: GEMM_ERR_INVALID_ARG for an unknown type, activation or transposition,
 * negative sizes or sizes above 2^30, a leading dimension shorter than its row,
 * a null or misaligned pointer of a non-empty operand, a workspace that is too
 * small, or a call whose kernels would need 2^32 threads or more (from about
 * 2^39 outputs on, or groups x N of 2^30 in dbias).  rows == 0 or N == 0
 * launches nothing (the gradients of empty sums are still written: dw and dbias
 * of no rows are zeros, or beta * dw).
 */
#ifndef DENSE_GEMM_03_AMD_GEMM_LINEAR_H
#define DENSE_GEMM_03_AMD_GEMM_LINEAR_H

#include "gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* act(z); gelu is z Phi(z) with the error function, gelu_tanh its tanh form
 * z sigmoid(2 sqrt(2/pi) (z + 0.044715 z^3)), silu z sigmoid(z).  A NaN stays
 * a NaN. */
typedef enum {
    GEMM_ACT_NONE = 0,
    GEMM_ACT_RELU = 1,
    GEMM_ACT_GELU = 2,
    GEMM_ACT_GELU_TANH = 3,
    GEMM_ACT_SILU = 4
} gemm_act;

typedef struct {
    int32_t dtype;       /* of x, w, dy and dz: GEMM_DTYPE_F32 or GEMM_DTYPE_BF16 */
    int32_t dtype_y;     /* of y, residual and pre */
    int32_t dtype_bias;
    int32_t transw;      /* GEMM_OP_N: w is K x N; GEMM_OP_T: w is N x K */
    int32_t act;         /* gemm_act */
    float alpha;
    int64_t rows, N, K;
    int64_t groups;      /* 0: one product over all rows */
    int64_t ldx, ldw, ldy, ldr, ldp; /* x, w (and dw), y, residual, pre */
    int64_t stride_w;    /* elements between the weights of consecutive groups */
    int64_t stride_bias; /* elements between the biases of consecutive groups */
} gemm_linear_params;

/* Bytes of scratch memory gemm_linear needs for these parameters (0: none,
 * workspace may be NULL); GEMM_ERR_INVALID_ARG (negative) on bad ones. */
int64_t gemm_linear_workspace_size(const gemm_linear_params *params);

/* y = act(alpha * x . w + bias) + residual, and pre = alpha * x . w + bias. */
int gemm_linear(const gemm_linear_params *params, const void *x, const void *w,
                const int32_t *offsets, const void *bias, const void *residual, void *pre, void *y,
                void *workspace, int64_t workspace_bytes, hipStream_t stream);

/* Scratch of gemm_linear_act_grad: only rows, N and groups matter. */
int64_t gemm_linear_act_grad_workspace_size(const gemm_linear_params *params);

/*
 * dz = dy * act'(pre) and dbias (fp32, N values; with groups, groups x N) =
 * the sum of dz over rows.  dy and dz are rows x N of params->dtype with
 * leading dimensions lddy and lddz; pre is rows x N of dtype_y with ldp, and
 * not read (may be NULL) for GEMM_ACT_NONE.  dz may be NULL (only dbias is
 * formed) and may be dy itself (lddz == lddy); dbias may be NULL.
 */
int gemm_linear_act_grad(const gemm_linear_params *params, const void *dy, int64_t lddy,
                         const void *pre, const int32_t *offsets, void *dz, int64_t lddz,
                         float *dbias, void *workspace, int64_t workspace_bytes,
                         hipStream_t stream);

/* Scratch of gemm_linear_weight_grad. */
int64_t gemm_linear_weight_grad_workspace_size(const gemm_linear_params *params);

/*
 * dw := alpha * x^T . dz + beta * dw in the layout of w (K x N, or N x K with
 * transw; one per group, stride_w apart), of type dtype_dw.  dz is rows x N of
 * params->dtype with leading dimension ldy.  dw is not read when beta == 0.
 */
int gemm_linear_weight_grad(const gemm_linear_params *params, const void *x, const void *dz,
                            const int32_t *offsets, int dtype_dw, float beta, void *dw,
                            void *workspace, int64_t workspace_bytes, hipStream_t stream);

/* What gemm_linear_grad writes. */
typedef struct {
    int32_t dtype_dx, dtype_dw;
    float beta;          /* dw := .. + beta * dw */
    int32_t reserved;    /* 0 */
    int64_t lddx;        /* of dx, rows x K */
    int64_t lddw, stride_dw; /* of dw, in the layout of w */
} gemm_linear_grad_outputs;

/* Scratch of gemm_linear_grad for these outputs (dx, dw, dbias: 1 for those it
 * will be asked for, else 0). */
int64_t gemm_linear_grad_workspace_size(const gemm_linear_params *params,
                                        const gemm_linear_grad_outputs *outputs,
                                        int dx, int dw, int dbias);

/*
 * The whole backward pass: gemm_linear_act_grad, gemm_linear on dz and
 * gemm_linear_weight_grad in one call.  params describes the layer: dtype,
 * transw, act, alpha, sizes, ldx, ldw, stride_w; dtype_y and ldp are pre's, ldy
 * is dy's leading dimension (dy is of params->dtype).  dx, dw and dbias may each
 * be NULL and are then left out; pre is needed for an activation only.  dz lives
 * in the workspace.
 */
int gemm_linear_grad(const gemm_linear_params *params, const gemm_linear_grad_outputs *outputs,
                     const void *dy, const void *x, const void *w, const int32_t *offsets,
                     const void *pre, void *dx, void *dw, float *dbias, void *workspace,
                     int64_t workspace_bytes, hipStream_t stream);

/*
 * Kernel-table hooks, for tests and tuning: as the tile-table hooks of gemm.h.
 * gemm_linear_num_configs and gemm_linear_config_name list the entries of a
 * type; gemm_linear_config_forms has bit 0 / 1 set when the entry has kernels
 * for gemm_linear with transw N / T, bit 2 for gemm_linear_weight_grad.
 * gemm_linear_select_config (weight_grad 0 or 1) is the entry the dispatcher
 * uses.  gemm_linear_force_config makes the calling thread's next calls use
 * entry cfg with split_k slices of the summed axis (cfg < 0: the dispatcher's
 * choice again; split_k <= 0: the dispatcher's slices); a call whose form the
 * entry lacks returns GEMM_ERR_INVALID_ARG.
 */
int gemm_linear_num_configs(int dtype);
const char *gemm_linear_config_name(int dtype, int cfg);
int gemm_linear_config_forms(int dtype, int cfg);
int gemm_linear_select_config(const gemm_linear_params *params, int weight_grad);
int gemm_linear_force_config(int cfg, int split_k);

#ifdef __cplusplus
}
#endif

#endif /* DENSE_GEMM_03_AMD_GEMM_LINEAR_H */
