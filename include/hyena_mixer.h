/*
 * hyena_mixer.h -- C ABI of the operators beside the gated FIR of hyena_conv.h in a mixer layer:
 * the gated linear recurrence (hyena_scan_*) and the projections (hyena_proj_*).
 *
 * Status codes, element types and the conventions on streams and buffers are those of
 * hyena_conv.h: DEVICE pointers, row-major contiguous tensors, buffers owned by the caller, no
 * device allocation, asynchronous on `stream`, argument errors found on the host before anything
 * is queued.  Outputs must not overlap inputs or each other unless an entry point says so.
 * Make the first call of each kind on a device before any stream capture (kernel attributes are
 * set then).  A timeout inside a kernel raises HYENA_DEVICE_TIMEOUT in the status word of
 * hyena_conv.h.
 */
#ifndef HYENA_MIXER_H
#define HYENA_MIXER_H

#include "hyena_conv.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Gated linear recurrence along time: the FIR operator's gates around a state that decays by a
 * factor of the data's choosing instead of a filter.
 *
 *     x_t = k_t v_t,   s_t = exp(g_t) s_{t-1} + x_t,   y_t = q_t s_t        (s_{-1} = s0 or 0)
 *
 * q, k, v, y: [B, L, D] of `dtype`.  g: [B, L, D / d_g] of `dtype`, the log decay of each token
 * and group of d_g contiguous channels (d_g = 1: one per channel), g <= 0; g = -inf drops the
 * state before the token (a reset, for packed sequences; a state that is not finite survives it,
 * 0 * inf being NaN).  For g > 0 the formula is evaluated, but a product of decays over a few
 * hundred tokens that leaves fp32's range gives inf or NaN.  s0: fp32 [B, D] or NULL.
 * s_out: fp32 [B, D], the state after the last token, or NULL.
 * ckpt: fp32 [B, hyena_scan_ckpt_tiles(L, dtype), D] or NULL: the states that hyena_scan_bwd
 * would otherwise find again by a pass over k, v and g.
 * The state is fp32 throughout; y is rounded once.  Sums have a fixed order: results are the
 * same in every call on one device.
 * Any B, L, D, d_g dividing D and element-aligned pointers.  Rows that are a multiple of 16 bytes
 * in 16-byte aligned tensors with d_g 1 or even are fastest (TMA); rows of 8 or 4 bytes come close;
 * odd D in bf16, or tensors on 2-byte boundaries, are read element by element.  L < 2^31 - 4096,
 * D <= 2^28.
 * workspace: at least hyena_scan_workspace_bytes(B, L, D, d_g, dtype) bytes, 16-byte aligned;
 * NULL where that is 0.
 * B == 0 or L == 0: nothing is launched, except that L == 0 copies s0 (zeros if NULL) to s_out.
 */
int hyena_scan_fwd(const void *q, const void *k, const void *v, const void *g, const float *s0,
                   void *y, float *s_out, float *ckpt, int64_t B, int64_t L, int64_t D, int d_g,
                   int dtype, void *workspace, size_t workspace_bytes, cudaStream_t stream);

/* Host-only: workspace of hyena_scan_fwd (a multiple of 256; 0 for most shapes), or minus
 * HYENA_ERR_INVALID_ARG. */
int64_t hyena_scan_workspace_bytes(int64_t B, int64_t L, int64_t D, int d_g, int dtype);

/* Host-only: time tiles of a checkpoint tensor, or minus HYENA_ERR_INVALID_ARG. */
int64_t hyena_scan_ckpt_tiles(int64_t L, int dtype);

/*
 * Gradients of hyena_scan_fwd for the upstream gradients dy (of y) and ds_out (of s_out, fp32
 * [B, D] or NULL):
 *
 *     u_t = q_t dy_t + exp(g_{t+1}) u_{t+1},   u_{L-1} += ds_out
 *     dq = dy s,  dk = u v,  dv = u k,  dg_t = sum over the group of exp(g_t) s_{t-1} u_t,
 *     ds0 = exp(g_0) u_0                               (ds0: fp32 [B, D] or NULL)
 *
 * dq, dk, dv, dg have the shapes and type of q, k, v, g and are overwritten.  ckpt: as written
 * by hyena_scan_fwd for the same inputs, or NULL.  workspace: at least
 * hyena_scan_bwd_workspace_bytes(..., have_ckpt) bytes, 16-byte aligned.
 * B == 0 or L == 0: nothing is launched, except that L == 0 copies ds_out (zeros if NULL) to ds0.
 */
int hyena_scan_bwd(const void *q, const void *k, const void *v, const void *g, const float *s0,
                   const void *dy, const float *ds_out, const float *ckpt, void *dq, void *dk,
                   void *dv, void *dg, float *ds0, int64_t B, int64_t L, int64_t D, int d_g,
                   int dtype, void *workspace, size_t workspace_bytes, cudaStream_t stream);

/* Host-only: workspace of hyena_scan_bwd (a multiple of 256), or minus HYENA_ERR_INVALID_ARG. */
int64_t hyena_scan_bwd_workspace_bytes(int64_t B, int64_t L, int64_t D, int d_g, int dtype,
                                       int have_ckpt);

/*
 * One token of B running sequences: q, k, v, y [B, D], g [B, D / d_g] of `dtype`; s, s_out fp32
 * [B, D], s_out = s allowed (the state advances in place).
 *     s_out = exp(g) s + k v,   y = q s_out
 */
int hyena_scan_step(const void *q, const void *k, const void *v, const void *g, const float *s,
                    void *y, float *s_out, int64_t B, int64_t D, int d_g, int dtype,
                    cudaStream_t stream);

enum hyena_act {
    HYENA_ACT_NONE = 0,
    HYENA_ACT_GELU = 1,          /* z Phi(z), the exact form (erf); at -inf NaN (inf times 0), as
                                    silu */
    HYENA_ACT_SILU = 2,          /* z sigmoid(z) */
    HYENA_ACT_SIGMOID = 3,
    HYENA_ACT_LOGSIGMOID = 4     /* log sigmoid(z): a log decay for hyena_scan_* */
};

/*
 * Projection: a matrix product with bias, activation and residual in its epilogue.
 *
 *     z[m][n] = sum_k x[m][k] w[n][k] + bias[n],     y = act(z) + residual
 *
 * x: [M, K], w: [N, K], residual, y, z: [M, N], all of `dtype`, 16-byte aligned.  bias: fp32 [N].
 * bias, residual and z may be NULL; z, where given, receives the value before the activation,
 * which hyena_proj_bwd wants (rounded to `dtype`).  y may be residual itself.
 * Any M >= 0, N, K >= 1 (M, N <= 2^30, K <= 2^24).  The products run on tensor cores with fp32
 * accumulation (which truncates: up to 2^-11 of sum |x| |w|, on sums of one sign): bf16 operands as
 * they are (rows that are no multiple of 8 elements are copied into the workspace first); fp32
 * operands as three bf16 planes each and six products, which keeps fp32's precision (relative to
 * sum |x| |w|) for finite operands that are 0 or at least 2^-110 in size.  bf16 ends at 2^-133: of
 * smaller ones what lies below 2^-134 is lost, at most 2^-133 (sum |x| + sum |w|) in all.  A product
 * with an infinite fp32 operand may give NaN in its place.
 * Bias, activation and residual are fp32, y is rounded once.  Deterministic.
 * workspace: at least hyena_proj_workspace_bytes(M, N, K, dtype) bytes, 256-byte aligned; NULL
 * where that is 0.
 */
int hyena_proj_fwd(const void *x, const void *w, const float *bias, const void *residual, void *y,
                   void *z, int64_t M, int64_t N, int64_t K, int act, int dtype, void *workspace,
                   size_t workspace_bytes, cudaStream_t stream);

/* Host-only: workspace of hyena_proj_fwd (a multiple of 256), or minus HYENA_ERR_INVALID_ARG, or
 * minus HYENA_ERR_UNSUPPORTED for more than 2^31 tiles of outputs (at most 256 x 256, in as many
 * cuts as K has pieces of 2^17), which the call refuses too. */
int64_t hyena_proj_workspace_bytes(int64_t M, int64_t N, int64_t K, int dtype);

/*
 * Gradients of hyena_proj_fwd for the upstream gradient dy [M, N] (the residual's is dy itself):
 *
 *     dz = dy act'(z),   dx = dz w (+ dx_add),   dw = dz^T x,   db[n] = sum_m dz[m][n]
 *
 * z: as the forward left it; NULL for HYENA_ACT_NONE.  dx_add: [M, K] or NULL, a gradient that
 * reaches x another way (the residual branch, another projection of x); dx may be dx_add itself.
 * dx [M, K], dw [N, K] of `dtype` and db fp32 [N] are overwritten; each may be NULL (x is not
 * read without dw, nor w without dx, and may then be NULL).  dz is rounded to `dtype` as an
 * operand of the products (db is not).  All tensors 16-byte aligned (db 4).  M == 0 zeroes dw and
 * db.  M up to 8388480 and N up to 2^24, else HYENA_ERR_UNSUPPORTED.  Deterministic.
 * workspace: at least hyena_proj_bwd_workspace_bytes(M, N, K, act, dtype) bytes, 256-byte aligned.
 */
int hyena_proj_bwd(const void *x, const void *w, const void *z, const void *dy,
                   const void *dx_add, void *dx, void *dw, float *db, int64_t M, int64_t N,
                   int64_t K, int act, int dtype, void *workspace, size_t workspace_bytes,
                   cudaStream_t stream);

/* Host-only: workspace of hyena_proj_bwd (a multiple of 256), or minus the error that the call
 * returns for such sizes. */
int64_t hyena_proj_bwd_workspace_bytes(int64_t M, int64_t N, int64_t K, int act, int dtype);

#ifdef __cplusplus
}
#endif

#endif /* HYENA_MIXER_H */
