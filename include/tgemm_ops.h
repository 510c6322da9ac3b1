/*
 * Operators around the matrix product of tgemm.h on AMD Instinct MI355X
 * (gfx950): the linear layer (bias, activation and residual in the product's
 * epilogue) with what its gradient needs, and the softmax cross entropy of a
 * product over a large vocabulary, with its gradient, without keeping the
 * logits. C ABI: plain pointers and sizes, no HIP or framework types.
 *
 * Operands are binary16 or bfloat16 (`type`: TGEMM_F16 or TGEMM_BF16), sums,
 * softmax statistics and epilogues are fp32. All arrays are row-major in device
 * memory with element strides between rows, at any alignment of their
 * elements. Sizes are 0 .. 2^31 - 1; a stride is at least the row length.
 *
 * Ownership, asynchrony and errors are those of tgemm.h: the caller owns every
 * buffer, the library allocates nothing and keeps no pointer, work is enqueued
 * on `stream`, and a call that returns TGEMM_ERR_INVALID or
 * TGEMM_ERR_UNSUPPORTED has enqueued nothing. An output must not overlap an
 * input or another output (exceptions are named). Inputs are only read.
 *
 * Workspaces: the *_workspace queries return the bytes a call with the same
 * arguments needs on the current device (16-byte aligned memory, contents
 * arbitrary before and undefined after; a negative value is a status). A call
 * with fewer workspace_bytes returns TGEMM_ERR_INVALID. A workspace may be used
 * again by any later work of the same stream.
 *
 * Results do not depend on timing: no atomics, every sum has a fixed order.
 */
#ifndef TGEMM_OPS_H_
#define TGEMM_OPS_H_

#include "tgemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Activations of the linear layer (0 and 1 as in tgemm_act):
 *   SILU       x / (1 + exp(-x))
 *   GELU       x/2 (1 + erf(x / sqrt 2))
 *   GELU_TANH  x/2 (1 + tanh(sqrt(2/pi) (x + 0.044715 x^3))) */
enum { TGEMM_ACT_SILU = 2, TGEMM_ACT_GELU = 3, TGEMM_ACT_GELU_TANH = 4 };

/*
 * Y = act(alpha * X * W + bias) + residual.
 *   X: M x K; W: w_layout TGEMM_B_NxK (N x K, a layer's weight) or TGEMM_B_KxN;
 *   Y: M x N of y_type (`type` or TGEMM_F32).
 *   bias: NULL or N values of bias_type (`type` or TGEMM_F32).
 *   residual: NULL or M x N of `type`; it may be Y itself (same pointer, stride
 *             and type).
 *   pre: NULL or M x N of `type` that receives alpha * X * W + bias, what
 *        tgemm_act_grad needs. It is rounded to 16 bits: a rounding of the
 *        values the activation's derivative is taken at, in return for half the
 *        bytes kept from the forward to the backward pass.
 * Rows of the residual and of pre lie at most 4,000,000 elements apart
 * (TGEMM_ERR_UNSUPPORTED otherwise), or at any distance where N is more than
 * that; X, W and Y may have any stride.
 * In fp32 after the fp32 sums: v = alpha * sum + bias (one fused multiply-add),
 * v = act(v) + residual, one rounding to y_type.
 * K == 0: the sums are zero. M == 0 or N == 0: nothing is done.
 *
 * Launch: up to 32 rows of X with W stored N x K read the weight once through a
 * kernel of their own, small products of up to 1024 rows once per 32 of them;
 * otherwise tiles of 256, 128 or 64 rows, with the K axis split and joined where
 * the tiles are too few for the device.
 */
int64_t tgemm_linear_workspace(int64_t M, int64_t N, int64_t K, int type, int64_t ldx, int64_t ldw, int w_layout,
                               int y_type, int64_t ldy);
int tgemm_linear(int64_t M, int64_t N, int64_t K, int type, const void* X, int64_t ldx, const void* W, int64_t ldw,
                 int w_layout, const void* bias, int bias_type, int act, const void* residual, int64_t ldr, int y_type,
                 void* Y, int64_t ldy, void* pre, int64_t ldpre, float alpha, void* workspace, int64_t workspace_bytes,
                 void* stream);

/*
 * The same with explicit launch choices, for tests and tuning.
 *   tile_m: 0 automatic, 256, 128 or 64 tile rows, 16 the kernel for few rows
 *           (M <= 1024, W stored N x K), 1 the general path (any stride).
 *   k_step: 0 automatic, or the tiles' K step: 64 (K > 64), or 32 (128 and 64
 *           rows).
 *   splits: 0 automatic, or 1..64 parts of the K axis (fewer where a part would
 *           hold 64 or less).
 * A choice that does not exist for the problem returns TGEMM_ERR_UNSUPPORTED.
 */
int64_t tgemm_linear_config_workspace(int64_t M, int64_t N, int64_t K, int type, int64_t ldx, int64_t ldw, int w_layout,
                                      int y_type, int64_t ldy, int tile_m, int k_step, int splits);
int tgemm_linear_config(int64_t M, int64_t N, int64_t K, int type, const void* X, int64_t ldx, const void* W,
                        int64_t ldw, int w_layout, const void* bias, int bias_type, int act, const void* residual,
                        int64_t ldr, int y_type, void* Y, int64_t ldy, void* pre, int64_t ldpre, float alpha,
                        void* workspace, int64_t workspace_bytes, void* stream, int tile_m, int k_step, int splits);

/*
 * C = alpha * A^T * B (+ C where accumulate is 1): A is K x M, B is K x N, both
 * row-major over the long axis K, as the activations and gradients of a layer
 * lie (the layer's weight gradient). C: M x N of c_type (`type` or TGEMM_F32),
 * rounded once. tile_m, k_step, splits: 0, or launch choices as above (tiles of
 * 256, 128 or 64 rows).
 */
int64_t tgemm_tn_workspace(int64_t M, int64_t N, int64_t K, int type, int64_t lda, int64_t ldb, int c_type, int64_t ldc,
                           int tile_m, int k_step, int splits);
int tgemm_tn(int64_t M, int64_t N, int64_t K, int type, const void* A, int64_t lda, const void* B, int64_t ldb,
             int c_type, void* C, int64_t ldc, float alpha, int accumulate, void* workspace, int64_t workspace_bytes,
             void* stream, int tile_m, int k_step, int splits);

/*
 * dP = dY * act'(pre), M x N of `type`, and (dbias not NULL) dbias[j] = sum over
 * rows of dY * act'(pre), before the rounding to dP's type, of dbias_type
 * (`type` or TGEMM_F32). act TGEMM_ACT_NONE: pre and dP must be NULL (dP is dY)
 * and only dbias is computed. The rectifier's derivative at zero is zero.
 */
int64_t tgemm_act_grad_workspace(int64_t M, int64_t N);
int tgemm_act_grad(int64_t M, int64_t N, int type, const void* dY, int64_t lddy, int act, const void* pre, int64_t ldpre,
                   void* dP, int64_t lddp, int dbias_type, void* dbias, void* workspace, int64_t workspace_bytes,
                   void* stream);

/*
 * Gradients of tgemm_linear (alpha = 1) in one call: with dP = dY * act'(pre)
 * (dY where act is TGEMM_ACT_NONE: pre must be NULL then), rounded to `type` as
 * an operand of both products,
 *   dX = dP * W^T (M x K), dW = dP^T * X in W's layout (N x K, or X^T * dP, K x N),
 *   dbias = the column sums of dP before its rounding, of dbias_type.
 * Each is rounded once; dX, dW and dbias may be NULL. The residual's gradient
 * is dY itself.
 */
int64_t tgemm_linear_grad_workspace(int64_t M, int64_t N, int64_t K, int type, int64_t ldx, int64_t ldw, int w_layout,
                                    int act, int64_t lddy, int64_t lddx, int64_t lddw);
int tgemm_linear_grad(int64_t M, int64_t N, int64_t K, int type, const void* X, int64_t ldx, const void* W, int64_t ldw,
                      int w_layout, int act, const void* pre, int64_t ldpre, const void* dY, int64_t lddy, void* dX,
                      int64_t lddx, void* dW, int64_t lddw, int dbias_type, void* dbias, void* workspace,
                      int64_t workspace_bytes, void* stream);

/*
 * tgemm_act_grad and tgemm_linear_grad for a dY in fp32 (an fp32 Y's gradient),
 * which is rounded once, as dP, after the product with act'(pre); dbias sums
 * values that were not rounded. Binary16 would lose values below 2^-25 and above
 * 65504: dP is multiplied there by the power of two 1 / *scale that takes the
 * largest finite |dY| into [2^14, 2^15) (bfloat16: *scale is 1).
 *   tgemm_act_grad_f32: dP = dY * act'(pre) / *scale, or NULL where only dbias is
 *     wanted; scale: one fp32 in device memory, NULL where dP is; it is not
 *     written where M or N is 0. TGEMM_ACT_NONE: pre must be NULL, dP is dY / *scale.
 *   tgemm_linear_grad_f32: the factor is undone in fp32 at the end of both
 *     products, before the one rounding of dX and dW.
 */
int64_t tgemm_act_grad_f32_workspace(int64_t M, int64_t N);
int tgemm_act_grad_f32(int64_t M, int64_t N, int type, const float* dY, int64_t lddy, int act, const void* pre,
                       int64_t ldpre, void* dP, int64_t lddp, float* scale, int dbias_type, void* dbias, void* workspace,
                       int64_t workspace_bytes, void* stream);
int64_t tgemm_linear_grad_f32_workspace(int64_t M, int64_t N, int64_t K, int type, int64_t ldx, int64_t ldw, int w_layout,
                                        int act, int64_t lddy, int64_t lddx, int64_t lddw);
int tgemm_linear_grad_f32(int64_t M, int64_t N, int64_t K, int type, const void* X, int64_t ldx, const void* W,
                          int64_t ldw, int w_layout, int act, const void* pre, int64_t ldpre, const float* dY,
                          int64_t lddy, void* dX, int64_t lddx, void* dW, int64_t lddw, int dbias_type, void* dbias,
                          void* workspace, int64_t workspace_bytes, void* stream);

/* Reduction of tgemm_xent's row losses. */
enum { TGEMM_REDUCE_NONE = 0, TGEMM_REDUCE_SUM = 1, TGEMM_REDUCE_MEAN = 2 };

/*
 * Softmax cross entropy of the logits z = H * W^T (H: rows x dim, W: vocab x
 * dim, target: rows int64), which are never stored:
 *   lse[i]  = log sum_v exp(z_iv)                                  (rows fp32)
 *   loss[i] = lse[i] - z_i,target(i), 0 where target(i) == ignore  (rows fp32)
 * reduction SUM or MEAN: also total = the sum of the losses, for MEAN divided
 * by count = the number of rows whose target is not `ignore`, at least 1 (no
 * such row: the mean is 0); `total` and `count` are one fp32 each, both written
 * for SUM and MEAN, NULL for NONE. A target outside the vocabulary that is not
 * `ignore` gives a loss of NaN; it is never used as an index.
 * dim >= 8, rows and vocab >= 1 (rows == 0 does nothing; SUM and MEAN then
 * return TGEMM_ERR_INVALID). vocab * 4 bytes must fit in 31 bits. Rows of H and W
 * (and of dH and dW in the calls below) lie at most 4,000,000 elements apart,
 * TGEMM_ERR_UNSUPPORTED otherwise.
 */
int64_t tgemm_xent_workspace(int64_t rows, int64_t vocab, int64_t dim, int type, int64_t ldh, int64_t ldw);
int tgemm_xent(int64_t rows, int64_t vocab, int64_t dim, int type, const void* H, int64_t ldh, const void* W,
               int64_t ldw, const int64_t* target, int64_t ignore, int reduction, float* lse, float* loss, float* total,
               float* count, void* workspace, int64_t workspace_bytes, void* stream);

/*
 * Gradient of tgemm_xent: with G = (g_i + e_i) softmax(z_i) - g_i onehot(target)
 * (e_i softmax(z_i) for an ignored row), dH = G * W and dW = G^T * H, each
 * rounded once to `type`. G is recomputed from lse in pieces of the vocabulary,
 * rounded to 16 bits as an operand of both products (after a division by its
 * largest factor that is undone in fp32).
 *   dloss: rows fp32 (dloss_stride 1), or one value for all rows (stride 0);
 *          NULL counts as zeros. g_i = dloss_i, divided by *count where count is
 *          not NULL (the mean).
 *   dlse:  NULL or rows fp32, the gradient e of lse.
 * dH or dW may be NULL. A row whose G is zero (ignored, no dlse) still meets
 * dW's product as 0 * h: its hidden state has to be finite. A target outside
 * the vocabulary gives NaN.
 */
int64_t tgemm_xent_grad_workspace(int64_t rows, int64_t vocab, int64_t dim, int type, int64_t ldh, int64_t ldw,
                                  int64_t lddh, int64_t lddw);
int tgemm_xent_grad(int64_t rows, int64_t vocab, int64_t dim, int type, const void* H, int64_t ldh, const void* W,
                    int64_t ldw, const int64_t* target, int64_t ignore, const float* lse, const float* dloss,
                    int dloss_stride, const float* count, const float* dlse, void* dH, int64_t lddh, void* dW,
                    int64_t lddw, void* workspace, int64_t workspace_bytes, void* stream);

/*
 * tgemm_xent and its gradients for a loss gradient of 1 in one call, without
 * computing the logits a second time: dH and dW (each may be NULL) as
 * tgemm_xent_grad gives them for total (dloss 1, `count` for the mean). The
 * exponentials of the logits, 16 bits, live in the workspace (2 bytes each for
 * rows times vocab rounded up to an odd multiple of 64: as much as 16-bit logits
 * take) and become the coefficients there: each is rounded twice to 16 bits, but
 * for the target's.
 * bfloat16 only, reduction SUM or MEAN, at most 2^30 of them (rows times the
 * rounded vocab) and 4,000,000 a row: TGEMM_ERR_UNSUPPORTED otherwise. rows >= 1.
 */
int64_t tgemm_xent_both_workspace(int64_t rows, int64_t vocab, int64_t dim, int type, int64_t ldh, int64_t ldw,
                                  int64_t lddh, int64_t lddw);
int tgemm_xent_both(int64_t rows, int64_t vocab, int64_t dim, int type, const void* H, int64_t ldh, const void* W,
                    int64_t ldw, const int64_t* target, int64_t ignore, int reduction, float* lse, float* loss, float* total,
                    float* count, void* dH, int64_t lddh, void* dW, int64_t lddw, void* workspace,
                    int64_t workspace_bytes, void* stream);

/* X *= *factor and X2 *= *factor in place: n and n2 contiguous values of `type`
 * at 16-byte alignment (n2 0, X2 NULL: one array), the factor one fp32 in device
 * memory, each product rounded once. A factor of 1 reads and writes nothing. */
int tgemm_scale(int type, int64_t n, void* X, int64_t n2, void* X2, const float* factor, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TGEMM_OPS_H_ */
