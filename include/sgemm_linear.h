/*
 * sgemm_linear.h — a product with bias, activation and residual, and its gradients, C ABI.
 *
 *     Y = act(X * W^T + b) + R
 *
 *   X is M x K (a row per token), W is N x K (a row per output feature), b has N
 *   entries, R and Y are M x N; all row-major with row strides, FP32 or bfloat16
 *   (one type for all). b and R may be left out. The product's result never goes
 *   to memory before bias, activation and residual are in it.
 *
 *   act      none, relu, gelu (z times the normal distribution at z), gelu_tanh
 *            (z / (1 + exp(-2 sqrt(2 / pi) (z + 0.044715 z^3)))), silu (z / (1 + exp(-z)))
 *   slope    act'(X W^T + b), M x N, which the forward call leaves where it is asked
 *            for and the gradients read: FP32 for FP32 operands; for bfloat16 operands
 *            16-bit integers in units of 2^-14 (-32768: NaN). Slopes lie in
 *            [-0.13, 1.13]: a unit is finer than bfloat16 from 2^-7 on, coarser
 *            below, and slopes below 2^-15, in the activations' tails, are 0. The
 *            gradients need neither the pre-activation nor the activation again.
 *
 *   gradients (sgemm_linear_grad), from dY and with dZ = dY * slope (dZ = dY without one):
 *       dX = dZ W + beta dX,  dW = dZ^T X + beta dW,  db = sum over rows of dZ + beta db;
 *   the residual's gradient is dY itself.
 *
 * Conventions:
 *   - All pointers are DEVICE pointers, everything runs asynchronously on `stream`, in
 *     the handle's workspace; a handle is used by one stream at a time, as with sgemm_run.
 *   - Y may be R itself (same address and row stride): the residual is added in place.
 *     Else outputs overlap neither what the call reads nor each other; those that start at
 *     the same address are refused, other overlaps are not looked for.
 *   - beta == 0: dX, dW and db are written without being read. Any of them may be NULL:
 *     that gradient is not computed.
 *   - M == 0: the layer does nothing; the gradients give dW = beta dW and db = beta db.
 *   - Rows need no alignment beyond their element's; operands whose rows start on 16-byte
 *     boundaries spare a copy into the workspace.
 *
 * Numerics: bfloat16 operands enter the products as they are, accumulated in FP32. The
 * tensor cores truncate every 16 products, so a sum of n products of one sign comes out
 * too small by up to n 2^-27 of itself (n is K for Y, N for dX, the number of tokens for
 * dW; measured with alike terms: 8e-6 at n = 4096, 6e-5 at 16384, 3.4e-4 at 65536; terms
 * of random signs stay below 1e-6). Bias, activation and residual are applied in FP32, the
 * activation within 2^-11 of itself, and Y, dX, dW and db rounded once; dZ enters the
 * products rounded to bfloat16.
 * FP32 operands enter the tensor cores as sums of two float16 parts (22 bits) of rows or
 * columns scaled by powers of two (those that are not the sum's index), 256 products deep
 * at most, the rest added in FP32: a result is off by less than 5e-7 of its 2-norm where
 * its terms are of random signs, 1.5e-6 where they are of one, whatever the math mode. An
 * element is held to 2^-39 of the largest in its row (X and W for Y; W, and dZ times the
 * sizes of W's rows, for dX) or column (dZ and X for dW), which shows where the other
 * operand is 0, or as small, in the largest one's place. Infinities and NaN give what the formula has (an element that is held as 0
 * counts as one beside an infinity). A few tokens are computed without tensor cores, in
 * FP32 fused multiply-adds.
 * Results are bitwise reproducible for a fixed shape, alignment and plan.
 *
 * Errors: sgemm_status values as for sgemm_run; an invalid argument touches nothing.
 * Sizes whose tiles do not count in 32 bits, or kernels that this build or machine
 * cannot run: SGEMM_ERR_NOT_SUPPORTED.
 * Device status (sgemm_check_device_status): the TF32 kernel's locations, and 40 where a cluster of
 * split tiles is launched in another shape than planned; in debug builds also 41 stores outside a result.
 *
 * CUDA graphs: as sgemm_run, once the workspace holds the plan's workspace_bytes.
 */
#ifndef SGEMM_GB300_LINEAR_H
#define SGEMM_GB300_LINEAR_H

#include "sgemm_vocab.h" /* sgemm_dtype_t */

#ifdef __cplusplus
extern "C" {
#endif

typedef enum sgemm_act {
    SGEMM_ACT_NONE = 0,
    SGEMM_ACT_RELU = 1,
    SGEMM_ACT_GELU = 2,
    SGEMM_ACT_GELU_TANH = 3,
    SGEMM_ACT_SILU = 4
} sgemm_act_t;

/*
 * Y, and slope unless that is NULL. Requirements: M >= 0; N, K >= 1; ldx, ldw >= K; ldr, ldy, lds >= N
 * (of what is given); X, W, Y non-NULL when M > 0; pointers aligned to their element. Any violation
 * returns SGEMM_ERR_INVALID_VALUE; SGEMM_ERR_ALLOC if the workspace cannot grow.
 */
int sgemm_linear(struct sgemm_handle_s *h, int M, int N, int K, int dtype,
                 const void *X, int ldx, const void *W, int ldw,
                 const void *bias, int act, const void *R, int ldr,
                 void *Y, int ldy, void *slope, int lds, struct CUstream_st *stream);

/*
 * dX (M x K), dW (N x K) and db (N) from dY and the slope that sgemm_linear left (NULL: act was none).
 * X is not read where dW is NULL, W not where dX is.
 */
int sgemm_linear_grad(struct sgemm_handle_s *h, int M, int N, int K, int dtype,
                      const void *X, int ldx, const void *W, int ldw,
                      const void *slope, int lds, const void *dY, int lddy,
                      float beta, void *dX, int lddx, void *dW, int lddw, void *db,
                      struct CUstream_st *stream);

/* What one call does (filled by sgemm_linear_plan). */
typedef struct sgemm_linear_plan_s {
    int few;                   /* 1: computed without tensor cores */
    int ctas;                  /* CTAs per tile: 2 = pairs computing 256 x 256, 1 = 128 x 256 (of the largest product) */
    int splits[2];             /* CTAs of a cluster that share a tile's K range: Y, or dX and dW (1: whole) */
    int launches;              /* kernels the call launches, with everything asked for */
    long long workspace_bytes; /* device workspace the handle holds for it (sgemm_reserve) */
} sgemm_linear_plan_t;

/*
 * Host-only planning: what the calls above do on a GPU with `num_sms` SMs. grad: 0 for the layer, 1 for its
 * gradients (all of them, with a slope; workspace_bytes is enough for any of them too, and for any number of CTA pairs
 * that the GPU holds at once). align_flags: bit 0 = rows of X are 16-byte aligned (base and row stride), bit 1 = rows of W, bit
 * 2 = rows of dY. math_mode: a handle's, as for the other plans; layers are computed alike in all. Needs no GPU.
 */
int sgemm_linear_plan(int M, int N, int K, int dtype, int grad, int align_flags, int num_sms, int math_mode,
                      sgemm_linear_plan_t *out);

#ifdef __cplusplus
}
#endif

#endif /* SGEMM_GB300_LINEAR_H */
