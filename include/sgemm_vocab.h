/*
 * sgemm_vocab.h — losses over a vocabulary projection, with their gradients, C ABI.
 *
 * The projection is the product at the end of a language model,
 *
 *     Z = scale * H * W^T
 *
 *   H is T x D (one row of hidden states per token), W is V x D (one row per
 *   vocabulary entry), both row-major with row strides ldh, ldw >= D, FP32 or
 *   bfloat16. Z (T x V) is never stored: the losses are computed from its tiles
 *   as they are produced, and the gradients from tiles recomputed in pieces of
 *   the vocabulary.
 *
 * With lse_t = log sum_v exp Z_tv and p_tv = exp(Z_tv - lse_t):
 *
 *   cross entropy       loss_t = lse_t - Z_t,y(t)
 *   (sgemm_xent)        for a label y(t) in [0, V); any other label masks the
 *                       token: loss_t = 0, and its gradient is 0.
 *
 *   distillation        with scale = 1 / temperature, n teacher logits per token
 *   (sgemm_distill)     and q_t = softmax(teacher logits of t / temperature):
 *                       loss_t = temperature^2 * sum_j q_tj (log q_tj - log p_t,id(t,j)),
 *                       the divergence of the student from the teacher's n best
 *                       entries. An entry whose id is outside [0, V) is left out
 *                       of the softmax and its logit is not looked at; a token
 *                       with no entry left (or none with a logit above -infinity)
 *                       is masked. An id that a token names twice counts as two
 *                       entries.
 *
 *   gradients           with dloss_t the gradient of the result with respect to
 *   (sgemm_*_grad)      loss_t, c = 1 or temperature^2, u_t = 1 or 0 for a masked
 *                       token, and q_tv the sum of q_tj over id(t,j) = v (for the
 *                       cross entropy 1 at the label, else 0):
 *                       dZ_tv = c * scale * dloss_t * (u_t p_tv - q_tv),
 *                       dH = dZ * W + beta * dH,  dW = dZ^T * H + beta * dW.
 *
 * Conventions:
 *   - All pointers are DEVICE pointers, everything runs asynchronously on
 *     `stream`, in the handle's workspace; a handle is used by one stream at a
 *     time, as with sgemm_run.
 *   - lse is written for masked tokens too. dloss of a masked token is not used;
 *     its row of H takes part in dW with the factor 0, so it has to be finite.
 *   - beta == 0: dH and dW are written without being read.
 *   - dH or dW may be NULL: that gradient is not computed. They must not overlap
 *     H or W.
 *   - T == 0: the losses do nothing; the gradients give dW = beta * dW.
 *   - Rows of H, W, dH and dW need no alignment beyond their element's; rows of H
 *     and W on 16-byte boundaries (on 128-byte ones from 2048 tokens on) spare a
 *     copy of bfloat16 operands into the workspace.
 *
 * Numerics: loss and lse are FP32 whatever the operands' type; products are
 * accumulated in FP32, softmax statistics are kept in FP32. The tensor cores
 * truncate as they accumulate, 1024 products deep at most for a logit: it lies up
 * to 2^-18 of itself nearer to 0, the same in a loss and in its gradients, where
 * that cancels in exp(Z - lse); dH and dW of FP32 operands are accumulated 256
 * deep (sums over terms of one sign, which lose most: dH 2.3e-6, dW 1e-7 of
 * themselves, the others 4e-7 to 8e-7). (Losses of a few tokens do without tensor cores;
 * their gradients take the logits at the targets in the same way.) FP32 Z overflows
 * where D max |W| is 5e33 and more, however small H. bfloat16 operands
 * enter the products as they are and dZ enters them rounded to bfloat16; dH and
 * dW are rounded once. FP32 operands enter the tensor cores as sums of 16-bit
 * parts: for the logits and dH two float16 parts (22 bits) of rows scaled by
 * powers of two, for dW three bfloat16 parts (24 bits; two parts with
 * SGEMM_MATH_TF32). For dH, entry v of dZ is held to within 2^-39 dloss (max |W|
 * of all rows) / (max |W| of row v): a row of W a million times larger than the
 * others leaves 3e-4 of dH where the others make it up. The gradients' p comes
 * from lse as it is stored, an FP32 number: its relative error grows as
 * 2^-22 |lse|, and p is held to at most 1. Probabilities and entries of dZ below
 * FP32's normal range (2^-126) may count as 0. Results are bitwise reproducible
 * for a fixed shape, alignment and plan.
 *
 * Errors: sgemm_status values as for sgemm_run; an invalid argument touches nothing.
 * T, V or D so large that their tiles do not count in 32 bits, or kernels that this
 * build or machine cannot run: SGEMM_ERR_NOT_SUPPORTED.
 * Device status (sgemm_check_device_status): the TF32 kernel's locations; in debug
 * builds also 35 the columns of dZ, 36 the softmax statistics, 37 the targets'
 * logits, 38 the rows of dW, 39 the splits of dH.
 *
 * CUDA graphs: as sgemm_run, once the workspace holds the plan's workspace_bytes.
 */
#ifndef SGEMM_GB300_VOCAB_H
#define SGEMM_GB300_VOCAB_H

#ifdef __cplusplus
extern "C" {
#endif

struct CUstream_st;
struct sgemm_handle_s;

/* Element types of H, W, dH and dW (one type for all four). */
typedef enum sgemm_dtype {
    SGEMM_DTYPE_F32 = 0,
    SGEMM_DTYPE_BF16 = 1
} sgemm_dtype_t;

#define SGEMM_DISTILL_MAX_ENTRIES 1024 /* teacher logits per token */

/*
 * loss[t] and lse[t] (FP32, T each) of the cross entropy; labels: T 64-bit ids.
 * Requirements: T >= 0; V, D >= 1; ldh, ldw >= D; scale > 0 and finite; pointers non-NULL
 * when T > 0 and aligned to their element (8 bytes for labels). Any violation
 * returns SGEMM_ERR_INVALID_VALUE; SGEMM_ERR_ALLOC if the workspace cannot grow.
 */
int sgemm_xent(struct sgemm_handle_s *h, int T, int V, int D, int dtype,
               const void *H, int ldh, const void *W, int ldw,
               const long long *labels, float scale,
               float *loss, float *lse, struct CUstream_st *stream);

/*
 * dH (T x D, row stride lddh) and dW (V x D, row stride lddw) of the cross
 * entropy, from the lse that sgemm_xent gave for the same operands and scale.
 */
int sgemm_xent_grad(struct sgemm_handle_s *h, int T, int V, int D, int dtype,
                    const void *H, int ldh, const void *W, int ldw,
                    const long long *labels, float scale,
                    const float *lse, const float *dloss,
                    float beta, void *dH, int lddh, void *dW, int lddw,
                    struct CUstream_st *stream);

/*
 * loss[t] and lse[t] of the distillation; ids (64-bit) and logits (FP32): T rows
 * of n entries, row stride ldn >= n, in any order; 1 <= n <=
 * SGEMM_DISTILL_MAX_ENTRIES (more: SGEMM_ERR_NOT_SUPPORTED); temperature > 0 and
 * finite. lse is that of Z = H W^T / temperature.
 */
int sgemm_distill(struct sgemm_handle_s *h, int T, int V, int D, int dtype,
                  const void *H, int ldh, const void *W, int ldw,
                  int n, const long long *ids, const float *logits, int ldn, float temperature,
                  float *loss, float *lse, struct CUstream_st *stream);

/* dH and dW of the distillation, from sgemm_distill's lse. */
int sgemm_distill_grad(struct sgemm_handle_s *h, int T, int V, int D, int dtype,
                       const void *H, int ldh, const void *W, int ldw,
                       int n, const long long *ids, const float *logits, int ldn, float temperature,
                       const float *lse, const float *dloss,
                       float beta, void *dH, int lddh, void *dW, int lddw,
                       struct CUstream_st *stream);

/* What one call does (filled by sgemm_vocab_plan). */
typedef struct sgemm_vocab_plan_s {
    int pieces;                /* pieces of the vocabulary a gradient call works through */
    int piece;                 /* vocabulary entries per piece (the last one may be shorter) */
    int launches;              /* kernels the call launches */
    long long workspace_bytes; /* device workspace the handle holds for it (sgemm_reserve) */
} sgemm_vocab_plan_t;

/*
 * Host-only planning: what the calls above do on a GPU with `num_sms` SMs. n: 0
 * for the cross entropy, else the teacher's entries. grad: 0 for the loss, 1 for
 * the gradients (both of them; workspace_bytes is enough for either alone too,
 * and for any number of CTA pairs that the GPU holds at once).
 * align_flags: bit 0 = rows of H are 16-byte aligned (base and row stride), bit 1 =
 * rows of W, bits 2 and 3 = the same with 128 bytes. Needs no GPU. The plan is
 * that of automatic pieces: with SGEMM_OPT_FORCE_VOCAB_PIECE set on a handle, a call
 * may need more workspace (one call outside a capture makes it large enough).
 */
int sgemm_vocab_plan(int T, int V, int D, int dtype, int n, int grad, int align_flags,
                     int num_sms, int math_mode, sgemm_vocab_plan_t *out);

#ifdef __cplusplus
}
#endif

#endif /* SGEMM_GB300_VOCAB_H */
