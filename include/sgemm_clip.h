/*
 * sgemm_clip.h — the global norm of many tensors, and clipping to a largest norm, C ABI.
 *
 *     norm   = sqrt(sum over all tensors and elements of x^2)
 *     factor = min(1, max_norm / (norm + 1e-6))
 *     out    = factor * x
 *
 * The step between a backward pass (sgemm_xent_grad, sgemm_distill_grad,
 * sgemm_linear_grad) and an update: all gradients together are scaled down to a
 * norm of max_norm, and left as they are where it is not above that.
 *
 * Conventions:
 *   - The array of tensors is HOST memory, read during the call only; the data and
 *     `norm` are DEVICE memory. Everything runs asynchronously on `stream`, without a
 *     copy to the host; a handle is used by one stream at a time.
 *   - A tensor is `rows` rows of `cols` elements, rows `ld` elements apart (a packed
 *     tensor of any shape: rows = 1, cols = its size). FP32 and bfloat16 tensors can be mixed.
 *   - out == NULL: in place. Otherwise out has the same rows, cols and type, a stride of
 *     its own (ld_out), and is written always, also with a factor of 1.
 *   - Tensors and outputs must not overlap each other, but for an output that is its own
 *     tensor (same address and stride). A tensor or an output named twice, or an output that
 *     starts where another tensor does, is refused; other overlaps are not looked for.
 *   - No tensors, or none with an element: norm = 0.
 *   - max_norm = infinity: the factor is 1 whatever the norm; max_norm = 0: factor 0.
 *   - A norm that is infinite makes the factor 0 (infinite elements become NaN), one that is
 *     NaN makes every element NaN: the caller sees it in `norm`.
 *
 * Numerics: squares are added up in FP32 over at most 32 elements and in FP64 from there;
 * groups whose FP32 sum would leave the range where it is accurate are added in FP64 from the
 * squares on, so the norm is within 2^-20 of itself for every finite tensor (infinite where
 * it leaves FP32's range). factor is FP32, out = factor * x rounded once to its type.
 * Results are bitwise reproducible for the same tensors.
 *
 * Errors: sgemm_status values as for sgemm_run; an invalid argument touches nothing.
 * CUDA graphs: as sgemm_run, once the workspace holds sgemm_clip_workspace(count) bytes.
 */
#ifndef SGEMM_GB300_CLIP_H
#define SGEMM_GB300_CLIP_H

#include "sgemm_vocab.h" /* sgemm_dtype_t */

#ifdef __cplusplus
extern "C" {
#endif

typedef struct sgemm_tensor_s {
    const void *data;
    void *out;           /* NULL: in place */
    long long rows, cols;
    long long ld, ld_out; /* elements from row to row (any value where rows <= 1) */
    int dtype;           /* sgemm_dtype_t */
} sgemm_tensor_t;

/*
 * Requirements: count >= 0; tensors non-NULL when count > 0; rows, cols >= 0; data non-NULL and
 * aligned to its element where rows and cols are not 0, out too where it is given; ld, ld_out >= cols
 * where rows > 1; max_norm >= 0; norm non-NULL, 4-byte aligned. Any violation returns
 * SGEMM_ERR_INVALID_VALUE; SGEMM_ERR_ALLOC if the workspace cannot grow.
 */
int sgemm_clip(struct sgemm_handle_s *h, int count, const sgemm_tensor_t *tensors, float max_norm, float *norm,
               struct CUstream_st *stream);

/* Device workspace that a call with `count` tensors takes at most (sgemm_reserve). Host-only. */
int sgemm_clip_workspace(int count, long long *bytes);

#ifdef __cplusplus
}
#endif

#endif /* SGEMM_GB300_CLIP_H */
