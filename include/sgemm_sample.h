/*
 * sgemm_sample.h — one token per row of logits, with temperature, top-k, top-p and min-p, C ABI.
 *
 * The logits are T x V, row-major with row stride ldl >= V, FP32 or bfloat16 (what
 * sgemm_linear leaves of hidden states and the vocabulary projection). For a row l with
 * largest entry m, its weights are w_i = exp((l_i - m) / temperature). Order the entries
 * by (l descending, index ascending). Each filter keeps a beginning of that order:
 *
 *   top-k    the first k entries;
 *   top-p    of those, the entries before which less than top_p of their mass lies
 *            (the first one always);
 *   min-p    of those, the entries with w_i >= min_p (the largest entry has w = 1).
 *
 * With S the mass of what is kept, the token is the first kept entry, in order of the
 * index, at which the cumulative mass is above u * S; u is the row's given random number
 * in [0, 1). logp = log(w_token / S), the log of the probability it was drawn with.
 *
 * Conventions:
 *   - All pointers in the calls are DEVICE pointers but `how`, which is HOST memory read
 *     during the call. Everything runs asynchronously on `stream`, without workspace.
 *   - A temperature of 0 takes the largest entry (the first of equal ones): logp = 0.
 *   - top_k = 0, top_p = 1, min_p = 0: that filter is off.
 *   - An entry of -infinity or NaN has no weight and is never the token. A row without
 *     any other entry: token -1, logp -infinity. Where entries are +infinity, they alone
 *     have weight, 1 each. A mask of the type's lowest value is an entry like others: far
 *     below the rest it has no weight, alone it is uniform.
 *   - The arrays of `how` hold one value per row, and a value that the call could not
 *     refuse is read so: a temperature that is not above 0 is 0 and an infinite one FP32's largest
 *     number, a top_k below 1 is off, a top_p below 0 is 0 and one that is not below 1 is off, a min_p
 *     that is not above 0 is off and one above 1 is 1. u is read as 0 where it is not above 0, and
 *     u >= 1 takes the last kept entry of weight.
 *
 * Numerics: weights are held to a unit of 2^-44 of the largest one (2^-(44 - d) for vocabularies of 2^18 to 2^(18 + d)
 * entries, so that the sum of V of them fits 64 bits) and summed exactly, as integers. Tokens and cuts are
 * so those of the formulas, but for borders that lie nearer to u S or to top_p's share than the roundings add up to: V
 * units at the very worst, some sqrt(V) as a rule. The result does not depend on the order of sums or on the launch.
 * logp is off by at most 2.5 * 2^-22 + 2^-22 |logp| and what its token's unit and those of S are of them.
 *
 * Errors: sgemm_status values as for sgemm_run; an invalid argument touches nothing.
 * CUDA graphs: a call may be captured at any time.
 */
#ifndef SGEMM_GB300_SAMPLE_H
#define SGEMM_GB300_SAMPLE_H

#include "sgemm_vocab.h" /* sgemm_dtype_t */

#ifdef __cplusplus
extern "C" {
#endif

#define SGEMM_SAMPLE_MAX_VOCAB (1 << 24)

/* The filters: one value for all rows, or where the pointer is not NULL, T values on the device. */
typedef struct sgemm_sampling_s {
    float temperature;  /* >= 0, finite */
    int top_k;          /* >= 0 */
    float top_p;        /* 0 .. 1 */
    float min_p;        /* 0 .. 1 */
    const float *temperatures;
    const int *top_ks;
    const float *top_ps;
    const float *min_ps;
} sgemm_sampling_t;

/*
 * ids (64-bit, T) and logp (FP32, T; may be NULL) from logits and u (FP32, T).
 * Requirements: T >= 0; V >= 1; ldl >= V; logits, u and ids non-NULL when T > 0; pointers aligned to
 * their element; `how` non-NULL with the single values in range (also those that an array replaces).
 * Any violation returns SGEMM_ERR_INVALID_VALUE. V above SGEMM_SAMPLE_MAX_VOCAB or T above 2^27:
 * SGEMM_ERR_NOT_SUPPORTED.
 */
int sgemm_sample(struct sgemm_handle_s *h, int T, int V, int dtype, const void *logits, int ldl, const float *u,
                 const sgemm_sampling_t *how, long long *ids, float *logp, struct CUstream_st *stream);

#ifdef __cplusplus
}
#endif

#endif /* SGEMM_GB300_SAMPLE_H */
