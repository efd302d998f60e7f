// Interface between the host side of the vocabulary losses (vocab_plan.cpp,
// vocab_api.cpp) and their kernels (vocab_rows.cu, vocab_kernels.cu). Public
// contract: include/sgemm_vocab.h. Not installed.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/sgemm.h"
#include "../../include/sgemm_vocab.h"

namespace sgemm_impl {

// The targets of each token as the kernels read them: for the cross entropy the
// caller's labels (one target of weight 1); for the distillation a table of n
// entries per token made by launch_vocab_targets, ascending by id, the entries
// that are left out at the end with the id kNoTarget.
constexpr int kNoTarget = 0x7fffffff;

struct VocabTargets {
    const long long *labels;  // cross entropy, else NULL
    int n;                    // targets per token (1 for the cross entropy)
    const int *id;            // [T][n]
    const float *q;           // [T][n] teacher probability
    const float *logq;        // [T][n]
};

struct VocabProblem {
    int T, V, D;
    int dtype;  // sgemm_dtype_t
    int n;      // teacher entries per token, 0 = cross entropy
    bool dh, dw;  // gradients asked for (both false: the loss)
    int align_flags;
    int num_sms;
    int math_mode;
};

// Byte offsets of the parts of the workspace (parts that a call does not use are empty).
struct VocabLayout {
    sgemm_vocab_plan_t pub;
    long long tid_off, tq_off, tlogq_off;  // target tables [T][n]
    long long zt_off;                      // logits at the targets, [T][n]
    long long part_off;                    // (max, sum of exp) per token and tile column, [parts][T]
    int parts;                             // tile columns of V
    long long g_off;                       // dZ of one piece
    long long ldg;
    long long acc_off;                     // FP32 sum of dH over the pieces, [T][D]
};

int validate_vocab(const VocabProblem &q);
VocabLayout vocab_layout(const VocabProblem &q);

// Row kernels (vocab_rows.cu).
cudaError_t launch_vocab_targets(int T, int V, int n, const long long *ids, const float *logits, long long ldn,
                                 float scale, int *tid, float *tq, float *tlogq, cudaStream_t stream);
// lse and loss of each token from the tile columns' (max, sum) pairs and the logits at its targets.
cudaError_t launch_vocab_combine(int T, int V, const VocabTargets &t, const float2 *part, int parts, const float *zt,
                                 float mult, float *loss, float *lse, cudaStream_t stream);
// dst = acc + beta * dst (acc == NULL: dst = beta * dst), rows x cols.
cudaError_t launch_vocab_finish(int rows, int cols, const float *acc, long long ldacc, float beta, void *dst,
                                long long ldd, int dtype, int num_sms, cudaStream_t stream);

// Tile kernels (vocab_kernels.cu).
struct VocabTileParams {
    int T, V, D;
    const void *H, *W;
    long long ldh, ldw;
    float scale;
    VocabTargets t;
    float2 *part;
    float *zt;
    const float *lse, *dloss;
    float gmult;       // c * scale
    int v0, vn;        // this piece of the vocabulary
    float *G;          // [T][ldg]
    long long ldg;
};
cudaError_t launch_vocab_forward(const VocabTileParams &p, int dtype, cudaStream_t stream);
cudaError_t launch_vocab_dz(const VocabTileParams &p, int dtype, cudaStream_t stream);
// acc (+)= dZ * W of the piece; `first`: written, else added to
cudaError_t launch_vocab_dh(const VocabTileParams &p, int dtype, float *acc, bool first, cudaStream_t stream);
// dW rows of the piece = dZ^T * H + beta * dW
cudaError_t launch_vocab_dw(const VocabTileParams &p, int dtype, float beta, void *dW, long long lddw,
                            cudaStream_t stream);

}  // namespace sgemm_impl
