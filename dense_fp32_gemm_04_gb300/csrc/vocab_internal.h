// Interface between the host side of the vocabulary losses (vocab_plan.cpp,
// vocab_api.cpp) and their kernels (vocab_rows.cu, vocab_few.cu,
// vocab_kernels.cu). Public contract: include/sgemm_vocab.h. Not installed.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/sgemm.h"
#include "../../include/sgemm_vocab.h"

namespace sgemm_impl {

// The targets of each token as the kernels read them: for the cross entropy the
// caller's labels (one target of weight 1); for the distillation a table of n
// entries per token made by launch_vocab_targets, ascending by id, the entries
// that are left out at the end with the id kNoTarget.
constexpr int kNoTarget = 0x7fffffff;

// Logits in powers of two whose FP32 neighbours are 2 and more apart.
constexpr float kHugeLog2 = 16777216.0f;

struct VocabTargets {
    const long long *labels;  // cross entropy, else NULL
    int n;                    // targets per token (1 for the cross entropy)
    const int *id;            // [T][n]
    const float *q;           // [T][n] teacher probability
    const float *logq;        // [T][n]
};

// Losses of up to this many tokens run without tensor cores (vocab_few.cu); `copied`: bfloat16 rows that the tensor
// cores would need copied first. Measured, us without / with tensor cores: FP32 50021 x 2048, 8 tokens 82 / 281, 24
// tokens 230 / 281, 32 tokens 302 / 281; bfloat16 131072 x 4096, 2 tokens 164 / 172, 3 tokens 290 / 173; rows at an odd
// stride, 50021 x 1531, 8 tokens 87 / 92, 12 tokens 165 / 92.
constexpr int kFewTokensF32 = 24, kFewTokensBf16 = 2, kFewTokensCopied = 8;

// Tile shape: 256 columns per tile, slabs of 64 along K; 128 rows per CTA.
constexpr int kVocabBN = 256, kVocabBK = 64;

struct VocabProblem {
    int T, V, D;
    int dtype;  // sgemm_dtype_t
    int n;      // teacher entries per token, 0 = cross entropy
    bool dh, dw;  // gradients asked for (both false: the loss)
    int align_flags;  // as sgemm_vocab_plan's
    int num_sms;
    int math_mode;
    int pairs;  // CTA pairs resident at once (0: num_sms / 2; < 0: none)
    int piece;  // entries per piece of the vocabulary (0: automatic)
};

// What a call does, and the byte offsets of the parts of its workspace (those a call does not use are empty).
struct VocabLayout {
    sgemm_vocab_plan_t pub;
    bool few;      // loss of a few tokens: vocab_few.cu, no parts
    bool few_targets;  // gradients of as few: their logits at the targets from there too
    int ctas;      // CTAs per worker: 2 = pairs computing 256 x 256 tiles, 1 = 128 x 256
    int workers;
    bool split;           // FP32 operands, used as 16-bit parts
    int parts, products;  // parts of dZ and of the operands of dW, products of parts
    bool copy_h, copy_w;  // workspace rows of H and W: an aligned copy; of a split H, bfloat16 parts for dW
    long long ldp;                         // elements of such a row
    long long h_off, w_off;                // [parts][rows][ldp]
    long long hz_off, wz_off;              // float16 parts, [2][rows][ldp]
    long long hs_off, ws_off;              // what undoes their rows' scaling; W's in whole tiles, after the largest of it
    long long gz_off[2];                   // dZ of a piece in float16 parts for dH, [2][g_blocks][T][64]
    long long tid_off, tq_off, tlogq_off;  // target tables [T][n]
    long long zt_off;                      // logits at the targets, [T][n]
    int targets;                           // of them, for a few tokens
    long long part_off;                    // (max, sum of exp) per token and 128 columns or warp, [stat_cols][T]
    int stat_cols;                         // pairs per token
    long long g_off[2];                    // dZ of a piece, [parts][g_blocks][T][64]; two of them, in turn
    int g_blocks;                          // blocks of 64 entries of a piece, in whole tiles
    int dh_splits, dh_kb;                  // dH tiles: parts of a piece along the vocabulary, k-blocks each
    long long acc_off, ldacc;              // FP32 sums of dH, [dh_splits][T][ldacc]
};

// K-blocks that a tile of `rows` rows (or D columns) along K counts for: no fewer than its epilogue takes.
inline int vocab_cost(int k) { return k > 6 * kVocabBK ? (k + kVocabBK - 1) / kVocabBK : 6; }

int validate_vocab(const VocabProblem &q);
VocabLayout vocab_layout(const VocabProblem &q);

// All launches: dependent = launched as a programmatic dependent of the call's previous kernel, whose end it waits
// for; a call's first kernel is not.
// Row kernels (vocab_rows.cu).
cudaError_t launch_vocab_targets(int T, int V, int n, const long long *ids, const float *logits, long long ldn,
                                 float scale, int *tid, float *tq, float *tlogq, bool dependent,
                                 cudaStream_t stream);
// lse and loss of each token from the columns' (max, sum) pairs and the logits at its targets.
cudaError_t launch_vocab_combine(int T, int V, const VocabTargets &t, const float2 *part, int parts, const float *zt,
                                 float mult, float *loss, float *lse, cudaStream_t stream);
// dst = sum of `splits` FP32 matrices + beta * dst (splits == 0: dst = beta * dst), rows x cols.
cudaError_t launch_vocab_finish(int rows, int cols, const float *acc, long long ldacc, long long split, int splits,
                                float beta, void *dst, long long ldd, int dtype, bool dependent, cudaStream_t stream);

// Losses of a few tokens without tensor cores (vocab_few.cu): the (max, sum) pair and the targets' logits of
// every warp's range of the vocabulary.
struct VocabFewParams {
    int T, V, D;
    const void *H, *W;
    long long ldh, ldw;
    float scale;
    VocabTargets t;
    float2 *part;  // [stat_rows][T]
    float *zt;     // [targets]
    int stat_rows, targets;  // what the workspace has room for (for the debug build's checks)
    int rows;  // of the vocabulary per warp (set by the launch)
    int *status;
};
int vocab_few_warps(int T, int num_sms);
cudaError_t launch_vocab_few(VocabFewParams p, int dtype, bool vec, int num_sms, bool dependent, cudaStream_t stream);

// The products at the targets, before the scaling, into p.zt.
cudaError_t launch_vocab_few_targets(const VocabFewParams &p, int dtype, bool vec, bool dependent, cudaStream_t stream);

// Tile kernel (vocab_kernels.cu): one launch's tiles.
enum VocabKind { kVocabLoss = 0, kVocabDz = 1, kVocabDw = 2, kVocabDh = 3 };

struct VocabTileParams {
    int T, V, D;
    int dtype;
    int parts, products;  // of dW
    bool f16;             // FP32 operands: those of Z and dH are float16 parts, scaled row by row
    int f16_products;     // of Z and dH (1 for bfloat16 operands)
    const float *h_unscale, *w_unscale, *w_most;
    int seg_z, seg_g;  // k-blocks per accumulator segment
    float scale;
    VocabTargets t;
    // Z tiles of columns [z_v0, z_v0 + 256 z_tn): the loss, or dZ of one piece
    int z_kind, z_v0, z_tm, z_tn;
    int z_items;
    float2 *part;
    float *zt;           // logits at the targets: left by the loss; read by dZ where a few tokens' products are there
    int stat_cols;       // pairs per token at part
    const float *lse, *dloss;
    int g_blocks;        // dZ's buffer: blocks of 64 entries per part, [parts][g_blocks][T][64]
    // dH and dW tiles of the piece [g_v0, g_v0 + g_vn), whose dZ an earlier launch left
    int g_v0, g_vn;
    int dw_tn;
    int dw_items;
    void *dW;
    long long lddw;
    bool dw_tma, dw_vec;  // dW is written by TMA stores; else whether 4 elements of a row at a time
    float alpha, beta;    // dH = alpha * G W (summed over the pieces), dW = alpha * G^T H + beta * dW, alpha = c * scale
    int dh_tm, dh_tn, dh_kb, dh_splits;
    int dh_items;
    int dh_extra;  // other tiles for a worker that has one dH tile fewer
    bool acc_add;  // dH: add to the sums (a later piece)
    int *status;
    long long timeout_ns;
};
cudaError_t vocab_set_attributes();
int vocab_max_pairs();
// Maps (elements of a row, rows, parts), all with the 128-byte swizzle: operands in boxes of 64 x 64 x 1 (H as Z
// and as dW read it, W, the piece's dZ as dW and as dH read it), results in boxes of 128 bytes x 32 rows (dZ written, twice, the sums of dH by split, dW where dw_tma).
struct VocabMaps {
    CUtensorMap Hz, H, W, G, Gz, Gw, Gzw, acc, dW;
};
cudaError_t launch_vocab_tiles(const VocabMaps &maps, const VocabTileParams &p, int ctas, int workers, bool dependent,
                               cudaStream_t stream);
// bfloat16 rows copied to a row stride of ldd; FP32 rows split into two float16 parts (with what undoes each row's
// scaling) and, where bf is given, bfloat16 parts, each part rows x ldd.
cudaError_t launch_vocab_copy(const void *src, long long ld, int rows, int cols, void *dst, long long ldd, bool dependent,
                              cudaStream_t stream);
cudaError_t launch_vocab_split(const void *src, long long ld, int rows, int cols, void *f16, float *unscale, int padded,
                               float *most, float *clear, void *bf, int parts, long long ldd, bool dependent,
                               cudaStream_t stream);

}  // namespace sgemm_impl
