// Interface between the host side of the linear layers (linear_plan.cpp,
// linear_api.cpp) and their kernels (linear_kernels.cu, linear_few.cu,
// linear_rows.cu). Public contract: include/sgemm_linear.h. Not installed.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/sgemm.h"
#include "../../include/sgemm_linear.h"

namespace sgemm_impl {

// Tile shape: 256 columns per tile, slabs of 64 along K; 128 rows per CTA.
constexpr int kLinearBN = 256, kLinearBK = 64;
constexpr int kLinearMaxSplits = 8;  // CTAs of a portable cluster

struct LinearProblem {
    int M, N, K;
    int dtype;
    bool grad;
    bool dx, dw, db, slope;  // gradients asked for, and whether dZ differs from dY
    int align_flags;         // as sgemm_linear_plan's
    int num_sms;
    int pairs;               // CTA pairs resident at once (0: num_sms / 2; < 0: none)
    const int *clusters;     // clusters of 1, 2, .. kLinearMaxSplits CTAs resident at once (NULL: as measured on a GB300)
};

// One product of a call: rows x cols over kblocks slabs.
struct LinearShape {
    int splits;  // CTAs of a cluster that share a tile's K range; 0: persistent, whole tiles
    int ctas;    // per whole tile
    int bn;      // columns of a tile: 256; split ones 256 or 128; Y's whole ones a multiple of 32
};

// What a call does, and the byte offsets of the parts of its workspace.
struct LinearLayout {
    sgemm_linear_plan_t pub;
    bool few;
    LinearShape y, dx, dw;
    bool together;  // dX and dW in one launch
    int workers;    // of the persistent launches with pairs
    bool split;     // FP32 operands, used as float16 parts
    bool copy_x, copy_w, make_dz;  // operands that are copied or made into the workspace
    long long ldk, ldn;            // elements of a copied row of X and W, and of dZ
    // bfloat16: [rows][ldk or ldn]. FP32: two float16 parts of each; X (for Y by rows, for dW by columns), W by rows, dZ by rows
    // for dX and by columns for dW
    long long x_off, w_off, dz_off, dzc_off;
    long long xs_off, ws_off, dzs_off, dzcs_off;  // the roots of what undoes their scaling: of X's rows or columns, W's rows, dZ's rows and columns
    long long db_off, most_off, mostx_off;        // of strips of kLinearStrip rows: dZ's columns' sums, and the largest values of
                                                  // dZ's and X's columns, [strips][N or K]
    int strips;
};

int validate_linear(const LinearProblem &q);
LinearLayout linear_layout(const LinearProblem &q);

constexpr int kLinearStrip = 64;  // rows of dZ that a block of the dZ kernel adds up

// All launches: dependent = launched as a programmatic dependent of the call's previous kernel, whose end it waits for;
// a call's first kernel is not.

// Layers of a few tokens (linear_few.cu). vec: rows of X and W start on 16-byte boundaries.
struct LinearFewParams {
    int M, N, K;
    const void *X, *W;
    long long ldx, ldw;
    const void *bias, *R;
    void *Y, *slope;
    long long ldr, ldy, lds;
    int act;
};
// Whether a layer is computed there (measurements: linear_few.cu).
inline bool linear_is_few(int M, long long N, long long K, bool f32) { return M <= (f32 ? 16 : 4) || (f32 && M <= 32 && N * K <= 1 << 22); }
cudaError_t launch_linear_few(const LinearFewParams &p, int dtype, bool vec, int num_sms, cudaStream_t stream);

// x = src (* slope), M x N: in bfloat16 (dz; bfloat16 operands only), its columns' sums over strips of rows (sums) and their
// largest finite |x| (most); what is NULL is not made.
cudaError_t launch_linear_strips(int M, int N, int dtype, const void *src, long long ld, const void *slope, long long lds, void *dz,
                                 long long ldz, float *sums, float *most, bool dependent, cudaStream_t stream);
// db = the strips' sums + beta * db; the root of what undoes the scaling of columns by their strips' largest values (NULL: not made).
cudaError_t launch_linear_columns(int N, int strips, const float *sums, float beta, void *db, int dtype, const float *most,
                                  float *unscale, bool dependent, cudaStream_t stream);
// FP32 x = src (* slope) as two float16 parts: by_row of x times factor[column]^2, each row scaled by a power of two
// (row_unscale^2 undoes it); by_column of x scaled by its columns' (column_unscale^2 undoes it); what is NULL is not made.
cudaError_t launch_linear_parts(int rows, int cols, const void *src, long long ld, const void *slope, long long lds,
                                const float *factor, void *by_row, float *row_unscale, const float *column_unscale, void *by_column,
                                long long ldp, bool dependent, cudaStream_t stream);

// Tile kernel (linear_kernels.cu): one or two products per launch.
enum LinearKind { kLinearY = 0, kLinearDx = 1, kLinearDw = 2 };

struct LinearProduct {
    int kind;
    int rows, cols, kblocks;   // of the result, and slabs along K
    int tiles_m, tiles_n;
    void *out;                 // rows x cols
    const void *add;           // + gamma * add (NULL: nothing)
    long long ldo, ldadd;
    float gamma;
    bool out_tma, add_tma;     // 16-byte aligned rows; else element by element
    bool out_vec, add_vec;     // 4 elements at a time where a split tile is put together
    const float *row_unscale, *col_unscale;  // of FP32 operands' parts: roots of the factors of the result's rows and columns (NULL: 1)
};

struct LinearParams {
    LinearProduct t[2];
    int products_of_launch;    // entries of t
    int extra;                 // tiles of t[1] for a worker that has one tile of t[0] fewer
    int dtype;
    int products;              // of parts of the operands: 1 for bfloat16, 3 of two float16 parts each
    int segment;               // slabs per accumulator segment
    const void *bias;          // t[0] of kind kLinearY
    int act;
    void *slope;
    long long lds;
    bool slope_tma, slope_vec;
    int splits, bn;  // as in LinearShape
    int *status;
    long long timeout_ns;
};

// Operands in boxes of 64 x 64 of 16-bit elements, b of kind Y of 64 x the columns a CTA has of a tile; results in boxes of
// 64 bytes x 32 rows (valid maps that are not used where the products' flags say so).
struct LinearMaps {
    CUtensorMap a[2], b[2], out[2], slope;
};

cudaError_t linear_set_attributes();
int linear_max_pairs();
void linear_max_clusters(int *clusters);  // as LinearProblem's
// ctas and splits as in LinearShape; workers: CTAs or pairs of a persistent launch.
cudaError_t launch_linear_tiles(const LinearMaps &maps, const LinearParams &p, int ctas, int workers, bool dependent,
                                cudaStream_t stream);

}  // namespace sgemm_impl
