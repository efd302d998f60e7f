// C ABI of the linear layers: argument checks, workspace, launches. Declarations and
// contracts: include/sgemm_linear.h.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include <cuda_runtime.h>

#include "handle.h"
#include "linear_internal.h"
#include "sgemm_internal.h"
#include "vocab_internal.h"

using namespace sgemm_impl;

namespace {

// The arguments of both calls in one place.
struct Call {
    sgemm_handle_t h;
    int M, N, K, dtype;
    const void *X;
    int ldx;
    const void *W;
    int ldw;
    const void *bias = nullptr;
    int act = SGEMM_ACT_NONE;
    const void *R = nullptr;
    int ldr = 0;
    void *Y = nullptr;
    int ldy = 0;
    void *slope = nullptr;  // left by the layer, read by the gradients
    int lds = 0;
    const void *dY = nullptr;
    int lddy = 0;
    float beta = 0.0f;
    void *dX = nullptr, *dW = nullptr, *db = nullptr;
    int lddx = 0, lddw = 0;
    cudaStream_t stream;
    mutable int launched = 0;  // kernels of this call so far: all but the first are dependents of the one before
    bool dependent() const { return launched++ > 0; }
    int size() const { return dtype == SGEMM_DTYPE_BF16 ? 2 : 4; }
};

bool aligned(const void *p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

// Rows on boundaries of `bytes`.
bool rows_on(const void *p, long long ld, int size, unsigned bytes) { return aligned(p, bytes) && ld * size % bytes == 0; }

LinearProblem problem(const Call &c, bool grad)
{
    const int align = (rows_on(c.X, c.ldx, c.size(), 16) ? 1 : 0) | (rows_on(c.W, c.ldw, c.size(), 16) ? 2 : 0) |
                      (rows_on(c.dY, c.lddy, c.size(), 16) ? 4 : 0);
    return LinearProblem{c.M, c.N, c.K, c.dtype, grad, c.dX != nullptr, c.dW != nullptr, c.db != nullptr, c.slope != nullptr,
                         align, c.h->num_sms, c.h->linear_pairs,
                         c.h->linear_ok ? c.h->linear_clusters : nullptr};
}

// What the handle knows of this file's kernels, asked for at the first call that needs it (the calls without them do not
// depend on them): whether they can run, and the pairs that are resident at once.
bool kernels_ready(sgemm_handle_t h)
{
    if (h->linear_pairs == 0) {
        if (linear_set_attributes() == cudaSuccess) {
            const int pairs = linear_max_pairs();
            h->linear_pairs = pairs > 0 ? std::min(pairs, h->num_sms / 2) : -1;
            linear_max_clusters(h->linear_clusters);
            h->linear_ok = true;
        } else {
            (void)cudaGetLastError();
            h->linear_pairs = -1;
        }
    }
    return h->linear_ok;
}

// An output that starts where something that the call reads or another output does, Y on R in the same rows apart.
bool over_each_other(const Call &c, bool grad)
{
    const void *const outs[] = {c.Y, grad ? nullptr : c.slope, c.dX, c.dW, c.db};
    const void *const read[] = {!grad || c.dW != nullptr ? c.X : nullptr, !grad || c.dX != nullptr ? c.W : nullptr, c.bias, c.R, c.dY,
                                grad ? c.slope : nullptr};
    for (const void *o : outs) {
        if (o == nullptr) continue;
        for (const void *p : read)
            if (o == p && !(o == c.Y && p == c.R && (c.M <= 1 || c.ldy == c.ldr))) return true;
        int same = 0;
        for (const void *p : outs) same += p == o;
        if (same > 1) return true;
    }
    return false;
}

int check(const Call &c, bool grad)
{
    if (c.h == nullptr) return SGEMM_ERR_INVALID_VALUE;
    const int rc = validate_linear(problem(c, grad));
    if (rc == SGEMM_ERR_INVALID_VALUE) return rc;
    for (const void *p : {c.X, c.W, c.bias, c.R, static_cast<const void *>(c.Y), static_cast<const void *>(c.slope), c.dY,
                          static_cast<const void *>(c.dX), static_cast<const void *>(c.dW), static_cast<const void *>(c.db)})
        if (!aligned(p, c.size())) return SGEMM_ERR_INVALID_VALUE;
    if (c.act < SGEMM_ACT_NONE || c.act > SGEMM_ACT_SILU || !std::isfinite(c.beta)) return SGEMM_ERR_INVALID_VALUE;
    const bool need_x = !grad || c.dW != nullptr, need_w = !grad || c.dX != nullptr;
    if ((need_x && c.ldx < c.K) || (need_w && c.ldw < c.K) || (c.R != nullptr && c.ldr < c.N) ||
        (c.slope != nullptr && c.lds < c.N))
        return SGEMM_ERR_INVALID_VALUE;
    if (grad ? c.lddy < c.N || (c.dX != nullptr && c.lddx < c.K) || (c.dW != nullptr && c.lddw < c.K) : c.ldy < c.N)
        return SGEMM_ERR_INVALID_VALUE;
    if (c.M > 0 && ((need_x && c.X == nullptr) || (need_w && c.W == nullptr) || (grad ? c.dY == nullptr : c.Y == nullptr)))
        return SGEMM_ERR_INVALID_VALUE;
    if (c.M > 0 && over_each_other(c, grad)) return SGEMM_ERR_INVALID_VALUE;
    return rc;
}

// Map of `parts` (rows x cols) matrices: operands are read in boxes of 64 x 64 bfloat16, results written in boxes of 64
// bytes x 32 rows.
int make_map(sgemm_handle_t h, CUtensorMap *map, const void *base, CUtensorMapDataType type, int size, int cols, int rows,
             long long ld, int parts, bool result, int box_rows = 64)
{
    const cuuint64_t bytes = static_cast<cuuint64_t>(size);
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(parts)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld) * bytes, static_cast<cuuint64_t>(ld) * rows * bytes};
    cuuint32_t box[3] = {static_cast<cuuint32_t>(result ? 64 / size : 64), result ? 32u : static_cast<cuuint32_t>(box_rows), 1};
    cuuint32_t estr[3] = {1, 1, 1};
    const CUresult r = h->encode(map, type, 3, const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                                 result ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                                 CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? SGEMM_OK : SGEMM_ERR_CUDA;
}

// An operand's map: bfloat16, or the two float16 parts of an FP32 one (elements of 16 bits; the products know which).
int operand_map(const Call &c, CUtensorMap *map, const void *base, int cols, int rows, long long ld, int box_rows = 64)
{
    return make_map(c.h, map, base, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, cols, rows, ld, c.size() / 2, false, box_rows);
}

int result_map(const Call &c, CUtensorMap *map, const void *base, bool slope, int cols, int rows, long long ld)
{
    const CUtensorMapDataType type = c.size() == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                     : slope       ? CU_TENSOR_MAP_DATA_TYPE_UINT16
                                                   : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    return make_map(c.h, map, base, type, c.size(), cols, rows, ld, 1, true);
}

// The map of X or W: the caller's matrix, an aligned copy of it, or its parts by rows, which are made first.
int map_operand(const Call &c, const LinearLayout &w, bool copy, const void *src, int rows, int ld, long long off, long long scale_off,
                CUtensorMap *map, int box_rows = 64)
{
    if (!copy) return operand_map(c, map, src, c.K, rows, ld, box_rows);
    char *ws = static_cast<char *>(c.h->workspace);
    const cudaError_t e = w.split ? launch_linear_parts(rows, c.K, src, ld, nullptr, 0, nullptr, ws + off,
                                                        reinterpret_cast<float *>(ws + scale_off), nullptr, nullptr, w.ldk, c.dependent(),
                                                        c.stream)
                                  : launch_vocab_copy(src, ld, rows, c.K, ws + off, w.ldk, c.dependent(), c.stream);
    if (e != cudaSuccess) return SGEMM_ERR_LAUNCH;
    return operand_map(c, map, ws + off, c.K, rows, w.ldk, box_rows);
}

void set_common(const Call &c, const LinearLayout &w, LinearParams *p)
{
    p->dtype = c.dtype;
    p->products = w.split ? 3 : 1;
    // FP32 operands: 256 deep (linear_kernels.cu); else one segment
    p->segment = w.split ? 4 : 1 << 24;
    p->status = c.h->d_status;
    p->timeout_ns = c.h->timeout_ns;
}

// The result of a product, and what is added to it.
int set_product(const Call &c, LinearProduct *t, int kind, int rows, int cols, int K, const LinearShape &s, void *out, long long ldo,
                const void *add, long long ldadd, float gamma, CUtensorMap *map)
{
    t->kind = kind;
    t->rows = rows;
    t->cols = cols;
    t->kblocks = K / kLinearBK + (K % kLinearBK != 0);
    t->tiles_m = rows / (128 * s.ctas) + (rows % (128 * s.ctas) != 0);
    t->tiles_n = cols / s.bn + (cols % s.bn != 0);
    t->out = out;
    t->ldo = ldo;
    t->add = add;
    t->ldadd = ldadd;
    t->gamma = gamma;
    t->out_tma = rows_on(out, ldo, c.size(), 16);
    t->add_tma = add != nullptr && rows_on(add, ldadd, c.size(), 16);
    t->out_vec = rows_on(out, ldo, c.size(), 4 * c.size());
    t->add_vec = add != nullptr && rows_on(add, ldadd, c.size(), 4 * c.size());
    return t->out_tma ? result_map(c, map, out, false, cols, rows, ldo) : SGEMM_OK;
}

int run_layer(const Call &c)
{
    int rc = check(c, false);
    if (rc != SGEMM_OK) return rc;
    if (c.M == 0) return SGEMM_OK;
    DeviceGuard g(c.h->device);
    if (!g.ok) return SGEMM_ERR_CUDA;
    LinearLayout w = linear_layout(problem(c, false));
    if (w.few) {
        const LinearFewParams f{c.M, c.N, c.K, c.X, c.W, c.ldx, c.ldw, c.bias, c.R, c.Y, c.slope, c.ldr, c.ldy, c.lds, c.act};
        return launch_linear_few(f, c.dtype, (problem(c, false).align_flags & 3) == 3, c.h->num_sms, c.stream) == cudaSuccess
                   ? SGEMM_OK
                   : SGEMM_ERR_LAUNCH;
    }
    if (!kernels_ready(c.h)) return SGEMM_ERR_NOT_SUPPORTED;
    w = linear_layout(problem(c, false));  // (the pairs are known now)
    if ((rc = ensure_workspace(c.h, static_cast<size_t>(w.pub.workspace_bytes), c.stream)) != SGEMM_OK) return rc;
    LinearParams p{};
    LinearMaps m;
    if ((rc = map_operand(c, w, w.copy_x, c.X, c.M, c.ldx, w.x_off, w.xs_off, &m.a[0])) != SGEMM_OK) return rc;
    if ((rc = map_operand(c, w, w.copy_w, c.W, c.N, c.ldw, w.w_off, w.ws_off, &m.b[0], w.y.bn / w.y.ctas)) != SGEMM_OK) return rc;
    // where a call has no such matrix, a valid map that no tile uses
    m.a[1] = m.b[1] = m.out[0] = m.out[1] = m.slope = m.a[0];
    set_common(c, w, &p);
    p.products_of_launch = 1;
    p.splits = w.y.splits;
    p.bn = w.y.bn;
    p.bias = c.bias;
    p.act = c.act;
    p.slope = c.slope;
    p.lds = c.lds;
    p.slope_tma = c.slope != nullptr && rows_on(c.slope, c.lds, c.size(), 16);
    p.slope_vec = c.slope != nullptr && rows_on(c.slope, c.lds, c.size(), 4 * c.size());
    if ((rc = set_product(c, &p.t[0], kLinearY, c.M, c.N, c.K, w.y, c.Y, c.ldy, c.R, c.ldr, c.R != nullptr ? 1.0f : 0.0f,
                          &m.out[0])) != SGEMM_OK)
        return rc;
    if (w.split) {
        p.t[0].row_unscale = reinterpret_cast<const float *>(static_cast<char *>(c.h->workspace) + w.xs_off);
        p.t[0].col_unscale = reinterpret_cast<const float *>(static_cast<char *>(c.h->workspace) + w.ws_off);
    }
    if (p.slope_tma && (rc = result_map(c, &m.slope, c.slope, true, c.N, c.M, c.lds)) != SGEMM_OK) return rc;
    if (launch_linear_tiles(m, p, w.y.ctas, w.y.ctas == 2 ? w.workers : c.h->num_sms, c.dependent(), c.stream) != cudaSuccess)
        return SGEMM_ERR_LAUNCH;
    return SGEMM_OK;
}

int run_grad(const Call &c)
{
    int rc = check(c, true);
    if (rc != SGEMM_OK) return rc;
    if (c.dX == nullptr && c.dW == nullptr && c.db == nullptr) return SGEMM_OK;
    DeviceGuard g(c.h->device);
    if (!g.ok) return SGEMM_ERR_CUDA;
    if (c.M == 0) {  // no rows: beta times what is there
        if (c.dW != nullptr && launch_vocab_finish(c.N, c.K, nullptr, 0, 0, 0, c.beta, c.dW, c.lddw, c.dtype, c.dependent(),
                                                   c.stream) != cudaSuccess)
            return SGEMM_ERR_LAUNCH;
        if (c.db != nullptr && launch_linear_columns(c.N, 0, nullptr, c.beta, c.db, c.dtype, nullptr, nullptr, c.dependent(),
                                                     c.stream) != cudaSuccess)
            return SGEMM_ERR_LAUNCH;
        return SGEMM_OK;
    }
    if (!kernels_ready(c.h)) return SGEMM_ERR_NOT_SUPPORTED;
    const LinearLayout w = linear_layout(problem(c, true));
    if ((rc = ensure_workspace(c.h, static_cast<size_t>(w.pub.workspace_bytes), c.stream)) != SGEMM_OK) return rc;
    char *ws = static_cast<char *>(c.h->workspace);
    auto floats = [&](bool there, long long off) { return there ? reinterpret_cast<float *>(ws + off) : nullptr; };
    const bool dx = c.dX != nullptr, dw = c.dW != nullptr, db = c.db != nullptr;
    float *sums = floats(db, w.db_off);
    LinearParams p{};
    LinearMaps m;
    CUtensorMap dz, dzc, x, wt;  // dZ as dX and as dW read it
    const float beta = c.beta;
    if (w.split) {
        // dW's operands are scaled by columns, dX's by rows (dZ's after W's row factors, the sum's index, are in it)
        float *most = floats(dw, w.most_off), *mostx = floats(dw, w.mostx_off);
        float *xs = floats(dw, w.xs_off), *wsc = floats(dx, w.ws_off), *zs = floats(dx, w.dzs_off), *zcs = floats(dw, w.dzcs_off);
        if ((db || dw) &&
            (launch_linear_strips(c.M, c.N, c.dtype, c.dY, c.lddy, c.slope, c.lds, nullptr, 0, sums, most, c.dependent(), c.stream) !=
                 cudaSuccess ||
             launch_linear_columns(c.N, w.strips, sums, c.beta, c.db, c.dtype, most, zcs, c.dependent(), c.stream) != cudaSuccess))
            return SGEMM_ERR_LAUNCH;
        if (dw && (launch_linear_strips(c.M, c.K, c.dtype, c.X, c.ldx, nullptr, 0, nullptr, 0, nullptr, mostx, c.dependent(), c.stream) !=
                       cudaSuccess ||
                   launch_linear_columns(c.K, w.strips, nullptr, 0.0f, nullptr, c.dtype, mostx, xs, c.dependent(), c.stream) !=
                       cudaSuccess ||
                   launch_linear_parts(c.M, c.K, c.X, c.ldx, nullptr, 0, nullptr, nullptr, nullptr, xs, ws + w.x_off, w.ldk,
                                       c.dependent(), c.stream) != cudaSuccess))
            return SGEMM_ERR_LAUNCH;
        if (dx && launch_linear_parts(c.N, c.K, c.W, c.ldw, nullptr, 0, nullptr, ws + w.w_off, wsc, nullptr, nullptr, w.ldk, c.dependent(),
                                      c.stream) != cudaSuccess)
            return SGEMM_ERR_LAUNCH;
        if ((dx || dw) && launch_linear_parts(c.M, c.N, c.dY, c.lddy, c.slope, c.lds, wsc, dx ? ws + w.dz_off : nullptr, zs, zcs,
                                              dw ? ws + w.dzc_off : nullptr, w.ldn, c.dependent(), c.stream) != cudaSuccess)
            return SGEMM_ERR_LAUNCH;
        if (dx && ((rc = operand_map(c, &dz, ws + w.dz_off, c.N, c.M, w.ldn)) != SGEMM_OK ||
                   (rc = operand_map(c, &wt, ws + w.w_off, c.K, c.N, w.ldk)) != SGEMM_OK))
            return rc;
        if (dw && ((rc = operand_map(c, &dzc, ws + w.dzc_off, c.N, c.M, w.ldn)) != SGEMM_OK ||
                   (rc = operand_map(c, &x, ws + w.x_off, c.K, c.M, w.ldk)) != SGEMM_OK))
            return rc;
    } else {
        if ((w.make_dz || db) && launch_linear_strips(c.M, c.N, c.dtype, c.dY, c.lddy, c.slope, c.lds, w.make_dz ? ws + w.dz_off : nullptr,
                                                      w.ldn, sums, nullptr, c.dependent(), c.stream) != cudaSuccess)
            return SGEMM_ERR_LAUNCH;
        if (db && launch_linear_columns(c.N, w.strips, sums, c.beta, c.db, c.dtype, nullptr, nullptr, c.dependent(), c.stream) !=
                      cudaSuccess)
            return SGEMM_ERR_LAUNCH;
        if (dx || dw) {
            rc = w.make_dz ? operand_map(c, &dz, ws + w.dz_off, c.N, c.M, w.ldn) : operand_map(c, &dz, c.dY, c.N, c.M, c.lddy);
            if (rc != SGEMM_OK) return rc;
            dzc = dz;
        }
        if (dw && (rc = map_operand(c, w, w.copy_x, c.X, c.M, c.ldx, w.x_off, 0, &x)) != SGEMM_OK) return rc;
        if (dx && (rc = map_operand(c, w, w.copy_w, c.W, c.N, c.ldw, w.w_off, 0, &wt)) != SGEMM_OK) return rc;
    }
    if (!dx && !dw) return SGEMM_OK;
    set_common(c, w, &p);
    // where a launch has no such matrix, a valid map that no tile uses
    m.a[0] = m.a[1] = m.b[0] = m.b[1] = m.out[0] = m.out[1] = m.slope = dx ? dz : dzc;
    auto add_dx = [&](int i) {
        m.a[i] = dz;
        m.b[i] = wt;
        p.t[i].row_unscale = floats(w.split, w.dzs_off);
        p.t[i].col_unscale = nullptr;
        return set_product(c, &p.t[i], kLinearDx, c.M, c.K, c.N, w.dx, c.dX, c.lddx, beta != 0.0f ? c.dX : nullptr, c.lddx, beta,
                           &m.out[i]);
    };
    auto add_dw = [&](int i) {
        m.a[i] = dzc;
        m.b[i] = x;
        p.t[i].row_unscale = floats(w.split, w.dzcs_off);
        p.t[i].col_unscale = floats(w.split, w.xs_off);
        return set_product(c, &p.t[i], kLinearDw, c.N, c.K, c.M, w.dw, c.dW, c.lddw, beta != 0.0f ? c.dW : nullptr, c.lddw, beta,
                           &m.out[i]);
    };
    auto launch = [&](int products, const LinearShape &s) {
        p.products_of_launch = products;
        p.splits = s.splits;
        p.bn = s.bn;
        return launch_linear_tiles(m, p, s.ctas, s.ctas == 2 ? w.workers : c.h->num_sms, c.dependent(), c.stream) == cudaSuccess
                   ? SGEMM_OK
                   : SGEMM_ERR_LAUNCH;
    };
    if (w.together) {
        // the longer tiles first; workers with one of them fewer take as many of the others as it is long
        const int first = c.N >= c.M ? 0 : 1;  // 0: dX's
        if ((rc = add_dx(first)) != SGEMM_OK || (rc = add_dw(1 - first)) != SGEMM_OK) return rc;
        const int workers = w.dx.ctas == 2 ? w.workers : c.h->num_sms;
        const int a = p.t[0].tiles_m * p.t[0].tiles_n, b = p.t[1].tiles_m * p.t[1].tiles_n, rem = a % workers;
        const int cost = std::max(p.t[1].kblocks * p.products, 6);  // no less than its epilogue takes
        p.extra = rem > 0 ? std::min((p.t[0].kblocks * p.products + cost / 2) / cost, b / (workers - rem)) : 0;
        return launch(2, w.dx);
    }
    if (c.dX != nullptr) {
        if ((rc = add_dx(0)) != SGEMM_OK || (rc = launch(1, w.dx)) != SGEMM_OK) return rc;
    }
    if (c.dW != nullptr) {
        if ((rc = add_dw(0)) != SGEMM_OK || (rc = launch(1, w.dw)) != SGEMM_OK) return rc;
    }
    return SGEMM_OK;
}

}  // namespace

extern "C" {

int sgemm_linear(sgemm_handle_s *h, int M, int N, int K, int dtype, const void *X, int ldx, const void *W, int ldw,
                 const void *bias, int act, const void *R, int ldr, void *Y, int ldy, void *slope, int lds, CUstream_st *stream)
{
    Call c{};
    c.h = h;
    c.M = M;
    c.N = N;
    c.K = K;
    c.dtype = dtype;
    c.X = X;
    c.ldx = ldx;
    c.W = W;
    c.ldw = ldw;
    c.bias = bias;
    c.act = act;
    c.R = R;
    c.ldr = ldr;
    c.Y = Y;
    c.ldy = ldy;
    c.slope = slope;
    c.lds = lds;
    c.stream = stream;
    return run_layer(c);
}

int sgemm_linear_grad(sgemm_handle_s *h, int M, int N, int K, int dtype, const void *X, int ldx, const void *W, int ldw,
                      const void *slope, int lds, const void *dY, int lddy, float beta, void *dX, int lddx, void *dW, int lddw,
                      void *db, CUstream_st *stream)
{
    Call c{};
    c.h = h;
    c.M = M;
    c.N = N;
    c.K = K;
    c.dtype = dtype;
    c.X = X;
    c.ldx = ldx;
    c.W = W;
    c.ldw = ldw;
    c.slope = const_cast<void *>(slope);
    c.lds = lds;
    c.dY = dY;
    c.lddy = lddy;
    c.beta = beta;
    c.dX = dX;
    c.lddx = lddx;
    c.dW = dW;
    c.lddw = lddw;
    c.db = db;
    c.stream = stream;
    return run_grad(c);
}

}  // extern "C"
