// C ABI of the vocabulary losses: argument checks, workspace, launches.
// Declarations and contracts: include/sgemm_vocab.h.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include <cuda_runtime.h>

#include "handle.h"
#include "sgemm_internal.h"
#include "vocab_internal.h"

using namespace sgemm_impl;

namespace {

// The arguments of the four calls in one place.
struct Call {
    sgemm_handle_t h;
    int T, V, D, dtype;
    const void *H;
    int ldh;
    const void *W;
    int ldw;
    const long long *labels = nullptr;  // cross entropy
    int n = 0;                          // distillation
    const long long *ids = nullptr;
    const float *logits = nullptr;
    int ldn = 0;
    float scale = 1.0f, mult = 1.0f;  // mult: 1 or temperature^2
    float *loss = nullptr, *lse_out = nullptr;
    const float *lse = nullptr, *dloss = nullptr;
    float beta = 0.0f;
    void *dH = nullptr, *dW = nullptr;
    int lddh = 0, lddw = 0;
    cudaStream_t stream;
    mutable int launched = 0;  // kernels of this call so far: all but the first are dependents of the one before
    bool dependent() const { return launched++ > 0; }
};

bool aligned(const void *p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

VocabProblem problem(const Call &c)
{
    const int size = c.dtype == SGEMM_DTYPE_BF16 ? 2 : 4;
    auto rows = [size](const void *p, long long ld, unsigned bytes) { return aligned(p, bytes) && ld * size % bytes == 0; };
    const int align = (rows(c.H, c.ldh, 16) ? 1 : 0) | (rows(c.W, c.ldw, 16) ? 2 : 0) | (rows(c.H, c.ldh, 128) ? 4 : 0) |
                      (rows(c.W, c.ldw, 128) ? 8 : 0);
    return VocabProblem{c.T, c.V, c.D, c.dtype, c.n, c.dH != nullptr, c.dW != nullptr, align, c.h->num_sms,
                        c.h->math_mode, c.h->vocab_pairs, c.h->vocab_piece};
}

int check(const Call &c, bool grad)
{
    if (c.h == nullptr) return SGEMM_ERR_INVALID_VALUE;
    const int rc = validate_vocab(problem(c));
    if (rc != SGEMM_OK) return rc;
    const unsigned size = c.dtype == SGEMM_DTYPE_BF16 ? 2 : 4;
    if (c.ldh < c.D || c.ldw < c.D || (c.n > 0 && c.ldn < c.n)) return SGEMM_ERR_INVALID_VALUE;
    if (!(c.scale > 0.0f) || !std::isfinite(c.scale) || !std::isfinite(c.mult) || c.mult == 0.0f || !std::isfinite(c.beta))
        return SGEMM_ERR_INVALID_VALUE;  // mult: a temperature whose square leaves FP32's range
    for (const void *p : {c.H, c.W, static_cast<const void *>(c.dH), static_cast<const void *>(c.dW)})
        if (!aligned(p, size)) return SGEMM_ERR_INVALID_VALUE;
    for (const void *p : {static_cast<const void *>(c.logits), static_cast<const void *>(c.loss),
                          static_cast<const void *>(c.lse_out), static_cast<const void *>(c.lse),
                          static_cast<const void *>(c.dloss)})
        if (!elem_aligned(p)) return SGEMM_ERR_INVALID_VALUE;
    if (!aligned(c.labels, 8) || !aligned(c.ids, 8)) return SGEMM_ERR_INVALID_VALUE;
    if (c.T > 0) {
        if (c.H == nullptr || c.W == nullptr) return SGEMM_ERR_INVALID_VALUE;
        if (c.n > 0 ? c.ids == nullptr || c.logits == nullptr : c.labels == nullptr) return SGEMM_ERR_INVALID_VALUE;
        if (grad ? c.lse == nullptr || c.dloss == nullptr : c.loss == nullptr || c.lse_out == nullptr)
            return SGEMM_ERR_INVALID_VALUE;
    }
    if ((c.dH != nullptr && c.lddh < c.D) || (c.dW != nullptr && c.lddw < c.D)) return SGEMM_ERR_INVALID_VALUE;
    if (!c.h->vocab_ok) return SGEMM_ERR_NOT_SUPPORTED;
    return SGEMM_OK;
}

// Map of a (rows x cols) matrix of `parts` parts: operands are read in boxes of 64 x 64, results written in boxes of
// 128 bytes x 32 rows.
int make_map(sgemm_handle_t h, CUtensorMap *map, const void *base, int dtype, int cols, int rows, long long ld, int parts,
             long long part, bool result)
{
    const cuuint64_t size = dtype == SGEMM_DTYPE_BF16 ? 2 : 4;
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(parts)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld) * size, static_cast<cuuint64_t>(part) * size};
    cuuint32_t box[3] = {static_cast<cuuint32_t>(128 / size), result ? 32u : 64u, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    const CUresult r = h->encode(map, size == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3,
                                 const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                                 CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                                 CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? SGEMM_OK : SGEMM_ERR_CUDA;
}

// The map of a bfloat16 operand: the caller's matrix, or an aligned copy of it, which is made first.
int map_operand(const Call &c, const VocabLayout &w, bool copy, const void *src, int rows, int ld, long long off,
                CUtensorMap *map)
{
    if (!copy) return make_map(c.h, map, src, SGEMM_DTYPE_BF16, c.D, rows, ld, 1, static_cast<long long>(ld) * rows, false);
    void *dst = static_cast<char *>(c.h->workspace) + off;
    if (launch_vocab_copy(src, ld, rows, c.D, dst, w.ldp, c.dependent(), c.stream) != cudaSuccess) return SGEMM_ERR_LAUNCH;
    return make_map(c.h, map, dst, SGEMM_DTYPE_BF16, c.D, rows, w.ldp, 1, rows * w.ldp, false);
}

// FP32 operands as parts: H (float16, and bfloat16 where dW reads it), then W (float16).
int split_operands(const Call &c, const VocabLayout &w, VocabTileParams *p, VocabMaps *m)
{
    char *ws = static_cast<char *>(c.h->workspace);
    float *hs = reinterpret_cast<float *>(ws + w.hs_off), *most = reinterpret_cast<float *>(ws + w.ws_off), *vs = most + 64;
    const int padded = (c.V + kVocabBN - 1) / kVocabBN * kVocabBN;
    const long long h_part = c.T * w.ldp, w_part = c.V * w.ldp;
    if (launch_vocab_split(c.H, c.ldh, c.T, c.D, ws + w.hz_off, hs, c.T, nullptr, most, w.copy_h ? ws + w.h_off : nullptr,
                           w.parts, w.ldp, c.dependent(), c.stream) != cudaSuccess ||
        launch_vocab_split(c.W, c.ldw, c.V, c.D, ws + w.wz_off, vs, padded, most, nullptr, nullptr, 0, w.ldp, c.dependent(),
                           c.stream) != cudaSuccess)
        return SGEMM_ERR_LAUNCH;
    p->h_unscale = hs;
    p->w_unscale = vs;
    p->w_most = most;
    int rc = make_map(c.h, &m->Hz, ws + w.hz_off, SGEMM_DTYPE_BF16, c.D, c.T, w.ldp, 2, h_part, false);
    if (rc == SGEMM_OK) rc = make_map(c.h, &m->W, ws + w.wz_off, SGEMM_DTYPE_BF16, c.D, c.V, w.ldp, 2, w_part, false);
    m->H = m->Hz;
    if (rc == SGEMM_OK && w.copy_h)
        rc = make_map(c.h, &m->H, ws + w.h_off, SGEMM_DTYPE_BF16, c.D, c.T, w.ldp, w.parts, h_part, false);
    return rc;
}

// Operands, targets (the distillation's tables are made first) and what every launch of the call shares.
int begin(const Call &c, const VocabLayout &w, VocabTileParams *p, VocabMaps *m)
{
    char *ws = static_cast<char *>(c.h->workspace);
    if (!w.few) {
        int rc;
        if (w.split) {
            if ((rc = split_operands(c, w, p, m)) != SGEMM_OK) return rc;
        } else {
            if ((rc = map_operand(c, w, w.copy_h, c.H, c.T, c.ldh, w.h_off, &m->H)) != SGEMM_OK) return rc;
            if ((rc = map_operand(c, w, w.copy_w, c.W, c.V, c.ldw, w.w_off, &m->W)) != SGEMM_OK) return rc;
            m->Hz = m->H;
        }
        // where a call has no such matrix, a valid map that no tile uses
        m->G = m->Gz = m->Gw = m->Gzw = m->acc = m->dW = m->W;
        p->f16 = w.split;
    }
    p->T = c.T;
    p->V = c.V;
    p->D = c.D;
    p->dtype = c.dtype;
    p->parts = w.parts;
    p->products = w.products;
    p->f16_products = w.split ? 3 : 1;
    // Segments (vocab_kernels.cu): 1024 deep for logits, 512 for those of FP32 operands, in the loss and in the gradients
    // alike: what truncation takes of a logit is then in lse too and cancels in exp(z - lse), which the label's entry of
    // dZ, p - 1, needs however dZ is rounded afterwards. The loss of a few tokens truncates nothing: their gradients
    // take the label's logit from its kernel (vocab_few.cu) and cut the others, in FP32, 64 deep (24 x 50021 x 4096: 1052
    // us at 512, 1054 at 128, 1063 at 64; a probability at a logit of 50 off by 1.2e-4, 3e-5 and 1.5e-5 of itself). 256
    // for dH and dW of FP32 operands, whole where they are rounded to bfloat16.
    const int whole = 1 << 24;
    p->seg_z = w.split ? w.few_targets ? 1 : 8 : 16;
    p->seg_g = w.split ? 4 : whole;
    p->scale = c.scale;
    p->lse = c.lse;
    p->dloss = c.dloss;
    p->status = c.h->d_status;
    p->timeout_ns = c.h->timeout_ns;
    p->t.labels = c.labels;
    p->t.n = c.n > 0 ? c.n : 1;
    if (c.n > 0) {
        int *tid = reinterpret_cast<int *>(ws + w.tid_off);
        float *tq = reinterpret_cast<float *>(ws + w.tq_off), *tlogq = reinterpret_cast<float *>(ws + w.tlogq_off);
        p->t.id = tid;
        p->t.q = tq;
        p->t.logq = tlogq;
        if (launch_vocab_targets(c.T, c.V, c.n, c.ids, c.logits, c.ldn, c.scale, tid, tq, tlogq, c.dependent(),
                                 c.stream) != cudaSuccess)
            return SGEMM_ERR_LAUNCH;
    }
    return SGEMM_OK;
}

VocabFewParams few_params(const Call &c, const VocabLayout &w, const VocabTileParams &p)
{
    return VocabFewParams{c.T,    c.V,  c.D,         c.H,       c.W, c.ldh,       c.ldw, c.scale, p.t,
                          p.part, p.zt, w.stat_cols, w.targets, 0,   c.h->d_status};
}

bool few_vec(const Call &c) { return (problem(c).align_flags & 3) == 3; }

int ceil_div(int a, int b) { return a / b + (a % b != 0); }

int run_loss(const Call &c)
{
    int rc = check(c, false);
    if (rc != SGEMM_OK) return rc;
    if (c.T == 0) return SGEMM_OK;
    DeviceGuard g(c.h->device);
    if (!g.ok) return SGEMM_ERR_CUDA;
    const VocabLayout w = vocab_layout(problem(c));
    if ((rc = ensure_workspace(c.h, static_cast<size_t>(w.pub.workspace_bytes), c.stream)) != SGEMM_OK) return rc;
    char *ws = static_cast<char *>(c.h->workspace);
    VocabTileParams p{};
    VocabMaps m;
    if ((rc = begin(c, w, &p, &m)) != SGEMM_OK) return rc;
    p.z_kind = kVocabLoss;
    p.z_tm = ceil_div(c.T, 128 * w.ctas);
    p.z_tn = ceil_div(c.V, kVocabBN);
    p.z_items = p.z_tm * p.z_tn;
    p.part = reinterpret_cast<float2 *>(ws + w.part_off);
    p.zt = reinterpret_cast<float *>(ws + w.zt_off);
    p.stat_cols = w.stat_cols;
    if (w.few) {
        const VocabFewParams f = few_params(c, w, p);
        if (launch_vocab_few(f, c.dtype, few_vec(c), c.h->num_sms, c.dependent(), c.stream) != cudaSuccess) return SGEMM_ERR_LAUNCH;
    } else if (launch_vocab_tiles(m, p, w.ctas, w.workers, c.dependent(), c.stream) != cudaSuccess) {
        return SGEMM_ERR_LAUNCH;
    }
    if (launch_vocab_combine(c.T, c.V, p.t, p.part, w.stat_cols, p.zt, c.mult, c.loss, c.lse_out, c.stream) != cudaSuccess)
        return SGEMM_ERR_LAUNCH;
    return SGEMM_OK;
}

int run_grad(const Call &c)
{
    int rc = check(c, true);
    if (rc != SGEMM_OK) return rc;
    if (c.dH == nullptr && c.dW == nullptr) return SGEMM_OK;
    DeviceGuard g(c.h->device);
    if (!g.ok) return SGEMM_ERR_CUDA;
    if (c.T == 0) {
        if (c.dW != nullptr && launch_vocab_finish(c.V, c.D, nullptr, 0, 0, 0, c.beta, c.dW, c.lddw, c.dtype,
                                                   c.dependent(), c.stream) != cudaSuccess)
            return SGEMM_ERR_LAUNCH;
        return SGEMM_OK;
    }
    const VocabLayout w = vocab_layout(problem(c));
    if ((rc = ensure_workspace(c.h, static_cast<size_t>(w.pub.workspace_bytes), c.stream)) != SGEMM_OK) return rc;
    char *ws = static_cast<char *>(c.h->workspace);
    VocabTileParams p{};
    VocabMaps m;
    if ((rc = begin(c, w, &p, &m)) != SGEMM_OK) return rc;
    if (w.few_targets) {
        p.zt = reinterpret_cast<float *>(ws + w.zt_off);
        if (launch_vocab_few_targets(few_params(c, w, p), c.dtype, few_vec(c), c.dependent(), c.stream) != cudaSuccess)
            return SGEMM_ERR_LAUNCH;
    }
    const int bm = 128 * w.ctas, tm = ceil_div(c.T, bm), tn = ceil_div(c.D, kVocabBN);
    const int elem = c.dtype == SGEMM_DTYPE_BF16 ? 2 : 4;
    p.z_kind = kVocabDz;
    p.z_tm = tm;
    p.g_blocks = w.g_blocks;
    const long long acc_split = c.T * w.ldacc;
    // dZ in blocks of 64 entries, T x 64 each: every copy of it is one contiguous piece of memory
    auto dz_map = [&](CUtensorMap *map, long long off, int parts, bool result) {
        return make_map(c.h, map, ws + off, SGEMM_DTYPE_BF16, 64, c.T, 64, parts * w.g_blocks, 64LL * c.T, result);
    };
    // as dW and as dH read it: the same for bfloat16 operands
    auto dz_maps = [&](CUtensorMap *map, CUtensorMap *map_dh, int i, bool result) {
        int e = SGEMM_OK;
        if (!w.split || c.dW != nullptr) e = dz_map(map, w.g_off[i], w.parts, result);
        *map_dh = *map;
        if (e == SGEMM_OK && w.split && c.dH != nullptr) e = dz_map(map_dh, w.gz_off[i], 2, result);
        return e;
    };
    float *acc = reinterpret_cast<float *>(ws + w.acc_off);
    p.dW = c.dW;
    p.lddw = c.lddw;
    p.dw_tma = c.beta == 0.0f && aligned(c.dW, 16) && static_cast<long long>(c.lddw) * elem % 16 == 0;
    p.dw_vec = aligned(c.dW, 4 * elem) && c.lddw % 4 == 0;
    p.alpha = c.mult * c.scale;
    p.beta = c.beta;
    p.dw_tn = c.dW != nullptr ? tn : 0;  // 0: no such gradient
    p.dh_tm = c.dH != nullptr ? tm : 0;
    p.dh_tn = tn;
    p.dh_kb = w.dh_kb;
    p.dh_splits = w.dh_splits;
    if (c.dW != nullptr && p.dw_tma &&
        (rc = make_map(c.h, &m.dW, c.dW, c.dtype, c.D, c.V, c.lddw, 1, static_cast<long long>(c.lddw) * c.V, true)) !=
            SGEMM_OK)
        return rc;
    if (c.dH != nullptr && (rc = make_map(c.h, &m.acc, acc, SGEMM_DTYPE_F32, c.D, c.T, w.ldacc, w.dh_splits, acc_split,
                                          true)) != SGEMM_OK)
        return rc;
    // Launch i: the dH and dW tiles of piece i - 1 and the dZ tiles of piece i.
    for (int i = 0; i <= w.pub.pieces; ++i) {
        p.dh_items = p.dw_items = p.z_items = 0;
        if (i > 0) {
            p.g_v0 = (i - 1) * w.pub.piece;
            p.g_vn = c.V - p.g_v0 < w.pub.piece ? c.V - p.g_v0 : w.pub.piece;
            const int splits = ceil_div(ceil_div(p.g_vn, kVocabBK), w.dh_kb > 0 ? w.dh_kb : 1);
            if (c.dH != nullptr) p.dh_items = tm * tn * splits;
            if (c.dW != nullptr) p.dw_items = ceil_div(p.g_vn, bm) * tn;
            p.acc_add = i > 1;
            if ((rc = dz_maps(&m.G, &m.Gz, (i - 1) & 1, false)) != SGEMM_OK) return rc;
        }
        if (i < w.pub.pieces) {
            p.z_v0 = i * w.pub.piece;
            p.z_tn = ceil_div(c.V - p.z_v0 < w.pub.piece ? c.V - p.z_v0 : w.pub.piece, kVocabBN);
            p.z_items = tm * p.z_tn;
            if ((rc = dz_maps(&m.Gw, &m.Gzw, i & 1, true)) != SGEMM_OK) return rc;
        }
        const int others = p.dw_items + p.z_items, rem = p.dh_items % w.workers;
        const int cost = vocab_cost(c.dW != nullptr ? c.T : c.D);
        const int own = w.products == 6 && c.dW != nullptr ? w.dh_kb / 2 : w.dh_kb;  // a k-block of dW has twice the products
        p.dh_extra = p.dh_items > 0 && rem > 0 ? std::min((own + cost / 2) / cost, others / (w.workers - rem)) : 0;
        if (launch_vocab_tiles(m, p, w.ctas, w.workers, c.dependent(), c.stream) != cudaSuccess) return SGEMM_ERR_LAUNCH;
    }
    if (c.dH != nullptr && launch_vocab_finish(c.T, c.D, acc, w.ldacc, acc_split, w.dh_splits, c.beta, c.dH, c.lddh,
                                               c.dtype, c.dependent(), c.stream) != cudaSuccess)
        return SGEMM_ERR_LAUNCH;
    return SGEMM_OK;
}

Call operands(sgemm_handle_t h, int T, int V, int D, int dtype, const void *H, int ldh, const void *W, int ldw,
              cudaStream_t stream)
{
    Call c{};
    c.h = h;
    c.T = T;
    c.V = V;
    c.D = D;
    c.dtype = dtype;
    c.H = H;
    c.ldh = ldh;
    c.W = W;
    c.ldw = ldw;
    c.stream = stream;
    return c;
}

// 1 / temperature and temperature^2; a temperature that is not positive and finite gives NaN, which check() refuses.
void set_distill(Call *c, int n, const long long *ids, const float *logits, int ldn, float temperature)
{
    c->n = n;
    c->ids = ids;
    c->logits = logits;
    c->ldn = ldn;
    const bool good = temperature > 0.0f && std::isfinite(temperature);
    c->scale = good ? 1.0f / temperature : NAN;
    c->mult = good ? temperature * temperature : NAN;
}

void set_grad(Call *c, const float *lse, const float *dloss, float beta, void *dH, int lddh, void *dW, int lddw)
{
    c->lse = lse;
    c->dloss = dloss;
    c->beta = beta;
    c->dH = dH;
    c->lddh = lddh;
    c->dW = dW;
    c->lddw = lddw;
}

}  // namespace

extern "C" {

int sgemm_xent(sgemm_handle_s *h, int T, int V, int D, int dtype, const void *H, int ldh, const void *W, int ldw,
               const long long *labels, float scale, float *loss, float *lse, CUstream_st *stream)
{
    Call c = operands(h, T, V, D, dtype, H, ldh, W, ldw, stream);
    c.labels = labels;
    c.scale = scale;
    c.loss = loss;
    c.lse_out = lse;
    return run_loss(c);
}

int sgemm_xent_grad(sgemm_handle_s *h, int T, int V, int D, int dtype, const void *H, int ldh, const void *W, int ldw,
                    const long long *labels, float scale, const float *lse, const float *dloss, float beta, void *dH,
                    int lddh, void *dW, int lddw, CUstream_st *stream)
{
    Call c = operands(h, T, V, D, dtype, H, ldh, W, ldw, stream);
    c.labels = labels;
    c.scale = scale;
    set_grad(&c, lse, dloss, beta, dH, lddh, dW, lddw);
    return run_grad(c);
}

int sgemm_distill(sgemm_handle_s *h, int T, int V, int D, int dtype, const void *H, int ldh, const void *W, int ldw,
                  int n, const long long *ids, const float *logits, int ldn, float temperature, float *loss, float *lse,
                  CUstream_st *stream)
{
    if (n < 1) return SGEMM_ERR_INVALID_VALUE;
    Call c = operands(h, T, V, D, dtype, H, ldh, W, ldw, stream);
    set_distill(&c, n, ids, logits, ldn, temperature);
    c.loss = loss;
    c.lse_out = lse;
    return run_loss(c);
}

int sgemm_distill_grad(sgemm_handle_s *h, int T, int V, int D, int dtype, const void *H, int ldh, const void *W,
                       int ldw, int n, const long long *ids, const float *logits, int ldn, float temperature,
                       const float *lse, const float *dloss, float beta, void *dH, int lddh, void *dW, int lddw,
                       CUstream_st *stream)
{
    if (n < 1) return SGEMM_ERR_INVALID_VALUE;
    Call c = operands(h, T, V, D, dtype, H, ldh, W, ldw, stream);
    set_distill(&c, n, ids, logits, ldn, temperature);
    set_grad(&c, lse, dloss, beta, dH, lddh, dW, lddw);
    return run_grad(c);
}

}  // extern "C"
