// C ABI of the vocabulary losses: argument checks, workspace, launches.
// Declarations and contracts: include/sgemm_vocab.h.
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
};

bool aligned(const void *p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

VocabProblem problem(const Call &c)
{
    const int size = c.dtype == SGEMM_DTYPE_BF16 ? 2 : 4;
    auto rows16 = [size](const void *p, long long ld) { return aligned(p, 16) && ld * size % 16 == 0; };
    const int align = (rows16(c.H, c.ldh) ? 1 : 0) | (rows16(c.W, c.ldw) ? 2 : 0);
    return VocabProblem{c.T, c.V, c.D, c.dtype, c.n, c.dH != nullptr, c.dW != nullptr, align, c.h->num_sms,
                        c.h->math_mode};
}

int check(const Call &c, bool grad)
{
    if (c.h == nullptr) return SGEMM_ERR_INVALID_VALUE;
    const int rc = validate_vocab(problem(c));
    if (rc != SGEMM_OK) return rc;
    const unsigned size = c.dtype == SGEMM_DTYPE_BF16 ? 2 : 4;
    if (c.ldh < c.D || c.ldw < c.D || (c.n > 0 && c.ldn < c.n)) return SGEMM_ERR_INVALID_VALUE;
    if (!std::isfinite(c.scale) || !std::isfinite(c.mult) || c.mult == 0.0f || !std::isfinite(c.beta))
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
    return SGEMM_OK;
}

// Targets (the distillation's tables are made first) and the parameters every tile kernel shares.
int begin(const Call &c, const VocabLayout &w, VocabTileParams *p)
{
    char *ws = static_cast<char *>(c.h->workspace);
    p->T = c.T;
    p->V = c.V;
    p->D = c.D;
    p->H = c.H;
    p->W = c.W;
    p->ldh = c.ldh;
    p->ldw = c.ldw;
    p->scale = c.scale;
    p->lse = c.lse;
    p->dloss = c.dloss;
    p->gmult = c.mult * c.scale;
    p->v0 = 0;
    p->vn = c.V;
    p->t.labels = c.labels;
    p->t.n = c.n > 0 ? c.n : 1;
    if (c.n > 0) {
        int *tid = reinterpret_cast<int *>(ws + w.tid_off);
        float *tq = reinterpret_cast<float *>(ws + w.tq_off), *tlogq = reinterpret_cast<float *>(ws + w.tlogq_off);
        p->t.id = tid;
        p->t.q = tq;
        p->t.logq = tlogq;
        if (launch_vocab_targets(c.T, c.V, c.n, c.ids, c.logits, c.ldn, c.scale, tid, tq, tlogq, c.stream) != cudaSuccess)
            return SGEMM_ERR_LAUNCH;
    }
    return SGEMM_OK;
}

int run_loss(const Call &c)
{
    int rc = check(c, false);
    if (rc != SGEMM_OK) return rc;
    if (c.T == 0) return SGEMM_OK;
    DeviceGuard g(c.h->device);
    if (!g.ok) return SGEMM_ERR_CUDA;
    VocabProblem q = problem(c);
    const VocabLayout w = vocab_layout(q);
    if ((rc = ensure_workspace(c.h, static_cast<size_t>(w.pub.workspace_bytes), c.stream)) != SGEMM_OK) return rc;
    char *ws = static_cast<char *>(c.h->workspace);
    VocabTileParams p{};
    if ((rc = begin(c, w, &p)) != SGEMM_OK) return rc;
    p.part = reinterpret_cast<float2 *>(ws + w.part_off);
    p.zt = reinterpret_cast<float *>(ws + w.zt_off);
    if (launch_vocab_forward(p, c.dtype, c.stream) != cudaSuccess) return SGEMM_ERR_LAUNCH;
    if (launch_vocab_combine(c.T, c.V, p.t, p.part, w.parts, p.zt, c.mult, c.loss, c.lse_out, c.stream) != cudaSuccess)
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
        if (c.dW != nullptr && launch_vocab_finish(c.V, c.D, nullptr, 0, c.beta, c.dW, c.lddw, c.dtype, c.h->num_sms,
                                                   c.stream) != cudaSuccess)
            return SGEMM_ERR_LAUNCH;
        return SGEMM_OK;
    }
    VocabProblem q = problem(c);
    const VocabLayout w = vocab_layout(q);
    if ((rc = ensure_workspace(c.h, static_cast<size_t>(w.pub.workspace_bytes), c.stream)) != SGEMM_OK) return rc;
    char *ws = static_cast<char *>(c.h->workspace);
    VocabTileParams p{};
    if ((rc = begin(c, w, &p)) != SGEMM_OK) return rc;
    p.G = reinterpret_cast<float *>(ws + w.g_off);
    p.ldg = w.ldg;
    float *acc = reinterpret_cast<float *>(ws + w.acc_off);
    for (int i = 0; i < w.pub.pieces; ++i) {
        p.v0 = i * w.pub.piece;
        p.vn = c.V - p.v0 < w.pub.piece ? c.V - p.v0 : w.pub.piece;
        if (launch_vocab_dz(p, c.dtype, c.stream) != cudaSuccess) return SGEMM_ERR_LAUNCH;
        if (c.dH != nullptr && launch_vocab_dh(p, c.dtype, acc, i == 0, c.stream) != cudaSuccess) return SGEMM_ERR_LAUNCH;
        if (c.dW != nullptr && launch_vocab_dw(p, c.dtype, c.beta, c.dW, c.lddw, c.stream) != cudaSuccess)
            return SGEMM_ERR_LAUNCH;
    }
    if (c.dH != nullptr &&
        launch_vocab_finish(c.T, c.D, acc, c.D, c.beta, c.dH, c.lddh, c.dtype, c.h->num_sms, c.stream) != cudaSuccess)
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
