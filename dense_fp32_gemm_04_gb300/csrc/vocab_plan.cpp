// Host-only planning of the vocabulary losses: argument checks that need no
// pointer, the pieces of the vocabulary, the workspace's layout. Contract:
// include/sgemm_vocab.h.
#include <algorithm>

#include "vocab_internal.h"

namespace sgemm_impl {

namespace {

// dZ of one piece of the vocabulary is at most this large (and a piece at least one tile column).
constexpr long long kPieceBytes = 256LL << 20;
constexpr int kTile = 64;

long long round_up(long long x, long long to) { return (x + to - 1) / to * to; }

}  // namespace

int validate_vocab(const VocabProblem &q)
{
    if (q.T < 0 || q.V < 1 || q.D < 1 || q.n < 0) return SGEMM_ERR_INVALID_VALUE;
    if (q.dtype != SGEMM_DTYPE_F32 && q.dtype != SGEMM_DTYPE_BF16) return SGEMM_ERR_INVALID_VALUE;
    if (q.align_flags < 0 || q.align_flags > 3 || q.num_sms < 1) return SGEMM_ERR_INVALID_VALUE;
    if (q.math_mode != SGEMM_MATH_FP32 && q.math_mode != SGEMM_MATH_TF32) return SGEMM_ERR_INVALID_VALUE;
    if (q.n > SGEMM_DISTILL_MAX_ENTRIES) return SGEMM_ERR_NOT_SUPPORTED;
    return SGEMM_OK;
}

VocabLayout vocab_layout(const VocabProblem &q)
{
    VocabLayout w{};
    const long long T = q.T;
    long long at = 0;
    auto take = [&](long long bytes) {
        const long long off = at;
        at = round_up(at + bytes, 256);
        return off;
    };
    const bool grad = q.dh || q.dw;
    if (q.n > 0) {
        w.tid_off = take(T * q.n * 4);
        w.tq_off = take(T * q.n * 4);
        w.tlogq_off = take(T * q.n * 4);
    }
    if (!grad) {
        w.parts = (q.V + kTile - 1) / kTile;
        w.zt_off = take(T * std::max(1, q.n) * 4);
        w.part_off = take(T * w.parts * 8);
        w.pub.pieces = 1;
        w.pub.piece = q.V;
        w.pub.launches = T > 0 ? 2 + (q.n > 0) : 0;
    } else {
        const long long fit = std::max<long long>(kPieceBytes / 4 / std::max<long long>(T, 1), kTile);
        const int piece = static_cast<int>(std::min<long long>(fit / kTile * kTile, round_up(q.V, kTile)));
        w.pub.piece = std::min(piece, q.V);
        w.pub.pieces = (q.V + piece - 1) / piece;
        w.ldg = round_up(w.pub.piece, kTile);
        w.g_off = take(T * w.ldg * 4);
        if (q.dh) w.acc_off = take(T * q.D * 4);
        w.pub.launches = T > 0 ? w.pub.pieces * (1 + q.dh + q.dw) + q.dh + (q.n > 0) : q.dw;
    }
    w.pub.workspace_bytes = at;
    return w;
}

}  // namespace sgemm_impl

extern "C" int sgemm_vocab_plan(int T, int V, int D, int dtype, int n, int grad, int align_flags, int num_sms,
                                int math_mode, sgemm_vocab_plan_t *out)
{
    using namespace sgemm_impl;
    if (out == nullptr || (grad != 0 && grad != 1)) return SGEMM_ERR_INVALID_VALUE;
    const VocabProblem q{T, V, D, dtype, n, grad != 0, grad != 0, align_flags, num_sms, math_mode};
    const int rc = validate_vocab(q);
    if (rc != SGEMM_OK) return rc;
    *out = vocab_layout(q).pub;
    return SGEMM_OK;
}
