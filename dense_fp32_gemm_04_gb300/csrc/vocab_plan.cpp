// Host-only planning of the vocabulary losses: argument checks that need no
// pointer, the pieces of the vocabulary, the workspace's layout. Contract:
// include/sgemm_vocab.h.
#include <algorithm>

#include "vocab_internal.h"

namespace sgemm_impl {

namespace {

// dZ of one piece of the vocabulary takes about this much at most (a piece is at least one tile wide), so that
// two pieces' dZ stay a small part of the logits' size while a launch still has many rounds of tiles.
constexpr long long kPieceBytes = 256LL << 20;

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
        at = round_up(at + bytes, 1024);
        return off;
    };
    const bool grad = q.dh || q.dw;
    const bool f32 = q.dtype == SGEMM_DTYPE_F32;
    w.parts = !f32 ? 1 : q.math_mode == SGEMM_MATH_TF32 ? 2 : 3;
    w.products = w.parts * (w.parts + 1) / 2;
    // Up to 128 tokens fill the rows of one CTA's tile: a pair would compute 128 rows of nothing.
    const int pairs = q.pairs > 0 ? q.pairs : q.pairs < 0 ? 0 : q.num_sms / 2;
    w.ctas = T > 128 && pairs > 0 ? 2 : 1;
    w.workers = w.ctas == 2 ? pairs : q.num_sms;
    const int bm = 128 * w.ctas;

    w.copy_h = f32 || !(q.align_flags & 1);
    w.copy_w = f32 || !(q.align_flags & 2);
    w.ldh = w.ldw = round_up(q.D, 8);
    if (w.copy_h) w.h_off = take(w.parts * T * w.ldh * 2);
    if (w.copy_w) w.w_off = take(w.parts * static_cast<long long>(q.V) * w.ldw * 2);
    if (q.n > 0) {
        w.tid_off = take(T * q.n * 4);
        w.tq_off = take(T * q.n * 4);
        w.tlogq_off = take(T * q.n * 4);
    }
    int launches = w.copy_h + w.copy_w + (q.n > 0);
    if (!grad) {
        w.stat_cols = 2 * ((q.V + kVocabBN - 1) / kVocabBN);
        w.zt_off = take(T * std::max(1, q.n) * 4);
        w.part_off = take(T * w.stat_cols * 8);
        w.pub.pieces = 1;
        w.pub.piece = q.V;
        launches = T > 0 ? launches + 2 : 0;
    } else {
        const long long fit = std::max<long long>(kPieceBytes / (2 * w.parts) / std::max<long long>(T, 1), kVocabBN);
        const long long piece = std::min<long long>(fit / kVocabBN * kVocabBN, round_up(q.V, kVocabBN));
        w.pub.piece = static_cast<int>(std::min<long long>(piece, q.V));
        w.pub.pieces = static_cast<int>((q.V + piece - 1) / piece);
        w.ldg = piece;
        w.g_off[0] = take(w.parts * T * w.ldg * 2);
        w.g_off[1] = w.pub.pieces > 1 ? take(w.parts * T * w.ldg * 2) : w.g_off[0];
        if (q.dh) {
            // A dH tile's K range is a piece of the vocabulary, the other tiles' are T and D: it is split
            // until its parts are about as long, and until there are two rounds of them, but not below 4 k-blocks.
            const int kblocks = (w.pub.piece + kVocabBK - 1) / kVocabBK;
            const long long tiles = ((T + bm - 1) / bm) * ((q.D + kVocabBN - 1) / kVocabBN);
            const long long even = (w.pub.piece + std::max<long long>({T, q.D, 1024}) - 1) / std::max<long long>({T, q.D, 1024});
            const long long fill = tiles > 0 ? (2LL * w.workers + tiles - 1) / tiles : 1;
            const long long s = std::min<long long>(std::max(even, fill), std::max(1, kblocks / 4));
            w.dh_kb = static_cast<int>((kblocks + s - 1) / s);
            w.dh_splits = (kblocks + w.dh_kb - 1) / w.dh_kb;
            w.ldacc = round_up(q.D, 4);
            w.acc_off = take(w.dh_splits * T * w.ldacc * 4);
        }
        launches = T > 0 ? launches + w.pub.pieces + 1 + q.dh : q.dw;
    }
    w.pub.launches = launches;
    w.pub.workspace_bytes = at;
    return w;
}

}  // namespace sgemm_impl

extern "C" int sgemm_vocab_plan(int T, int V, int D, int dtype, int n, int grad, int align_flags, int num_sms,
                                int math_mode, sgemm_vocab_plan_t *out)
{
    using namespace sgemm_impl;
    if (out == nullptr || (grad != 0 && grad != 1)) return SGEMM_ERR_INVALID_VALUE;
    const VocabProblem q{T, V, D, dtype, n, grad != 0, grad != 0, align_flags, num_sms, math_mode, 0};
    const int rc = validate_vocab(q);
    if (rc != SGEMM_OK) return rc;
    *out = vocab_layout(q).pub;
    return SGEMM_OK;
}
