// Host-only planning of the vocabulary losses: argument checks that need no
// pointer, the pieces of the vocabulary, the workspace's layout. Contract:
// include/sgemm_vocab.h.
#include <algorithm>

#include "vocab_internal.h"

namespace sgemm_impl {

namespace {

// dZ of the pieces of the vocabulary that are alive, in all the parts that are held of it, takes twice this much at most
// (but a piece is at least one tile wide): the whole vocabulary in one piece where it fits that, else pieces of one size,
// two of them alive at a time. A launch still has many rounds of tiles (training 4096 tokens, 131072 x 4096 in bfloat16:
// the same time within 2 % with pieces of 128 MB to 1 GB; 2048 x 32768 x 2048 in FP32 2.71 ms with two pieces of 425 MB, 2.74
// with three; 1000 x 32003 x 1001 738 us with one of 320 MB, 778 with two). Beside it a call holds what its operands and
// dH's partial sums take, so for FP32, whose parts of W are as large as W, and for a few hundred tokens the workspace can be
// larger than the logits would be.
constexpr long long kPieceBytes = 256LL << 20;

// From this many tokens on bfloat16 rows that do not start on 128-byte lines are copied to rows that do, though the copy
// engine could read them: a slab's row is then one line and not parts of two (50000 x 1496, loss in us, read as they are
// / with the copies: 2048 tokens 242 / 232, 4096 tokens 446 / 399; gradients 589 / 590 and 1155 / 1110; with rows on
// lines from the start 337 and 1030 at 4096 tokens).
constexpr int kLineTokens = 2048;

long long round_up(long long x, long long to) { return (x + to - 1) / to * to; }

}  // namespace

int validate_vocab(const VocabProblem &q)
{
    if (q.T < 0 || q.V < 1 || q.D < 1 || q.n < 0) return SGEMM_ERR_INVALID_VALUE;
    if (q.dtype != SGEMM_DTYPE_F32 && q.dtype != SGEMM_DTYPE_BF16) return SGEMM_ERR_INVALID_VALUE;
    if (q.align_flags < 0 || q.align_flags > 15 || q.num_sms < 1) return SGEMM_ERR_INVALID_VALUE;
    if (q.math_mode != SGEMM_MATH_FP32 && q.math_mode != SGEMM_MATH_TF32) return SGEMM_ERR_INVALID_VALUE;
    if (q.n > SGEMM_DISTILL_MAX_ENTRIES) return SGEMM_ERR_NOT_SUPPORTED;
    // tiles and coordinates are counted in 32 bits
    const long long tiles_t = q.T / 128 + 1LL, tiles_v = q.V / 128 + 1LL, tiles_d = q.D / 128 + 1LL;
    for (long long x : {tiles_t * tiles_v, tiles_t * tiles_d, tiles_v * tiles_d})
        if (x > 1LL << 30) return SGEMM_ERR_NOT_SUPPORTED;
    if (q.T > 0x7fff0000 || q.V > 0x7fff0000 || q.D > 0x7fff0000) return SGEMM_ERR_NOT_SUPPORTED;
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
    // A pair's 256 rows cost less per row than a CTA's 128, but a last pair that is half empty costs the whole: the
    // loss takes single CTAs where the tokens end in the first half of one of up to three pairs (131072 x 4096, us with
    // single CTAs / pairs: 128 tokens 173 / 178, 256 tokens 202 / 184, 384 tokens 281 / 300, 640 tokens 448 / 450, 768
    // tokens 525 / 460). Of the gradient's products only one has its rows counted in tokens, and with few tokens the
    // wider tiles wait for operands: single CTAs up to 384 tokens (128 tokens 626 / 687, 256 tokens 699 / 741, 300
    // tokens 867 / 894, 384 tokens 974 / 933, but 203 / 206 at 50021 x 2048 and 86 / 88 at 32768 x 1024; 500 tokens
    // 1187 / 981).
    const int pairs = q.pairs > 0 ? q.pairs : q.pairs < 0 ? 0 : q.num_sms / 2;
    const long long halves = (T + 127) / 128;
    const bool single = grad ? halves <= 3 : halves % 2 == 1 && halves <= 5;
    w.ctas = single || pairs == 0 ? 1 : 2;
    w.workers = w.ctas == 2 ? pairs : q.num_sms;
    const int bm = 128 * w.ctas;

    const int few = f32 ? kFewTokensF32 : (q.align_flags & 3) == 3 ? kFewTokensBf16 : kFewTokensCopied;
    w.few = !grad && T <= few;
    w.few_targets = grad && T <= few;
    w.split = f32 && !w.few;
    const int lines = T >= kLineTokens ? 5 : 1;  // the flags that spare H's copy; W's are the next bits
    w.copy_h = f32 ? w.split && q.dw : !w.few && (q.align_flags & lines) != lines;
    w.copy_w = !f32 && !w.few && (q.align_flags >> 1 & lines) != lines;
    w.ldp = round_up(q.D, 64);  // whole 128-byte lines: a copied row of a slab is one of them, not parts of two
    if (w.copy_h) w.h_off = take(w.parts * T * w.ldp * 2);
    if (w.copy_w) w.w_off = take(w.parts * static_cast<long long>(q.V) * w.ldp * 2);
    if (w.split) {
        w.hz_off = take(2 * T * w.ldp * 2);
        w.wz_off = take(2 * static_cast<long long>(q.V) * w.ldp * 2);
        w.hs_off = take(T * 4);
        w.ws_off = take(256 + round_up(q.V, kVocabBN) * 4);
    }
    if (q.n > 0) {
        w.tid_off = take(T * q.n * 4);
        w.tq_off = take(T * q.n * 4);
        w.tlogq_off = take(T * q.n * 4);
    }
    int launches = (w.split ? 2 : w.copy_h + w.copy_w) + (q.n > 0);
    if (w.few || w.few_targets) w.targets = static_cast<int>(T * std::max(1, q.n));
    if (w.few_targets) w.zt_off = take(T * std::max(1, q.n) * 4);
    if (!grad) {
        w.stat_cols = w.few ? vocab_few_warps(q.T, q.num_sms) : 2 * ((q.V + kVocabBN - 1) / kVocabBN);
        w.zt_off = take(T * std::max(1, q.n) * 4);
        w.part_off = take(T * w.stat_cols * 8);
        w.pub.pieces = 1;
        w.pub.piece = q.V;
        launches = T > 0 ? launches + 2 : 0;
    } else {
        const int held = (q.dw || !w.split ? w.parts : 0) + (w.split && q.dh ? 2 : 0);  // for dW or both; float16 for dH
        const long long column = 2LL * held * std::max<long long>(T, 1), all = round_up(q.V, kVocabBN);
        long long piece = all;
        if (q.piece > 0) {
            piece = std::min(round_up(q.piece, kVocabBN), all);
        } else if (all * column > 2 * kPieceBytes) {
            const long long fit = std::max<long long>(kPieceBytes / column / kVocabBN, 1) * kVocabBN;
            const long long pieces = (q.V + fit - 1) / fit;
            piece = round_up((q.V + pieces - 1) / pieces, kVocabBN);
        }
        w.pub.piece = static_cast<int>(std::min<long long>(piece, q.V));
        w.pub.pieces = static_cast<int>((q.V + piece - 1) / piece);
        w.g_blocks = static_cast<int>(piece / 64);
        for (int i = 0; i < std::min(w.pub.pieces, 2); ++i) {
            w.g_off[i] = q.dw || !w.split ? take(w.parts * T * piece * 2) : 0;
            w.gz_off[i] = w.split ? q.dh ? take(2 * T * piece * 2) : 0 : w.g_off[i];
        }
        if (q.dh) {
            // A dH tile's K range is a piece of the vocabulary, the other tiles' are T and D. It is split so far
            // that no part of it takes a worker more than half its share of a launch (the other tiles fill what
            // that leaves uneven), a quarter where there are no others; every split costs a pass over T x D sums.
            const int kblocks = (w.pub.piece + kVocabBK - 1) / kVocabBK;
            const long long tm = (T + bm - 1) / bm, tn = (q.D + kVocabBN - 1) / kVocabBN;
            const long long own = tm * tn * kblocks * 3 / (w.products == 6 ? 6 : 3);  // in units of a k-block of dW
            const long long others = q.dw ? (w.pub.piece + bm - 1) / bm * tn * vocab_cost(q.T) : 0;
            const long long share = (own + others) / w.workers / (q.dw ? 2 : 4);
            const long long longest = (w.products == 6 ? 2 : 1) * std::max<long long>(4, share);
            const long long s = std::max<long long>(1, (kblocks + longest - 1) / longest);
            w.dh_kb = static_cast<int>((kblocks + s - 1) / s);
            w.dh_splits = (kblocks + w.dh_kb - 1) / w.dh_kb;
            w.ldacc = round_up(q.D, 4);
            w.acc_off = take(w.dh_splits * T * w.ldacc * 4);
        }
        launches = T > 0 ? launches + w.few_targets + w.pub.pieces + 1 + q.dh : q.dw;
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
    VocabProblem q{T, V, D, dtype, n, grad != 0, grad != 0, align_flags, num_sms, math_mode, 0, 0};
    const int rc = validate_vocab(q);
    if (rc != SGEMM_OK) return rc;
    *out = vocab_layout(q).pub;
    // A call for one gradient alone splits its work differently, and so does one on a machine that holds no CTA pairs (fewer
    // pairs than half the SMs split it less): the workspace fits them too.
    for (int pairs : {0, -1}) {
        q.pairs = pairs;
        for (int one : {0, 1, 2}) {
            q.dh = grad != 0 && one != 1;
            q.dw = grad != 0 && one != 2;
            out->workspace_bytes = std::max(out->workspace_bytes, vocab_layout(q).pub.workspace_bytes);
        }
    }
    return SGEMM_OK;
}
