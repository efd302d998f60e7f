// Host-only planning of the linear layers: argument checks that need no pointer, the
// form of each product, the workspace's layout. Contract: include/sgemm_linear.h.
#include <algorithm>

#include "linear_internal.h"

namespace sgemm_impl {

namespace {

long long round_up(long long x, long long to) { return (x + to - 1) / to * to; }
long long ceil_div(long long x, long long by) { return (x + by - 1) / by; }

// Clusters of c CTAs of the split kernel that a GB300 holds at once: 152 SMs, in groups that clusters do not straddle.
constexpr int kClusters[kLinearMaxSplits] = {152, 76, 46, 36, 28, 23, 15, 15};

// How a product of rows x cols over K runs. With no more than half as many tiles as SMs their K ranges are split over
// clusters, as far as all clusters are resident at once (a second round would double the time: 48 x 2048 x 8192 in 8 parts,
// 16 clusters where 15 fit, 23 us) and there are slabs to split. Tiles of half the width where that keeps more SMs busy,
// or for one row of tiles as many with fewer parts to add (16 x 4096 x 4096: 22 us in 8 parts of 256 columns, 12.6 in 4
// of 128). With more tiles they are whole, on the form that ends first.
LinearShape shape_of(long long rows, long long cols, long long K, const LinearProblem &q, int pairs)
{
    const long long m = ceil_div(rows, 128), n = ceil_div(cols, kLinearBN), single = m * n, half = m * ceil_div(cols, 128);
    LinearShape s{0, 1, kLinearBN};
    if (2 * single <= q.num_sms) {
        auto parts = [&](long long tiles) {
            long long c = std::min<long long>(ceil_div(K, kLinearBK), kLinearMaxSplits);
            while (c > 1 && tiles > (q.clusters != nullptr ? q.clusters[c - 1] : kClusters[c - 1] * q.num_sms / 152)) --c;
            return c;
        };
        const long long wide = parts(single) * single, narrow = half <= q.num_sms ? parts(half) * half : 0;
        if (m == 1 ? narrow >= wide : narrow > wide) s.bn = 128;
        s.splits = static_cast<int>(parts(s.bn == 128 ? half : single));
        return s;
    }
    // rounds of tiles, times a tile's: a slab takes the tensor core 2 cycles a column, and as long as its operands take to
    // come, 1 a column and 256 for the rows; beside it the epilogue, which FP32 sums leave nothing to overlap with. Y's tiles
    // may be narrower, so that the last round is full (2047 x 3001 x 1531 in FP32: 96 tiles for 76 pairs, with 160 columns 152).
    const long long slabs = ceil_div(K, kLinearBK) * (q.dtype == SGEMM_DTYPE_F32 ? 3 : 1);
    const long long epilogue = q.dtype == SGEMM_DTYPE_F32 ? 50 : 16;  // cycles a column (FP32, 3000 x 3000 x 256: 38.8 us, with 100 42.2)
    long long best = -1;
    for (int ctas = pairs > 0 ? 2 : 1; ctas >= 1; --ctas) {
        const long long workers = ctas == 2 ? pairs : q.num_sms, tiles = ceil_div(rows, 128 * ctas);
        for (int bn = kLinearBN; bn >= (q.grad ? kLinearBN : 128); bn -= 32) {
            const long long rounds = ceil_div(tiles * ceil_div(cols, bn), workers);
            const long long cost = rounds * (slabs * std::max(2 * bn, 256 + bn) + epilogue * bn);
            if (best < 0 || cost < best) {
                best = cost;
                s.ctas = ctas;
                s.bn = bn;
            }
        }
    }
    return s;
}

}  // namespace

int validate_linear(const LinearProblem &q)
{
    if (q.M < 0 || q.N < 1 || q.K < 1) return SGEMM_ERR_INVALID_VALUE;
    if (q.dtype != SGEMM_DTYPE_F32 && q.dtype != SGEMM_DTYPE_BF16) return SGEMM_ERR_INVALID_VALUE;
    if (q.align_flags < 0 || q.align_flags > 7 || q.num_sms < 1) return SGEMM_ERR_INVALID_VALUE;
    // tiles and coordinates are counted in 32 bits
    const long long tiles_m = q.M / 128 + 1LL, tiles_n = q.N / 128 + 1LL, tiles_k = q.K / 128 + 1LL;
    for (long long x : {tiles_m * tiles_n, tiles_m * tiles_k, tiles_n * tiles_k})
        if (x > 1LL << 29) return SGEMM_ERR_NOT_SUPPORTED;
    if (q.M > 0x7fff0000 || q.N > 0x7fff0000 || q.K > 0x7fff0000) return SGEMM_ERR_NOT_SUPPORTED;
    return SGEMM_OK;
}

LinearLayout linear_layout(const LinearProblem &q)
{
    LinearLayout w{};
    long long at = 0;
    auto take = [&](long long bytes) {
        const long long off = at;
        at = round_up(at + bytes, 1024);
        return off;
    };
    const bool f32 = q.dtype == SGEMM_DTYPE_F32;
    const int pairs = q.pairs > 0 ? q.pairs : q.pairs < 0 ? 0 : q.num_sms / 2;
    w.y = w.dx = w.dw = LinearShape{0, 1, kLinearBN};
    w.few = !q.grad && linear_is_few(q.M, q.N, q.K, f32);
    w.ldk = round_up(q.K, 64);  // whole 128-byte lines
    w.ldn = round_up(q.N, 64);
    w.strips = static_cast<int>(ceil_div(q.M, kLinearStrip));
    int launches = 0;
    if (q.M == 0) {
        launches = q.grad ? q.dw + q.db : 0;
    } else if (w.few) {
        launches = 1;
    } else {
        w.split = f32;
        const bool x = !q.grad || q.dw, m = !q.grad || q.dx;  // operands of the call
        w.copy_x = x && (f32 || !(q.align_flags & 1));
        w.copy_w = m && (f32 || !(q.align_flags & 2));
        w.make_dz = q.grad && (q.dx || q.dw) && (f32 || q.slope || !(q.align_flags & 4));
        const long long size = f32 ? 4 : 2;  // bytes of an element, all parts together
        if (w.copy_x) w.x_off = take(size * q.M * w.ldk);
        if (w.copy_w) w.w_off = take(size * q.N * w.ldk);
        if (w.make_dz && (!f32 || q.dx)) w.dz_off = take(size * q.M * w.ldn);
        if (q.db) w.db_off = take(4LL * w.strips * q.N);
        if (f32) {
            w.xs_off = take(4LL * (q.grad ? q.K : q.M));
            w.ws_off = take(4LL * q.N);
            if (q.grad && q.dx) w.dzs_off = take(4LL * q.M);
            if (q.grad && q.dw) {
                w.dzc_off = take(size * q.M * w.ldn);
                w.dzcs_off = take(4LL * q.N);
                w.most_off = take(4LL * w.strips * q.N);
                w.mostx_off = take(4LL * w.strips * q.K);
            }
        }
        launches = w.copy_x + w.copy_w;
        if (!q.grad) {
            w.y = shape_of(q.M, q.N, q.K, q, pairs);
            w.pub.ctas = w.y.ctas;
            ++launches;
        } else {
            launches += f32 ? (q.db || q.dw) + (q.db || q.dw) + 2 * q.dw + w.make_dz : (w.make_dz || q.db) + q.db;
            if (q.dx) w.dx = shape_of(q.M, q.K, q.N, q, pairs);
            if (q.dw) w.dw = shape_of(q.N, q.K, q.M, q, pairs);
            // whole tiles of both in one launch, on one form
            w.together = q.dx && q.dw && w.dx.splits == 0 && w.dw.splits == 0;
            if (w.together) {
                const int ctas = pairs > 0 && (w.dx.ctas == 2 || w.dw.ctas == 2) ? 2 : 1;
                w.dx.ctas = w.dw.ctas = ctas;
            }
            w.pub.ctas = std::max(q.dx ? w.dx.ctas : 1, q.dw ? w.dw.ctas : 1);
            launches += q.dx + q.dw - w.together;
        }
    }
    w.workers = pairs;
    w.pub.few = w.few;
    w.pub.ctas = std::max(w.pub.ctas, 1);
    w.pub.splits[0] = std::max(1, q.grad ? w.dx.splits : w.y.splits);
    w.pub.splits[1] = std::max(1, w.dw.splits);
    w.pub.launches = launches;
    w.pub.workspace_bytes = at;
    return w;
}

}  // namespace sgemm_impl

extern "C" int sgemm_linear_plan(int M, int N, int K, int dtype, int grad, int align_flags, int num_sms, int math_mode,
                                 sgemm_linear_plan_t *out)
{
    using namespace sgemm_impl;
    if (out == nullptr || (grad != 0 && grad != 1)) return SGEMM_ERR_INVALID_VALUE;
    if (math_mode != SGEMM_MATH_FP32 && math_mode != SGEMM_MATH_TF32) return SGEMM_ERR_INVALID_VALUE;
    const bool g = grad != 0;
    const LinearProblem q{M, N, K, dtype, g, g, g, g, g, align_flags, num_sms, 0, nullptr};
    const int rc = validate_linear(q);
    if (rc != SGEMM_OK) return rc;
    // (a call for some of the gradients takes some of the parts; none of them depends on the pairs or the clusters)
    *out = linear_layout(q).pub;
    return SGEMM_OK;
}
