// Row kernels of the vocabulary losses: the teacher's entries made into sorted
// target tables, the losses put together from the tiles' partial softmax
// statistics, and the end of the sum of dH. All of them are bound by a few
// megabytes of traffic beside the products. What the call's previous kernel wrote is read
// with plain loads: these kernels may be resident before it has ended, and the read-only
// path is for memory that nobody writes meanwhile.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "device_ptx.cuh"
#include "sgemm_internal.h"
#include "vocab_internal.h"

namespace sgemm_impl {
namespace {

using namespace sgemm_dev;

constexpr float kInf = __builtin_huge_valf();

// One block per token. q = softmax over the entries that count of logit * scale (of
// the differences from the largest: a logit of the type's largest or lowest value
// times a scale above 1 would leave FP32),
// then the entries in ascending order of id: an entry's place is the number of
// entries before it (n <= 1024, so n^2 comparisons in shared memory are less work
// than the passes of a sort), equal ids staying in the given order. What is left
// out sorts to the end as kNoTarget with q = 0. (4096 x 64 entries: 9 us.)
template <int THREADS>
__global__ void __launch_bounds__(THREADS)
vocab_targets_kernel(int V, int n, const long long *__restrict__ ids, const float *__restrict__ logits, long long ldn,
                     float scale, int *__restrict__ tid, float *__restrict__ tq, float *__restrict__ tlogq)
{
    __shared__ int s_id[SGEMM_DISTILL_MAX_ENTRIES];
    __shared__ float s_x[SGEMM_DISTILL_MAX_ENTRIES];
    __shared__ float s_red[2][THREADS / 32];
    pdl_wait();
    pdl_trigger();
    const long long row = blockIdx.x;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float best = -kInf;
    for (int j = threadIdx.x; j < n; j += THREADS) {
        const long long id = ids[row * ldn + j];
        const bool counts = id >= 0 && id < V;
        const float x = counts ? logits[row * ldn + j] : -kInf;
        s_id[j] = counts && x > -kInf ? static_cast<int>(id) : kNoTarget;
        if (x != x) s_id[j] = static_cast<int>(id);  // a NaN logit stays and makes the token's loss NaN
        s_x[j] = x;
        best = x != x ? x : fmaxf(best, x);
    }
    for (int o = 16; o > 0; o >>= 1) best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, o));
    if (lane == 0) s_red[0][warp] = best;
    __syncthreads();
    best = s_red[0][0];
    for (int w = 1; w < THREADS / 32; ++w) best = fmaxf(best, s_red[0][w]);
    float sum = 0.0f;
    for (int j = threadIdx.x; j < n; j += THREADS)
        if (s_id[j] != kNoTarget) sum += expf((s_x[j] - best) * scale);
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) s_red[1][warp] = sum;
    __syncthreads();
    sum = 0.0f;
    for (int w = 0; w < THREADS / 32; ++w) sum += s_red[1][w];
    const float logsum = logf(sum);
    for (int j = threadIdx.x; j < n; j += THREADS) {
        const int id = s_id[j];
        int at = 0;
        for (int i = 0; i < n; ++i) at += s_id[i] < id || (s_id[i] == id && i < j);
        const bool counts = id != kNoTarget;
        const float t = (s_x[j] - best) * scale;
        tid[row * n + at] = id;
        tq[row * n + at] = counts ? expf(t) / sum : 0.0f;
        tlogq[row * n + at] = counts ? t - logsum : 0.0f;
    }
}

// ROWS tokens per block, kCombineThreads / ROWS lanes for each: lane l folds the
// (max, sum) pairs of columns l, l + lanes, ... (8 tokens' pairs are 64 contiguous
// bytes), then a warp per token folds the lanes'; a fixed order, so the result does
// not depend on scheduling. Latency decides: few tokens get fewer rows per block
// and so more lanes each (60 tokens of 1024 pairs: 5 us, 15.7 with 32 lanes; 8192
// tokens of 1024 pairs 25 us).
constexpr int kCombineThreads = 512;

__device__ __forceinline__ void fold(float &m, float &s, float m2, float s2)
{
    const float top = fmaxf(m, m2);
    if (top == -kInf) {  // nothing but -infinity so far (both sums 0), or NaN, which fmaxf leaves out of m but s holds
        s += s2;
        return;
    }
    s = s * exp2f(m - top) + s2 * exp2f(m2 - top);
    m = top;
}

template <int ROWS>
__global__ void __launch_bounds__(kCombineThreads)
vocab_combine_kernel(int T, int V, VocabTargets t, const float2 *part, int parts, const float *zt, float mult, float *loss,
                     float *lse)
{
    constexpr int LANES = kCombineThreads / ROWS;
    __shared__ float sm[LANES][ROWS + 1], ss[LANES][ROWS + 1];
    const int r = threadIdx.x % ROWS, l = threadIdx.x / ROWS;
    const long long first = static_cast<long long>(blockIdx.x) * ROWS;
    float m = -kInf, s = 0.0f;
    pdl_wait();
    if (first + r < T) {
        const float2 *row = part + first + r;
#pragma unroll 4
        for (int c = l; c < parts; c += LANES) {
            const float2 x = row[static_cast<long long>(c) * T];
            fold(m, s, x.x, x.y);
        }
    }
    sm[l][r] = m;
    ss[l][r] = s;
    __syncthreads();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp >= ROWS) return;  // a warp per token from here on
    const long long row = first + warp;
    if (row >= T) return;
    m = -kInf;
    s = 0.0f;
    for (int i = lane; i < LANES; i += 32) fold(m, s, sm[i][warp], ss[i][warp]);
    for (int o = 16; o > 0; o >>= 1) {
        const float m2 = __shfl_xor_sync(0xffffffffu, m, o), s2 = __shfl_xor_sync(0xffffffffu, s, o);
        const bool low = (lane & o) == 0;  // both lanes fold in the same order
        float am = low ? m : m2, as = low ? s : s2;
        fold(am, as, low ? m2 : m, low ? s2 : s);
        m = am;
        s = as;
    }
    const float total = (m + log2f(s)) * 0.6931471805599453f;  // m counts powers of two
    float sum = 0.0f;
    if (t.labels != nullptr) {
        const long long y = t.labels[row];
        if (lane == 0 && y >= 0 && y < V) sum = total - zt[row];
    } else {
        for (int j = lane; j < t.n; j += 32) {
            const float q = t.q[row * t.n + j];
            if (t.id[row * t.n + j] != kNoTarget && q != 0.0f)  // q of 0: the limit of q log q
                sum += q * (t.logq[row * t.n + j] + (total - zt[row * t.n + j]));
        }
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    if (lane == 0) {
        lse[row] = total;
        loss[row] = mult * sum;
    }
}

// The partial sums of four neighbouring dH elements in split order, then beta * dst, rounded once. One
// block per row and 1024 columns; bound by the sums' bytes (4096 x 4096, one split: 26 us; ldacc is a multiple of 4).
template <typename E>
__global__ void __launch_bounds__(256)
vocab_finish_kernel(int cols, const float *acc, long long ldacc, long long split, int splits, float beta,
                    E *__restrict__ dst, long long ldd)
{
    const long long r = blockIdx.x;
    const int c = (blockIdx.y * 256 + threadIdx.x) * 4;
    if (c >= cols) return;
    pdl_wait();
    float x[4] = {};
    const float *a = acc + r * ldacc + c;
#pragma unroll 4
    for (int s = 0; s < splits; ++s) {
        const float4 y = *reinterpret_cast<const float4 *>(a + s * split);
        x[0] += y.x;
        x[1] += y.y;
        x[2] += y.z;
        x[3] += y.w;
    }
    E *d = dst + r * ldd + c;
    for (int e = 0; e < 4 && c + e < cols; ++e) {
        if (beta != 0.0f) x[e] = fmaf(beta, static_cast<float>(d[e]), x[e]);
        d[e] = static_cast<E>(x[e]);
    }
}

}  // namespace

cudaError_t launch_vocab_targets(int T, int V, int n, const long long *ids, const float *logits, long long ldn,
                                 float scale, int *tid, float *tq, float *tlogq, bool dependent,
                                 cudaStream_t stream)
{
    return launch_kernel(dependent, vocab_targets_kernel<128>, dim3(T), dim3(128), 0, stream, V, n, ids, logits, ldn, scale,
                         tid, tq, tlogq);
}

cudaError_t launch_vocab_combine(int T, int V, const VocabTargets &t, const float2 *part, int parts, const float *zt,
                                 float mult, float *loss, float *lse, cudaStream_t stream)
{
    // eight rows per block read whole sectors; below a block of them per SM more lanes per row are worth more
    if (T > 1024)
        return launch_kernel(true, vocab_combine_kernel<8>, dim3((T + 7) / 8), dim3(kCombineThreads), 0, stream, T, V, t,
                             part, parts, zt, mult, loss, lse);
    return launch_kernel(true, vocab_combine_kernel<2>, dim3((T + 1) / 2), dim3(kCombineThreads), 0, stream, T, V, t, part,
                         parts, zt, mult, loss, lse);
}

cudaError_t launch_vocab_finish(int rows, int cols, const float *acc, long long ldacc, long long split, int splits,
                                float beta, void *dst, long long ldd, int dtype, bool dependent, cudaStream_t stream)
{
    const dim3 grid(rows, (cols + 1023) / 1024);
    if (dtype == SGEMM_DTYPE_BF16)
        return launch_kernel(dependent, vocab_finish_kernel<__nv_bfloat16>, grid, dim3(256), 0, stream, cols, acc, ldacc,
                             split, splits, beta, static_cast<__nv_bfloat16 *>(dst), ldd);
    return launch_kernel(dependent, vocab_finish_kernel<float>, grid, dim3(256), 0, stream, cols, acc, ldacc, split, splits,
                         beta, static_cast<float *>(dst), ldd);
}

}  // namespace sgemm_impl
