// Losses of a few tokens (scoring calls). The head's bytes are the cost. For FP32
// the tensor-core path would first write W as 16-bit parts and read those, 3.5
// times its size in all; for bfloat16 its tiles of 128 tokens x 256 entries leave
// SMs idle or uneven in a single wave. Here every row of W is read once, as it
// is, by warps with equal shares of the vocabulary.
//
// A warp takes a contiguous range of the vocabulary, R rows at a time, its lanes
// side by side along D, and up to TG tokens at once: R * TG FP32 sums per lane from
// R + TG loads of 16 bytes (H comes from the L1). The lanes' sums meet in a
// reduce-scatter over shuffles, and lane t carries token t's running maximum and
// sum of exponentials through the range. More than TG tokens are done in groups,
// each reading the range again.
//
// Bound by W's bytes up to 4 tokens (1 token x 131072 x 4096: bfloat16 158 us the
// call, FP32 301 us the kernel, 7.1 TB/s; FP32, 50021 x 2048, 4 tokens 62 us, 6.6
// TB/s), then by the latency of the loads at the 8 warps per
// SM that R * TG sums leave room for (8 tokens 76 us, 16 tokens 147). The FP32 form for 4
// tokens spills 120 bytes a thread at the 128 registers of two blocks per SM. Sums of 16
// tokens, R of 4, packed FP32 and H in shared memory measured the same or slower.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "device_ptx.cuh"
#include "sgemm_internal.h"
#include "vocab_internal.h"

namespace sgemm_impl {
namespace {

using namespace sgemm_dev;

constexpr int WARPS = 8;
constexpr int R = 8;
constexpr float kInf = __builtin_huge_valf();

// Elements of a row per lane and step: 16 bytes where rows are 16-byte aligned, else 4, one of every 32 elements.
template <typename E, bool VEC>
constexpr int kPerLane = VEC ? 16 / static_cast<int>(sizeof(E)) : 4;

template <typename E, bool VEC, bool ONCE>
__device__ __forceinline__ void load_part(const E *row, int d, int lane, float (&x)[kPerLane<E, VEC>])
{
    if constexpr (VEC) {
        uint4 v;
        const E *at = row + d + lane * kPerLane<E, VEC>;
        if constexpr (ONCE)
            asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                         : "l"(at));
        else
            v = __ldg(reinterpret_cast<const uint4 *>(at));
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(E) == 4) {
                x[i] = __uint_as_float(u[i]);
            } else {  // a bfloat16 is the upper half of its FP32
                x[2 * i] = __uint_as_float(u[i] << 16);
                x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = static_cast<float>(__ldg(row + d + lane + 32 * i));
    }
}

// v[0..N) summed over the warp: afterwards v[0..max(1, N / 32)) of a lane are the sums from
// index lane * N / 32 on (N < 32: lane l has index l * N / 32, as its neighbours have).
template <int N>
__device__ __forceinline__ void reduce_scatter(float (&v)[N], int lane)
{
    int n = N;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        if (n > 1) {
            n >>= 1;
            const bool up = lane & off;
#pragma unroll
            for (int i = 0; i < N / 2; ++i)
                if (i < n) {
                    const float give = up ? v[i] : v[i + n], keep = up ? v[i + n] : v[i];
                    v[i] = keep + __shfl_xor_sync(0xffffffffu, give, off);
                }
        } else {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], off);
        }
    }
}

template <typename E, int TG, bool VEC>
__global__ void __launch_bounds__(WARPS * 32, TG > 4 ? 1 : 2) vocab_few_kernel(const VocabFewParams p)
{
    constexpr int PART = kPerLane<E, VEC>, STEP = 32 * PART;
    const E *H = static_cast<const E *>(p.H), *W = static_cast<const E *>(p.W);
    constexpr int N = R * TG, PER = N >= 32 ? N / 32 : 1;
    __shared__ float sums[WARPS][N];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int gw = blockIdx.x * WARPS + warp;
    const int va = static_cast<int>(min(static_cast<long long>(gw) * p.rows, static_cast<long long>(p.V)));
    const int vb = static_cast<int>(min(va + static_cast<long long>(p.rows), static_cast<long long>(p.V)));
    const int whole = p.D / STEP * STEP;
    pdl_wait();
    pdl_trigger();
    for (int t0 = 0; t0 < p.T; t0 += TG) {
        const E *h[TG];
#pragma unroll
        for (int t = 0; t < TG; ++t) h[t] = H + min(t0 + t, p.T - 1) * p.ldh;  // past the end: computed, not kept
        const int token = t0 + lane;
        const bool mine = lane < TG && token < p.T;
        float m = -kInf, s = 0.0f;
        int entry = 0;  // distillation: the token's first target from the current rows on
        if (mine && p.t.labels == nullptr) {
            int hi = p.t.n;
            while (entry < hi) {
                const int mid = (entry + hi) >> 1;
                if (p.t.id[static_cast<long long>(token) * p.t.n + mid] < va)
                    entry = mid + 1;
                else
                    hi = mid;
            }
        }
        for (int v = va; v < vb; v += R) {
            const int rows = min(R, vb - v);
            const E *w[R];  // past the end the last row again: computed, not kept
#pragma unroll
            for (int r = 0; r < R; ++r) w[r] = W + min(v + r, vb - 1) * p.ldw;
            float acc[N] = {};
#pragma unroll 2
            for (int d = 0; d < whole; d += STEP) {
                float a[R][PART];
#pragma unroll
                for (int r = 0; r < R; ++r) load_part<E, VEC, true>(w[r], d, lane, a[r]);
#pragma unroll
                for (int t = 0; t < TG; ++t) {
                    float b[PART];
                    load_part<E, VEC, false>(h[t], d, lane, b);
#pragma unroll
                    for (int r = 0; r < R; ++r)
#pragma unroll
                        for (int i = 0; i < PART; ++i) acc[t * R + r] = fmaf(a[r][i], b[i], acc[t * R + r]);
                }
            }
            for (int d = whole + lane; d < p.D; d += 32)
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float a = static_cast<float>(__ldg(w[r] + d));
#pragma unroll
                    for (int t = 0; t < TG; ++t) acc[t * R + r] = fmaf(a, static_cast<float>(__ldg(h[t] + d)), acc[t * R + r]);
                }
            reduce_scatter<N>(acc, lane);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < PER; ++i) sums[warp][lane * N / 32 + i] = acc[i];
            __syncwarp();
            if (!mine) continue;
            // as powers of two, the rounded maximum M being what is kept: exp(z - m) = 2^(k sum - M)
            float z[R], best = -kInf;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                z[r] = r < rows ? sums[warp][lane * R + r] : -kInf;
                best = fmaxf(best, z[r]);
            }
            const float k = p.scale * 1.4426950408889634f, top = fmaxf(m, k * best);
            const float base = top == -kInf ? 0.0f : top;
            s *= exp2f(m - base);
#pragma unroll
            for (int r = 0; r < R; ++r)  // (M so large that its rounding would show: the products rounded as it was)
                s += exp2f(fabsf(base) < kHugeLog2 ? fmaf(z[r], k, -base) : __fmul_rn(k, z[r]) - base);
            m = top;
            if (p.t.labels != nullptr) {
                const long long y = p.t.labels[token];
                if (y >= v && y < v + rows && index_ok(token < p.targets, p.status, kWhereIdxVocabTarget))
                    p.zt[token] = p.scale * sums[warp][lane * R + static_cast<int>(y - v)];
            } else {
                const long long list = static_cast<long long>(token) * p.t.n;
                for (; entry < p.t.n; ++entry) {
                    const int y = p.t.id[list + entry];
                    if (y >= v + rows) break;  // kNoTarget ends the list too
                    if (index_ok(y >= v && list + entry < p.targets, p.status, kWhereIdxVocabTarget))
                        p.zt[list + entry] = p.scale * sums[warp][lane * R + y - v];
                }
            }
        }
        if (mine && index_ok(gw < p.stat_rows, p.status, kWhereIdxVocabStat))
            p.part[static_cast<long long>(gw) * p.T + token] = make_float2(m, s);
    }
}

// The products at the targets alone, a warp for each, for the gradients of tokens whose loss came from the kernel above:
// the same sums in the same order (reduce_scatter adds what a butterfly adds), so the label's entry p - 1 of dZ is made of
// the very logit in lse, where the tensor cores' truncated one would be off by up to 2^-18 of itself (1 token, 32768 x 2048:
// 5 us of the call's 90).
template <typename E, bool VEC>
__global__ void __launch_bounds__(WARPS * 32) vocab_few_targets_kernel(const VocabFewParams p)
{
    constexpr int PART = kPerLane<E, VEC>, STEP = 32 * PART;
    const int lane = threadIdx.x & 31, pair = blockIdx.x * WARPS + (threadIdx.x >> 5);
    pdl_wait();
    pdl_trigger();
    if (pair >= p.T * p.t.n) return;
    const int token = pair / p.t.n;
    const long long y = p.t.labels != nullptr ? p.t.labels[token] : p.t.id[pair];
    if (y < 0 || y >= p.V) return;  // (kNoTarget too)
    const E *h = static_cast<const E *>(p.H) + token * p.ldh, *w = static_cast<const E *>(p.W) + y * p.ldw;
    const int whole = p.D / STEP * STEP;
    float acc = 0.0f;
#pragma unroll 4
    for (int d = 0; d < whole; d += STEP) {
        float a[PART], b[PART];
        load_part<E, VEC, false>(w, d, lane, a);
        load_part<E, VEC, false>(h, d, lane, b);
#pragma unroll
        for (int i = 0; i < PART; ++i) acc = fmaf(a[i], b[i], acc);
    }
    for (int d = whole + lane; d < p.D; d += 32)
        acc = fmaf(static_cast<float>(__ldg(w + d)), static_cast<float>(__ldg(h + d)), acc);
    for (int off = 16; off > 0; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
    if (lane == 0 && index_ok(pair < p.targets, p.status, kWhereIdxVocabTarget)) p.zt[pair] = acc;
}

int warps_per_sm(int T) { return WARPS * (T > 4 ? 1 : 2); }

template <typename E, int TG, bool VEC>
cudaError_t launch(const VocabFewParams &p, int blocks, bool dependent, cudaStream_t stream)
{
    return launch_kernel(dependent, vocab_few_kernel<E, TG, VEC>, dim3(blocks), dim3(WARPS * 32), 0, stream, p);
}

// MOST: tokens that a call of this type and alignment can have here (vocab_plan.cpp).
template <typename E, bool VEC, int MOST>
cudaError_t launch_tokens(const VocabFewParams &p, int blocks, bool dependent, cudaStream_t stream)
{
    if (p.T > MOST) return cudaErrorInvalidValue;
    if constexpr (MOST > 4)
        if (p.T > 4) return launch<E, 8, VEC>(p, blocks, dependent, stream);
    if constexpr (MOST > 2)
        if (p.T > 2) return launch<E, 4, VEC>(p, blocks, dependent, stream);
    if (p.T > 1) return launch<E, 2, VEC>(p, blocks, dependent, stream);
    return launch<E, 1, VEC>(p, blocks, dependent, stream);
}

}  // namespace

int vocab_few_warps(int T, int num_sms) { return warps_per_sm(T) * num_sms; }

cudaError_t launch_vocab_few(VocabFewParams p, int dtype, bool vec, int num_sms, bool dependent, cudaStream_t stream)
{
    const int warps = vocab_few_warps(p.T, num_sms);
    p.rows = (p.V + warps - 1) / warps;
    const int blocks = warps / WARPS;
    if (dtype == SGEMM_DTYPE_BF16)
        return vec ? launch_tokens<__nv_bfloat16, true, kFewTokensBf16>(p, blocks, dependent, stream)
                   : launch_tokens<__nv_bfloat16, false, kFewTokensCopied>(p, blocks, dependent, stream);
    return vec ? launch_tokens<float, true, kFewTokensF32>(p, blocks, dependent, stream)
               : launch_tokens<float, false, kFewTokensF32>(p, blocks, dependent, stream);
}

cudaError_t launch_vocab_few_targets(const VocabFewParams &p, int dtype, bool vec, bool dependent, cudaStream_t stream)
{
    const dim3 blocks((p.T * p.t.n + WARPS - 1) / WARPS);
    if (dtype == SGEMM_DTYPE_BF16)
        return launch_kernel(dependent, vec ? vocab_few_targets_kernel<__nv_bfloat16, true>
                                            : vocab_few_targets_kernel<__nv_bfloat16, false>,
                             blocks, dim3(WARPS * 32), 0, stream, p);
    return launch_kernel(dependent, vec ? vocab_few_targets_kernel<float, true> : vocab_few_targets_kernel<float, false>,
                         blocks, dim3(WARPS * 32), 0, stream, p);
}

}  // namespace sgemm_impl
