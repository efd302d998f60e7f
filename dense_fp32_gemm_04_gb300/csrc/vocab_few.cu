// Losses of a few FP32 tokens (scoring calls). The head's bytes are the cost: the
// tensor-core path would first write W as bfloat16 parts and read those, 4 times
// its size in all, so here every row of W is read once and multiplied as it is.
//
// A warp takes a contiguous range of the vocabulary, R rows at a time, its lanes
// side by side along D, and up to TG tokens at once: R * TG FP32 sums per lane from
// R + TG loads of 16 bytes (H comes from the L1). The lanes' sums meet in a
// reduce-scatter over shuffles, and lane t carries token t's running maximum and
// sum of exponentials through the range. More than TG tokens are done in groups,
// each reading the range again (from the L2).
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

__device__ __forceinline__ float4 load_once(const float *p)
{
    float4 v;
    asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "l"(p));
    return v;
}

// Four elements of a row for this lane: 16 bytes of 512 where rows are 16-byte aligned, else one of each 128 bytes.
template <bool VEC, bool ONCE>
__device__ __forceinline__ float4 load_four(const float *row, int d, int lane)
{
    if constexpr (VEC) {
        if constexpr (ONCE) return load_once(row + d + 4 * lane);
        return __ldg(reinterpret_cast<const float4 *>(row + d + 4 * lane));
    }
    const float *p = row + d + lane;
    return make_float4(__ldg(p), __ldg(p + 32), __ldg(p + 64), __ldg(p + 96));
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

template <int TG, bool VEC>
__global__ void __launch_bounds__(WARPS * 32, TG > 4 ? 1 : 2) vocab_few_kernel(const VocabFewParams p)
{
    constexpr int N = R * TG, PER = N >= 32 ? N / 32 : 1;
    __shared__ float sums[WARPS][N];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int gw = blockIdx.x * WARPS + warp;
    const int va = static_cast<int>(min(static_cast<long long>(gw) * p.rows, static_cast<long long>(p.V)));
    const int vb = static_cast<int>(min(va + static_cast<long long>(p.rows), static_cast<long long>(p.V)));
    const int whole = p.D / 128 * 128;
    pdl_wait();
    pdl_trigger();
    for (int t0 = 0; t0 < p.T; t0 += TG) {
        const float *h[TG];
#pragma unroll
        for (int t = 0; t < TG; ++t) h[t] = p.H + min(t0 + t, p.T - 1) * p.ldh;  // past the end: computed, not kept
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
            const float *w[R];
#pragma unroll
            for (int r = 0; r < R; ++r) w[r] = p.W + min(v + r, vb - 1) * p.ldw;
            float acc[N] = {};
#pragma unroll 2
            for (int d = 0; d < whole; d += 128) {
                float4 a[R];
#pragma unroll
                for (int r = 0; r < R; ++r) a[r] = load_four<VEC, true>(w[r], d, lane);
#pragma unroll
                for (int t = 0; t < TG; ++t) {
                    const float4 b = load_four<VEC, false>(h[t], d, lane);
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        float &x = acc[t * R + r];
                        x = fmaf(a[r].x, b.x, x);
                        x = fmaf(a[r].y, b.y, x);
                        x = fmaf(a[r].z, b.z, x);
                        x = fmaf(a[r].w, b.w, x);
                    }
                }
            }
            for (int d = whole + lane; d < p.D; d += 32)
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float a = __ldg(w[r] + d);
#pragma unroll
                    for (int t = 0; t < TG; ++t) acc[t * R + r] = fmaf(a, __ldg(h[t] + d), acc[t * R + r]);
                }
            reduce_scatter<N>(acc, lane);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < PER; ++i) sums[warp][lane * N / 32 + i] = acc[i];
            __syncwarp();
            if (!mine) continue;
            // as powers of two, the rounded maximum M being what is kept: exp(z - m) = 2^(k sum - M)
            float z[R], best = -kInf;
            const int rows = min(R, vb - v);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                z[r] = r < rows ? sums[warp][lane * R + r] : -kInf;
                best = fmaxf(best, z[r]);
            }
            const float k = p.scale * 1.4426950408889634f, top = fmaxf(m, k * best);
            const float base = top == -kInf ? 0.0f : top;
            s *= exp2f(m - base);
#pragma unroll
            for (int r = 0; r < R; ++r) s += exp2f(fmaf(z[r], k, -base));
            m = top;
            if (p.t.labels != nullptr) {
                const long long y = p.t.labels[token];
                if (y >= v && y < v + rows) p.zt[token] = p.scale * sums[warp][lane * R + static_cast<int>(y - v)];
            } else {
                const long long list = static_cast<long long>(token) * p.t.n;
                for (; entry < p.t.n; ++entry) {
                    const int y = p.t.id[list + entry];
                    if (y >= v + rows) break;  // kNoTarget ends the list too
                    p.zt[list + entry] = p.scale * sums[warp][lane * R + y - v];
                }
            }
        }
        if (mine) p.part[static_cast<long long>(gw) * p.T + token] = make_float2(m, s);
    }
}

int warps_per_sm(int T) { return WARPS * (T > 4 ? 1 : 2); }

template <int TG>
cudaError_t launch(const VocabFewParams &p, bool vec, int blocks, bool dependent, cudaStream_t stream)
{
    return launch_kernel(dependent, vec ? vocab_few_kernel<TG, true> : vocab_few_kernel<TG, false>, dim3(blocks),
                         dim3(WARPS * 32), 0, stream, p);
}

}  // namespace

int vocab_few_warps(int T, int num_sms) { return warps_per_sm(T) * num_sms; }

cudaError_t launch_vocab_few(VocabFewParams p, bool vec, int num_sms, bool dependent, cudaStream_t stream)
{
    const int warps = vocab_few_warps(p.T, num_sms);
    p.rows = (p.V + warps - 1) / warps;
    const int blocks = warps / WARPS;
    if (p.T > 8) return launch<16>(p, vec, blocks, dependent, stream);
    if (p.T > 4) return launch<8>(p, vec, blocks, dependent, stream);
    if (p.T > 2) return launch<4>(p, vec, blocks, dependent, stream);
    return launch<2>(p, vec, blocks, dependent, stream);
}

}  // namespace sgemm_impl
