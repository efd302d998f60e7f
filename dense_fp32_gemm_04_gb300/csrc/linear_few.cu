// Linear layers of a few tokens, without tensor cores: W is read once as it is, 16
// bytes a lane, and multiplied in FP32. A warp takes ROWS output features (or a part
// of their K range: KS warps of a block share the features where there are too few of
// them to fill the machine), so the tokens' elements, which come from the first-level
// cache, are used ROWS times.
//
// Bound by W's bytes for one or two tokens (8192 x 2048 in bfloat16, W from memory: 7.7 us, 4.4 TB/s with the launch, 5.1 where
// the L2 holds it), by the multiplications from some 8 on. Against the tensor cores, which take as long for 1 token as for 100,
// in us, here / there, W from memory:
//   bfloat16  8192 x 2048    1 token 7.7 / 15.2   4 tokens 10.4 / 13.8   5 tokens 14.3 / 13.9
//             2048 x 8192    1 token 9.0 / 17.1   4 tokens 10.4 / 15.6   5 tokens 14.3 / 14.8
//             16384 x 4096   1 token 23.0 / 36.7  4 tokens 31.9 / 34.5   5 tokens 41.4 / 33.4
//   FP32      4096 x 4096    1 token 13.4 / 55.0  16 tokens 47.1 / 44.0 (36.5 / 44.0 with W in the L2)  24 tokens 71.4 / 44.0
//             1000 x 1000    1 token 4.9 / 14.4   16 tokens 8.1 / 14.6   32 tokens 12.7 / 14.7
// so up to 4 tokens in bfloat16 and 16 in FP32, and up to 32 where W is small: there (FP32 operands become parts first) the tile
// kernel takes 13 us and 2 us per million elements of W, these warps 3 us and M / 8 per million.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "device_ptx.cuh"
#include "linear_act.cuh"
#include "linear_internal.h"

namespace sgemm_impl {
namespace {

using namespace sgemm_dev;

constexpr int WARPS = 4;

template <typename E>
struct Wide;
template <>
struct Wide<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void open(const uint4 &v, float (&x)[4])
    {
        x[0] = __uint_as_float(v.x);
        x[1] = __uint_as_float(v.y);
        x[2] = __uint_as_float(v.z);
        x[3] = __uint_as_float(v.w);
    }
};
template <>
struct Wide<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void open(const uint4 &v, float (&x)[8])
    {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
};

__device__ __forceinline__ void put_slope(float *p, float s) { *p = s; }
__device__ __forceinline__ void put_slope(short *p, float s) { *p = slope_close(s); }

template <typename E, int TOKENS, int ROWS, int UNROLL, int BLOCKS, bool VEC>
__global__ void __launch_bounds__(32 * WARPS, BLOCKS)
linear_few_kernel(const LinearFewParams p, int ks, int tg)
{
    constexpr int N = VEC ? Wide<E>::N : 1;
    constexpr bool F32 = sizeof(E) == 4;
    __shared__ float part[WARPS][ROWS * TOKENS];
    const int lane = threadIdx.x, warp = threadIdx.y;
    // warps that share features: tg of them for other tokens (W comes from the cache for all but one), ks for parts of K
    const int share = warp % ks, sharing = ks * tg;
    const long long n0 = (static_cast<long long>(blockIdx.x) * (WARPS / sharing) + warp / sharing) * ROWS;
    const int m0 = (blockIdx.y * tg + warp / ks % tg) * TOKENS;
    // this warp's part of K, in steps of the whole warp's accesses
    const int step = 32 * N, steps = (p.K + step - 1) / step;
    const int s0 = static_cast<int>(static_cast<long long>(steps) * share / ks);
    const int s1 = static_cast<int>(static_cast<long long>(steps) * (share + 1) / ks);
    const E *w[ROWS], *x[TOKENS];  // rows past the end: the last one, whose result is not used
#pragma unroll
    for (int r = 0; r < ROWS; ++r) w[r] = static_cast<const E *>(p.W) + min(n0 + r, static_cast<long long>(p.N) - 1) * p.ldw;
#pragma unroll
    for (int m = 0; m < TOKENS; ++m) x[m] = static_cast<const E *>(p.X) + min(m0 + m, p.M - 1) * p.ldx;
    float acc[ROWS][TOKENS] = {};
    typedef typename std::conditional<VEC, uint4, E>::type Raw;  // 16 bytes of a row, or one element
    auto load = [](const E *q) {
        if constexpr (VEC)
            return __ldg(reinterpret_cast<const uint4 *>(q));
        else
            return __ldg(q);
    };
    auto open = [](const Raw &v, float (&x)[N]) {
        if constexpr (VEC)
            Wide<E>::open(v, x);
        else
            x[0] = static_cast<float>(v);
    };
    auto multiply = [&](const Raw (&v)[ROWS], int k) {
        float a[ROWS][N], b[N];
#pragma unroll
        for (int r = 0; r < ROWS; ++r) open(v[r], a[r]);
#pragma unroll
        for (int m = 0; m < TOKENS; ++m) {
            open(load(x[m] + k), b);
#pragma unroll
            for (int r = 0; r < ROWS; ++r)
#pragma unroll
                for (int i = 0; i < N; ++i) acc[r][m] = fmaf(a[r][i], b[i], acc[r][m]);
        }
    };
    const int whole = min(s1, p.K / step);  // steps without an end in them
    int s = s0;
    for (; s + UNROLL <= whole; s += UNROLL) {  // W of several steps is on its way before the first is used
        Raw v[UNROLL][ROWS];
#pragma unroll
        for (int j = 0; j < UNROLL; ++j)
#pragma unroll
            for (int r = 0; r < ROWS; ++r) v[j][r] = load(w[r] + (s + j) * step + lane * N);
#pragma unroll
        for (int j = 0; j < UNROLL; ++j) multiply(v[j], (s + j) * step + lane * N);
    }
    auto take = [&](int k) {
        Raw v[ROWS];
#pragma unroll
        for (int r = 0; r < ROWS; ++r) v[r] = load(w[r] + k);
        multiply(v, k);
    };
    for (; s < whole; ++s) take(s * step + lane * N);
    if (s < s1) {  // the last, partial one
        const int k = s * step + lane * N;
        if (k + N <= p.K) {
            take(k);
        } else if (k < p.K) {
#pragma unroll 1
            for (int i = k; i < p.K; ++i)
#pragma unroll
                for (int m = 0; m < TOKENS; ++m)
#pragma unroll
                    for (int r = 0; r < ROWS; ++r)
                        acc[r][m] = fmaf(static_cast<float>(w[r][i]), static_cast<float>(x[m][i]), acc[r][m]);
        }
    }
#pragma unroll
    for (int r = 0; r < ROWS; ++r)
#pragma unroll
        for (int m = 0; m < TOKENS; ++m) {
            float v = acc[r][m];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
            if (lane == 0) part[warp][m * ROWS + r] = v;
        }
    __syncthreads();
    if (share != 0) return;
    for (int j = lane; j < ROWS * TOKENS; j += 32) {
        const int m = m0 + j / ROWS;
        const long long n = n0 + j % ROWS;
        if (m >= p.M || n >= p.N) continue;
        float z = 0.0f;
        for (int i = 0; i < ks; ++i) z += part[warp + i][j];
        if (p.bias != nullptr) z += static_cast<float>(static_cast<const E *>(p.bias)[n]);
        float y, slope;
        activate_by<F32>(p.act, z, y, slope);
        if (p.slope != nullptr) {
            typedef typename std::conditional<F32, float, short>::type S;
            put_slope(static_cast<S *>(p.slope) + m * p.lds + n, slope);
        }
        if (p.R != nullptr) y += static_cast<float>(static_cast<const E *>(p.R)[m * p.ldr + n]);
        static_cast<E *>(p.Y)[m * p.ldy + n] = static_cast<E>(y);
    }
}

// BLOCKS: blocks that an SM holds at once. The features' K ranges are split as far as that leaves all blocks in one wave:
// a second one with a few blocks in it would double the time (4096 x 4096 in FP32, one token: 17.7 us in 1.1 waves).
template <typename E, int TOKENS, int ROWS, int UNROLL, int BLOCKS>
cudaError_t launch(const LinearFewParams &p, bool vec, int num_sms, cudaStream_t stream)
{
    const long long groups = (p.N + ROWS - 1) / ROWS;
    int tg = 1, ks = 1;
    while (tg < WARPS && tg * TOKENS < p.M) tg *= 2;
    const long long passes = (p.M + tg * TOKENS - 1) / (tg * TOKENS);
    while (ks * tg < WARPS && groups * passes * (2 * ks * tg) <= static_cast<long long>(WARPS) * BLOCKS * num_sms &&
           p.K / (32 * Wide<E>::N * 2 * ks) >= UNROLL)
        ks *= 2;
    const dim3 grid(static_cast<unsigned>((groups * ks * tg + WARPS - 1) / WARPS), static_cast<unsigned>(passes)), block(32, WARPS);
    return launch_kernel(false, vec ? linear_few_kernel<E, TOKENS, ROWS, UNROLL, BLOCKS, true>
                                    : linear_few_kernel<E, TOKENS, ROWS, UNROLL, BLOCKS, false>, grid, block, 0, stream, p, ks, tg);
}

template <typename E>
cudaError_t launch_tokens(const LinearFewParams &p, bool vec, int num_sms, cudaStream_t stream)
{
    if (p.M == 1) return launch<E, 1, 4, 2, 8>(p, vec, num_sms, stream);
    if (p.M == 2) return launch<E, 2, 4, 2, 8>(p, vec, num_sms, stream);
    if (p.M <= 4) return launch<E, 4, 4, 2, 4>(p, vec, num_sms, stream);
    return launch<E, 8, 4, 2, 4>(p, vec, num_sms, stream);
}

}  // namespace

cudaError_t launch_linear_few(const LinearFewParams &p, int dtype, bool vec, int num_sms, cudaStream_t stream)
{
    return dtype == SGEMM_DTYPE_BF16 ? launch_tokens<__nv_bfloat16>(p, vec, num_sms, stream)
                                     : launch_tokens<float>(p, vec, num_sms, stream);
}

}  // namespace sgemm_impl
