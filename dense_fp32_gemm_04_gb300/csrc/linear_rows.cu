// Row and column kernels of the linear layers: dZ = dY * slope with its columns' sums
// and largest values, the bias' gradient, and FP32 operands as two float16 parts.
// Bound by memory: every matrix is read once (a row that does not fit a block's
// registers twice) and its parts written once. From the L2, where a training step has
// them: strips of 2048 x 8192 in bfloat16 with slopes 19 us (101 MB, 5.3 TB/s), of 2047 x
// 3001 in FP32 at odd strides 12.7 us (49 MB, 3.9 TB/s), parts of 3001 x 1531 8.5 us (37 MB,
// 4.3 TB/s), of dZ by rows and by columns 25.5 us (98 MB, 3.8 TB/s).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstring>
#include <type_traits>

#include "device_ptx.cuh"
#include "linear_act.cuh"
#include "linear_internal.h"

namespace sgemm_impl {
namespace {

using namespace sgemm_dev;

constexpr float kInf = __builtin_huge_valf();

template <typename E>
struct Slope;
template <>
struct Slope<float> {
    typedef float type;
    static __device__ __forceinline__ float open(float s) { return s; }
};
template <>
struct Slope<__nv_bfloat16> {
    typedef short type;
    static __device__ __forceinline__ float open(short s) { return slope_open(s); }
};

// 4, 8 or 16 bytes as one access (an array of a class type would be copied element by element).
template <int BYTES>
struct Bits;
template <>
struct Bits<4> {
    typedef uint32_t type;
};
template <>
struct Bits<8> {
    typedef uint2 type;
};
template <>
struct Bits<16> {
    typedef uint4 type;
};

// W neighbouring elements, `n` of which exist, in one access where VEC (the rows start on boundaries of W elements).
template <int W, bool VEC, typename T>
__device__ __forceinline__ void load_some(const T *p, int n, T (&x)[W])
{
    if (VEC && n >= W) {
        const typename Bits<W * sizeof(T)>::type t = *reinterpret_cast<const typename Bits<W * sizeof(T)>::type *>(p);
        memcpy(x, &t, sizeof(t));
    } else {
#pragma unroll
        for (int i = 0; i < W; ++i) x[i] = i < n ? p[i] : T{};
    }
}

// A block: 32 W columns of a strip of kLinearStrip rows, W columns a lane (16 bytes of them where the rows allow it: 2048 x 8192
// in bfloat16 26 us with 4), 8 rows at a time. x = src (* slope); what is asked for of: x in bfloat16, the columns' sums of
// x (before it is rounded), their largest finite |x|.
template <typename E, int W, bool VEC>
__global__ void __launch_bounds__(256, 4)
linear_strips_kernel(int M, int N, const E *__restrict__ src, long long ld, const typename Slope<E>::type *__restrict__ slope,
                     long long lds, __nv_bfloat16 *__restrict__ dz, long long ldz, float *__restrict__ sums,
                     float *__restrict__ most)
{
    constexpr int WIDTH = 32 * W;
    __shared__ float part[2][8][WIDTH];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x, warp = threadIdx.y;
    const int blocks = (N + WIDTH - 1) / WIDTH, c0 = blockIdx.x % blocks * WIDTH, c = c0 + W * lane, n = N - c;
    const long long strip = blockIdx.x / blocks, r0 = strip * kLinearStrip;
    const int rows = static_cast<int>(min(static_cast<long long>(kLinearStrip), M - r0));
    float sum[W] = {}, top[W] = {};
    // WHOLE: all of the lane's columns exist (asked once: a branch at every load would keep them from being on their way together)
    auto walk = [&](auto whole) {
        constexpr bool WHOLE = decltype(whole)::value;
#pragma unroll 4
        for (int i = warp; i < rows; i += 8) {
            const long long r = r0 + i;
            E g[W];
            typename Slope<E>::type s[W];
            load_some<W, VEC && WHOLE>(src + r * ld + c, WHOLE ? W : n, g);
            if (slope != nullptr) load_some<W, VEC && WHOLE>(slope + r * lds + c, WHOLE ? W : n, s);
            float x[W];
#pragma unroll
            for (int e = 0; e < W; ++e) {
                x[e] = static_cast<float>(g[e]);
                if (slope != nullptr) x[e] = WHOLE || e < n ? x[e] * Slope<E>::open(s[e]) : 0.0f;
                sum[e] += x[e];
                if constexpr (sizeof(E) == 4) {  // (bfloat16 operands are not scaled)
                    const float a = fabsf(x[e]);
                    top[e] = a < kInf ? fmaxf(top[e], a) : top[e];
                }
            }
            if (dz != nullptr) {  // (its rows have room for whole groups)
                uint32_t y[W / 2];
#pragma unroll
                for (int e = 0; e < W; e += 2) {
                    const __nv_bfloat162 two = __floats2bfloat162_rn(x[e], x[e + 1]);
                    memcpy(&y[e / 2], &two, 4);
                }
                typename Bits<2 * W>::type all;
                memcpy(&all, y, sizeof(all));
                *reinterpret_cast<typename Bits<2 * W>::type *>(dz + r * ldz + c) = all;
            }
        }
    };
    if (n >= W)
        walk(std::true_type());
    else if (n > 0)
        walk(std::false_type());
    if (sums == nullptr && most == nullptr) return;
#pragma unroll
    for (int e = 0; e < W; ++e) {
        part[0][warp][W * lane + e] = sum[e];
        part[1][warp][W * lane + e] = top[e];
    }
    __syncthreads();
    for (int j = warp * 32 + lane; j < WIDTH && c0 + j < N; j += 256) {
        float x = 0.0f, y = 0.0f;
#pragma unroll
        for (int w = 0; w < 8; ++w) {
            x += part[0][w][j];
            y = fmaxf(y, part[1][w][j]);
        }
        if (sums != nullptr) sums[strip * N + c0 + j] = x;
        if (most != nullptr) most[strip * N + c0 + j] = y;
    }
}

// Scaling by powers of two: numbers whose largest is at least 2^e and below 2^(e + 1) take 2^s, s the even number that brings that
// into [2^14, 2^16). What is kept of it is 2^(-s / 2): a result's factors, of its row and of its column, are squares, and the
// product of their roots is within FP32's range whatever the operands, as are the sum times it and that times it again, unless
// the result itself is outside. (The factors one after the other left the range at X = 1e33 with W = 0.02.) s ends at `most`:
// 126 takes FP32's smallest number to 2^-23, which float16 holds, and keeps the product of two roots above 2^-127.
__device__ __forceinline__ float root_unscale(int e, int most = 126) { return __int_as_float((127 - min((15 - e) & ~1, most) / 2) << 23); }

// The exponent of a >= 0; of numbers below 2^-126, 0 too, -127: s is at its end there or holds them all the same.
__device__ __forceinline__ int exponent_of(float a) { return (__float_as_int(a) >> 23) - 127; }

// 1 / x for a power of two from 2^-126 to 2^126.
__device__ __forceinline__ float inverse_power(float x) { return __int_as_float((254 << 23) - __float_as_int(x)); }

// The strips' sums put together: db = sum + beta * db; and their largest values: the root of what undoes the columns' scaling. 32 columns a
// block, the strips dealt to 8 rows of threads: few columns still have many loads in flight. (Plain loads: the
// kernel before it in the call wrote them.)
template <typename E>
__global__ void __launch_bounds__(256)
linear_columns_kernel(int N, int strips, const float *sums, float beta, E *db, const float *most, float *unscale)
{
    __shared__ float part[2][8][32];
    pdl_wait();
    pdl_trigger();
    const int c = blockIdx.x * 32 + threadIdx.x;
    float x = 0.0f, y = 0.0f;
    if (c < N) {
#pragma unroll 4
        for (int s = threadIdx.y; s < strips; s += 8) {
            if (db != nullptr) x += sums[static_cast<long long>(s) * N + c];
            if (most != nullptr) y = fmaxf(y, most[static_cast<long long>(s) * N + c]);
        }
    }
    part[0][threadIdx.y][threadIdx.x] = x;
    part[1][threadIdx.y][threadIdx.x] = y;
    __syncthreads();
    if (threadIdx.y != 0 || c >= N) return;
    x = y = 0.0f;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
        x += part[0][w][threadIdx.x];
        y = fmaxf(y, part[1][w][threadIdx.x]);
    }
    if (db != nullptr) {
        if (beta != 0.0f) x = fmaf(beta, static_cast<float>(db[c]), x);
        db[c] = static_cast<E>(x);
    }
    if (most != nullptr) unscale[c] = root_unscale(exponent_of(y));
}

// Two scaled values as two float16 numbers each (22 bits). The first is finite and what is left, infinities and NaN too, is in the
// second: that only meets the other operand's first number, whose sign and zero are the operand's, so an infinity gives what the
// formula has. (In the first one it would also meet the other operand's second number, which may be 0 or of the other sign.)
__device__ __forceinline__ void two_halves(const float (&x)[2], __half *to, long long part)
{
    const __half2 most = __float2half2_rn(65504.0f);  // the largest float16
    const __half2 hi = __hmax2(__hmin2(__floats2half2_rn(x[0], x[1]), most), __hneg2(most));
    const float2 back = __half22float2(hi);
    *reinterpret_cast<__half2 *>(to) = hi;
    *reinterpret_cast<__half2 *>(to + part) = __floats2half2_rn(x[0] - back.x, x[1] - back.y);
}

// FP32 rows x = src (* slope) as float16 parts, a block per row. by_row: x times factor[column]^2 (if given), scaled for each row
// such that its largest finite value lies in [2^14, 2^16), the root of what undoes it in row_unscale; by_column: x scaled by the
// columns' own factors, whose roots linear_columns_kernel left. Rows of ldp elements on 128-byte lines, the second part `rows` of
// them further on. A thread keeps PAIRS pairs of a row in registers (of up to 16 THREADS
// columns: the whole row).
template <bool VEC, int THREADS>
__global__ void __launch_bounds__(THREADS)
linear_parts_kernel(int rows, int cols, const float *__restrict__ src, long long ld, const float *__restrict__ slope, long long lds,
                    const float *factor, __half *by_row, float *row_unscale, const float *column_unscale, __half *by_column,
                    long long ldp)
{
    constexpr int PAIRS = 8;
    __shared__ unsigned red[THREADS / 32];
    const long long r = blockIdx.x, part = rows * ldp;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const float *s = src + r * ld, *t = slope != nullptr ? slope + r * lds : nullptr;
    auto load = [&](int c, float (&x)[2]) {
        load_some<2, VEC>(s + c, cols - c, x);
        if (t != nullptr) {
            float y[2];
            load_some<2, VEC>(t + c, cols - c, y);
            x[0] *= y[0];
            x[1] = c + 1 < cols ? x[1] * y[1] : 0.0f;
        }
    };
    float x[PAIRS][2];
    pdl_wait();
    pdl_trigger();
#pragma unroll
    for (int j = 0; j < PAIRS; ++j) {
        const int c = 2 * (threadIdx.x + THREADS * j);
        x[j][0] = x[j][1] = 0.0f;
        if (c < cols) load(c, x[j]);
    }
    float up = 1.0f;
    if (by_row != nullptr) {
        // The largest of |x| factor^2 by its exponent and half of its digits, (E + 2 F) 2^22 for the exponents as they stand in x and
        // factor: as a number it may be far outside FP32's range although the results are not. (Without a factor plain numbers,
        // the same in the end: 24 tokens of 4096 x 4096 50.5 us with exponents there too, 44.5 so.)
        unsigned most = 0;
        float top = 0.0f;
        auto walk = [&](auto with_factor) {
            auto look = [&](int c, const float (&v)[2]) {
                if constexpr (decltype(with_factor)::value) {
                    const float f[2] = {factor[c], c + 1 < cols ? factor[c + 1] : 1.0f};
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const unsigned a = __float_as_uint(v[e]) & 0x7fffffffu;
                        most = max(most, a - 1u < 0x7f7fffffu ? (a >> 1) + __float_as_uint(f[e]) : 0);  // (no zeros, they weigh nothing)
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 2; ++e) top = fabsf(v[e]) < kInf ? fmaxf(top, fabsf(v[e])) : top;
                }
            };
#pragma unroll
            for (int j = 0; j < PAIRS; ++j) {
                const int c = 2 * (threadIdx.x + THREADS * j);
                if (c < cols) look(c, x[j]);
            }
            for (int c = 2 * (threadIdx.x + THREADS * PAIRS); c < cols; c += 2 * THREADS) {
                float v[2];
                load(c, v);
                look(c, v);
            }
        };
        if (factor != nullptr) {
            walk(std::true_type());
        } else {
            walk(std::false_type());
            most = (__float_as_uint(top) >> 1) + __float_as_uint(1.0f);
        }
        most = __reduce_max_sync(0xffffffffu, most);
        if (lane == 0) red[warp] = most;
        __syncthreads();
        most = red[0];
#pragma unroll
        for (int w = 1; w < THREADS / 32; ++w) most = max(most, red[w]);
        // (with a factor in them these rows' results have no other: its root may be as small as 2^-126)
        const float back = root_unscale(static_cast<int>(most >> 22) - 3 * 127, factor != nullptr ? 252 : 126);
        if (threadIdx.x == 0) row_unscale[r] = back;
        up = inverse_power(back);
    }
    auto leave = [&](int c, const float (&v)[2]) {
        const bool second = c + 1 < cols;
        if (by_row != nullptr) {
            float y[2];
            if (factor != nullptr) {
                const float f[2] = {factor[c], second ? factor[c + 1] : 1.0f};
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    // (a finite number other than 0 never meets these ends and has bits left)
                    const float g = fminf(fmaxf(f[e] * up, 1.17549435e-38f), 8.5070592e37f);
                    y[e] = v[e] * g * g;
                }
            } else {
                y[0] = v[0] * (up * up);  // (2^-112 to 2^126)
                y[1] = v[1] * (up * up);
            }
            two_halves(y, by_row + r * ldp + c, part);
        }
        if (by_column != nullptr) {
            const float f[2] = {inverse_power(column_unscale[c]), second ? inverse_power(column_unscale[c + 1]) : 1.0f};
            const float y[2] = {v[0] * f[0] * f[0], second ? v[1] * f[1] * f[1] : 0.0f};
            two_halves(y, by_column + r * ldp + c, part);
        }
    };
#pragma unroll
    for (int j = 0; j < PAIRS; ++j) {
        const int c = 2 * (threadIdx.x + THREADS * j);
        if (c < cols) leave(c, x[j]);
    }
    for (int c = 2 * (threadIdx.x + THREADS * PAIRS); c < cols; c += 2 * THREADS) {
        float v[2];
        load(c, v);
        leave(c, v);
    }
}

// Rows start on boundaries of `count` elements.
bool in_groups(const void *p, long long ld, size_t size, int count)
{
    return reinterpret_cast<uintptr_t>(p) % (count * size) == 0 && ld % count == 0;
}

template <typename E, int W, bool VEC>
cudaError_t launch_strips(int M, int N, const E *src, long long ld, const typename Slope<E>::type *slope, long long lds,
                          __nv_bfloat16 *dz, long long ldz, float *sums, float *most, bool dependent, cudaStream_t stream)
{
    const dim3 grid(static_cast<unsigned>((N + 32 * W - 1) / (32 * W)) * static_cast<unsigned>((M + kLinearStrip - 1) / kLinearStrip));
    return launch_kernel(dependent, linear_strips_kernel<E, W, VEC>, grid, dim3(32, 8), 0, stream, M, N, src, ld, slope, lds, dz, ldz,
                         sums, most);
}

template <typename E>
cudaError_t launch_strips(int M, int N, const void *src, long long ld, const void *slope, long long lds, void *dz, long long ldz,
                          float *sums, float *most, bool dependent, cudaStream_t stream)
{
    typedef typename Slope<E>::type S;
    constexpr int W = 16 / sizeof(E);
    const E *x = static_cast<const E *>(src);
    const S *s = static_cast<const S *>(slope);
    __nv_bfloat16 *z = static_cast<__nv_bfloat16 *>(dz);
    if (in_groups(src, ld, sizeof(E), W) && (slope == nullptr || in_groups(slope, lds, sizeof(S), W)))
        return launch_strips<E, W, true>(M, N, x, ld, s, lds, z, ldz, sums, most, dependent, stream);
    return launch_strips<E, 2, false>(M, N, x, ld, s, lds, z, ldz, sums, most, dependent, stream);
}

}  // namespace

cudaError_t launch_linear_strips(int M, int N, int dtype, const void *src, long long ld, const void *slope, long long lds, void *dz,
                                 long long ldz, float *sums, float *most, bool dependent, cudaStream_t stream)
{
    if (dtype == SGEMM_DTYPE_BF16)
        return launch_strips<__nv_bfloat16>(M, N, src, ld, slope, lds, dz, ldz, sums, most, dependent, stream);
    return launch_strips<float>(M, N, src, ld, slope, lds, dz, ldz, sums, most, dependent, stream);
}

cudaError_t launch_linear_columns(int N, int strips, const float *sums, float beta, void *db, int dtype, const float *most,
                                  float *unscale, bool dependent, cudaStream_t stream)
{
    const dim3 grid((N + 31) / 32), block(32, 8);
    if (dtype == SGEMM_DTYPE_BF16)
        return launch_kernel(dependent, linear_columns_kernel<__nv_bfloat16>, grid, block, 0, stream, N, strips, sums, beta,
                             static_cast<__nv_bfloat16 *>(db), most, unscale);
    return launch_kernel(dependent, linear_columns_kernel<float>, grid, block, 0, stream, N, strips, sums, beta, static_cast<float *>(db),
                         most, unscale);
}

cudaError_t launch_linear_parts(int rows, int cols, const void *src, long long ld, const void *slope, long long lds,
                                const float *factor, void *by_row, float *row_unscale, const float *column_unscale, void *by_column,
                                long long ldp, bool dependent, cudaStream_t stream)
{
    const bool vec = in_groups(src, ld, 4, 2) && (slope == nullptr || in_groups(slope, lds, 4, 2));
    auto launch = [&](auto kernel, int threads) {
        return launch_kernel(dependent, kernel, dim3(rows), dim3(threads), 0, stream, rows, cols, static_cast<const float *>(src), ld,
                             static_cast<const float *>(slope), lds, factor, static_cast<__half *>(by_row), row_unscale, column_unscale,
                             static_cast<__half *>(by_column), ldp);
    };
    // As few threads as have room for the row: each then has more on its way to it (2047 x 3001 x 1531 with the parts of X and W:
    // 85.7 us with 256 threads to a row, 81.2 with 128; 128 to rows of 3001 as well, in two turns, 83.2).
    if (cols <= 1024) return vec ? launch(linear_parts_kernel<true, 64>, 64) : launch(linear_parts_kernel<false, 64>, 64);
    if (cols <= 2048) return vec ? launch(linear_parts_kernel<true, 128>, 128) : launch(linear_parts_kernel<false, 128>, 128);
    return vec ? launch(linear_parts_kernel<true, 256>, 256) : launch(linear_parts_kernel<false, 256>, 256);
}

}  // namespace sgemm_impl
