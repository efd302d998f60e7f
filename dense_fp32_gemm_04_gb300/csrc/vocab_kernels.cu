// Tile kernels of the vocabulary losses. Z = scale * H * W^T is computed tile by
// tile with FP32 FMAs from operands widened to FP32 and leaves a tile either as
// the softmax statistics of its columns (and the logits at the targets), or as dZ
// for the two products of the gradients.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "sgemm_internal.h"
#include "vocab_internal.h"

namespace sgemm_impl {
namespace {

constexpr int TILE = 64, BK = 16, THREADS = 256;
constexpr float kInf = __builtin_huge_valf();

// acc[i][j] of C rows 4 ty + i, columns 4 tx + j of the tile at (m0, n0):
// sum over k of A(m, k) B(n, k), element (r, k) of an operand at base + r * sr + k * sk.
template <typename EA, typename EB>
__device__ void tile_product(const EA *A, long long a_sr, long long a_sk, int m0, int M, const EB *B, long long b_sr,
                             long long b_sk, int n0, int N, int K, float (&acc)[4][4])
{
    __shared__ float sa[BK][TILE + 1], sb[BK][TILE + 1];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    for (int k0 = 0; k0 < K; k0 += BK) {
        for (int i = threadIdx.x; i < BK * TILE; i += THREADS) {
            // consecutive threads along the operand's contiguous axis
            const int ra = a_sk == 1 ? i / BK : i % TILE, ka = a_sk == 1 ? i % BK : i / TILE;
            const int rb = b_sk == 1 ? i / BK : i % TILE, kb = b_sk == 1 ? i % BK : i / TILE;
            sa[ka][ra] = m0 + ra < M && k0 + ka < K ? static_cast<float>(A[(m0 + ra) * a_sr + (k0 + ka) * a_sk]) : 0.0f;
            sb[kb][rb] = n0 + rb < N && k0 + kb < K ? static_cast<float>(B[(n0 + rb) * b_sr + (k0 + kb) * b_sk]) : 0.0f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < BK; ++k) {
            float a[4], b[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                a[i] = sa[k][4 * ty + i];
                b[i] = sb[k][4 * tx + i];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
        }
        __syncthreads();
    }
}

template <typename E, bool DZ>
__global__ void __launch_bounds__(THREADS) vocab_z_kernel(const VocabTileParams p)
{
    const int n0 = p.v0 + blockIdx.x * TILE, m0 = blockIdx.y * TILE, nend = p.v0 + p.vn;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float acc[4][4] = {};
    tile_product(static_cast<const E *>(p.H), p.ldh, 1LL, m0, p.T, static_cast<const E *>(p.W), p.ldw, 1LL, n0, nend, p.D,
                 acc);
    for (int i = 0; i < 4; ++i) {
        const long long row = m0 + 4 * ty + i;
        const bool live = row < p.T;  // every thread takes part in the shuffles
        float z[4], m = -kInf, s = 0.0f;
        for (int j = 0; j < 4; ++j) {
            const int col = n0 + 4 * tx + j;
            z[j] = col < nend ? p.scale * acc[i][j] : -kInf;
            m = fmaxf(m, z[j]);
        }
        float dz[4] = {};
        if (!DZ) {
            for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            const float base = m == -kInf ? 0.0f : m;
            for (int j = 0; j < 4; ++j) s += expf(z[j] - base);
            for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            if (live && tx == 0) p.part[static_cast<long long>(blockIdx.x) * p.T + row] = make_float2(m, s);
        }
        if (!live) continue;
        float g = 0.0f;
        if (DZ) {
            const long long y = p.t.labels != nullptr ? p.t.labels[row] : p.t.id[row * p.t.n];
            const bool used = p.t.labels != nullptr ? y >= 0 && y < p.V : y != kNoTarget;
            if (used) {
                g = p.gmult * p.dloss[row];
                const float l = p.lse[row];
                for (int j = 0; j < 4; ++j) dz[j] = g * expf(z[j] - l);
            }
        }
        for (int e = 0; e < p.t.n; ++e) {
            const long long id = p.t.labels != nullptr ? p.t.labels[row] : p.t.id[row * p.t.n + e];
            const float q = p.t.labels != nullptr ? 1.0f : p.t.q[row * p.t.n + e];
            for (int j = 0; j < 4; ++j) {
                const int col = n0 + 4 * tx + j;
                if (id != col || col >= nend) continue;
                if (DZ)
                    dz[j] -= g * q;
                else
                    p.zt[row * p.t.n + e] = z[j];
            }
        }
        if (DZ)
            for (int j = 0; j < 4; ++j) {
                const int col = n0 + 4 * tx + j;
                if (col < nend) p.G[row * p.ldg + col - p.v0] = dz[j];
            }
    }
}

template <typename E>
__global__ void __launch_bounds__(THREADS) vocab_dh_kernel(const VocabTileParams p, float *out, bool first)
{
    const int n0 = blockIdx.x * TILE, m0 = blockIdx.y * TILE;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float acc[4][4] = {};
    tile_product(p.G, p.ldg, 1LL, m0, p.T, static_cast<const E *>(p.W) + p.v0 * p.ldw, 1LL, p.ldw, n0, p.D, p.vn, acc);
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const long long row = m0 + 4 * ty + i, col = n0 + 4 * tx + j;
            if (row < p.T && col < p.D) {
                float *d = out + row * p.D + col;
                *d = first ? acc[i][j] : *d + acc[i][j];
            }
        }
}

template <typename E>
__global__ void __launch_bounds__(THREADS)
vocab_dw_kernel(const VocabTileParams p, float beta, E *__restrict__ dW, long long lddw)
{
    const int n0 = blockIdx.x * TILE, m0 = blockIdx.y * TILE;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float acc[4][4] = {};
    tile_product(p.G, 1LL, p.ldg, m0, p.vn, static_cast<const E *>(p.H), 1LL, p.ldh, n0, p.D, p.T, acc);
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const long long row = m0 + 4 * ty + i, col = n0 + 4 * tx + j;
            if (row < p.vn && col < p.D) {
                E *d = dW + (p.v0 + row) * lddw + col;
                *d = static_cast<E>(beta != 0.0f ? fmaf(beta, static_cast<float>(*d), acc[i][j]) : acc[i][j]);
            }
        }
}

unsigned tiles(int x) { return static_cast<unsigned>((x + TILE - 1) / TILE); }

}  // namespace

cudaError_t launch_vocab_forward(const VocabTileParams &p, int dtype, cudaStream_t stream)
{
    const dim3 grid(tiles(p.vn), tiles(p.T));
    if (dtype == SGEMM_DTYPE_BF16)
        vocab_z_kernel<__nv_bfloat16, false><<<grid, THREADS, 0, stream>>>(p);
    else
        vocab_z_kernel<float, false><<<grid, THREADS, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_vocab_dz(const VocabTileParams &p, int dtype, cudaStream_t stream)
{
    const dim3 grid(tiles(p.vn), tiles(p.T));
    if (dtype == SGEMM_DTYPE_BF16)
        vocab_z_kernel<__nv_bfloat16, true><<<grid, THREADS, 0, stream>>>(p);
    else
        vocab_z_kernel<float, true><<<grid, THREADS, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_vocab_dh(const VocabTileParams &p, int dtype, float *acc, bool first, cudaStream_t stream)
{
    const dim3 grid(tiles(p.D), tiles(p.T));
    if (dtype == SGEMM_DTYPE_BF16)
        vocab_dh_kernel<__nv_bfloat16><<<grid, THREADS, 0, stream>>>(p, acc, first);
    else
        vocab_dh_kernel<float><<<grid, THREADS, 0, stream>>>(p, acc, first);
    return cudaGetLastError();
}

cudaError_t launch_vocab_dw(const VocabTileParams &p, int dtype, float beta, void *dW, long long lddw,
                            cudaStream_t stream)
{
    const dim3 grid(tiles(p.D), tiles(p.vn));
    if (dtype == SGEMM_DTYPE_BF16)
        vocab_dw_kernel<<<grid, THREADS, 0, stream>>>(p, beta, static_cast<__nv_bfloat16 *>(dW), lddw);
    else
        vocab_dw_kernel<<<grid, THREADS, 0, stream>>>(p, beta, static_cast<float *>(dW), lddw);
    return cudaGetLastError();
}

}  // namespace sgemm_impl
