// Tile kernel of the vocabulary losses on the 5th-generation tensor cores. One
// persistent kernel computes all three products of 16-bit operands with FP32
// accumulation, 128 x 256 tiles per CTA or 256 x 256 tiles per CTA pair:
//   Z   = scale * H W^T   A = H (T x D, K-major), B = W (V x D, K-major); leaves
//                         the tile as softmax statistics (loss), or as dZ in
//                         bfloat16 parts (dz). Z itself is never stored.
//   dW  = dZ^T H          A = dZ (T x piece, read MN-major), B = H (MN-major)
//   dH  = dZ W            A = dZ (K-major), B = W (MN-major), split along the
//                         vocabulary into partial sums that vocab_finish adds.
// One launch of a gradient call holds the dH and dW tiles of one piece of the
// vocabulary and the dZ tiles of the next, so the partial last round of one
// product is filled by another's tiles.
//
// FP32 operands (vocab_split_kernel) are sums of 16-bit parts, a product of them
// the products of parts down to about 2^-22 of the leading one, small ones first:
// the same loop over more slabs. For Z and dH two float16 parts (22 bits) of rows
// scaled by powers of two, 3 products: an element far below its row's largest has
// fewer bits, but in the sum it stands next to the largest (for dH, dZ carries
// back the scaling of W's rows, the sum's index). For dW, where dZ spans many
// orders of magnitude and a row may be made of small ones alone, three bfloat16
// parts (24 bits at any magnitude), 6 products.
//
// Accumulation: the tensor core truncates its FP32 accumulator at every K = 16
// step (measured: rel. error 4.4e-6 at K = 4096 and up to 1.3e-5 where one sign
// prevails, all of it toward zero), which a logit of 12 would show in its loss. So
// a tile's K range is cut into segments (1024 deep for logits, 512 for those of
// FP32 operands, 256 for their dH and dW); the epilogue warps add the segments in
// registers, rounded to nearest, while the next ones run. A segment's end costs the
// tensor cores 600 to 1400 cycles, the time in which the accumulator is read beside
// them (1024 x 65536 x 2048: 190 us at 512 deep, 170 at 1024, 165 undivided).
// Logits are cut alike in a loss and in its gradients: the two calls then truncate
// them to the same bits, and p = exp(z - lse) does not see it. (Undivided in the
// gradients, p of a label's logit of 64 at K = 4096 was 8e-4 low, as much as the
// label's whole entry p - 1 where the token is learnt.) What is rounded to bfloat16
// in the end and subtracted from nothing (dW, dH of bfloat16 operands) is one
// segment: 2^-9 hides what truncation loses. Depth and error (2-norm, 2048 x 32768
// x 2048 in FP32): 256 throughout dH 4.2e-7, 2.82 ms; 512 for Z 5.3e-7, 2.76 ms;
// 512 throughout 7.3e-7, 2.76 ms.
//
// Warps of a CTA (three warpgroups): 0 TMA producer, 1 MMA issuer (rank 0 of a
// pair), 2 and 3 idle; 4..11 epilogue: warp w reads TMEM lanes 32 (w % 4) and
// columns 128 (w / 8) of the accumulator, so a thread holds 128 columns of one
// row. That takes more registers than an even share: the first warpgroup hands
// most of its own over (setmaxnreg). Ring and accumulator barriers are those of
// the TF32 kernel (tf32_kernels.cu): full / empty per stage, acc_full / acc_empty
// per accumulator, all waits bounded.
//
// What bounds it: from about 1000 tokens on the tensor cores at the clock that the
// power limit leaves them (8192 x 131072 x 4096, one loss: 4.2 to 4.5 ms = 1.95 to
// 2.1 PFLOP/s from a cool start, about 5 ms in a loop); below, the operands' way
// from memory and the start of the pipeline in each of a call's launches (256
// tokens, 32768 x 1024: 25 us for the loss, 65 us for the gradients).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "device_ptx.cuh"
#include "sgemm_internal.h"
#include "tcgen05_ptx.cuh"
#include "vocab_internal.h"

namespace sgemm_impl {
namespace {

using namespace sgemm_dev;

constexpr int kTimeoutCode = 5 << 16;
constexpr int kLayoutCode = 7 << 16;
constexpr int BK = kVocabBK;   // 64 bfloat16 = 128 bytes, one swizzle row
constexpr int BN = kVocabBN;   // 256 accumulator columns
constexpr int MMA_K = 16;
constexpr int BOX_BYTES = 64 * 64 * 2;  // every copy: 64 rows of 64 elements
constexpr int THREADS = 384;
constexpr int EPI_WARPS = 8;
// Registers per thread: at launch (the most that 384 threads can have), and after the warpgroups' exchange.
constexpr int REGS_LAUNCH = 168, REGS_ISSUE = 72, REGS_EPILOGUE = 216;
static_assert(REGS_ISSUE + 2 * REGS_EPILOGUE <= 3 * REGS_LAUNCH, "an exchange above the launch's registers never ends");
constexpr int COLS = 128;      // accumulator columns of one epilogue thread
constexpr uint32_t TMEM_COLS = 512;
constexpr int kWarpStaging = 32 * 128;  // bytes: 32 rows of 128 (64 bfloat16 or 32 floats)
constexpr float kLog2e = 1.4426950408889634f;                              // log2(e) in two FP32 parts
constexpr float kLog2eLow = static_cast<float>(1.4426950408889634 - static_cast<double>(kLog2e));
constexpr float kInf = __builtin_huge_valf();
constexpr float kLeast = 1.40129846e-45f;  // the smallest positive FP32 number

template <int CTAS>
struct Shape {
    static constexpr int BM = 128 * CTAS;
    static constexpr int CTA_N = BN / CTAS;  // columns of B staged per CTA
    static constexpr int STAGES = CTAS == 2 ? 6 : 4;
    static constexpr int A_BYTES = 128 * BK * 2;
    static constexpr int B_BYTES = CTA_N * BK * 2;
    static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
    static constexpr int SMEM = 1024 + STAGES * STAGE_BYTES + EPI_WARPS * kWarpStaging + 512;
    static_assert(SMEM <= 227 * 1024, "shared memory per CTA");
};

template <int STAGES>
struct Bars {
    uint64_t full[STAGES];
    uint64_t empty[STAGES];
    uint64_t acc_full[2];
    uint64_t acc_empty[2];
    uint64_t mma_done;
    uint32_t tmem_base;
    uint32_t ring_offset;
    int abort_flag;
    int issued[STAGES];
};
static_assert(sizeof(Bars<6>) <= 512, "barrier block");

template <int STAGES>
__device__ __forceinline__ void raise_abort(Bars<STAGES> *b, const VocabTileParams &p, int code)
{
    volatile int *f = &b->abort_flag;
    if (!*f) {
        *f = 1;
        report_status(p.status, code);
    }
}

// One tile of a launch: rows from m0, columns from n0, k-blocks [kb0, kb1).
struct Item {
    int kind, m0, n0, kb0, kb1, split;
};

// Item i of a worker. First its dH tiles (tile t, split s of all tiles, then the
// next split), which are the longest: W workers take them in turn, and those left
// with one fewer take dh_extra other tiles each in its place. Then the others in
// turn: the dW tiles (along D first: they share their slice of dZ), and the Z tiles
// (in groups of 16 tile rows, along T first: they share their rows of W, and the
// group's rows of H stay in the L2).
__device__ __forceinline__ bool item_at(const VocabTileParams &p, int i, int worker, int workers, int bm, Item &w)
{
    const int turns = p.dh_items / workers, rem = p.dh_items - turns * workers;
    const int mine = turns + (worker < rem ? 1 : 0);
    if (i < mine) {
        const int u = worker + i * workers, tiles = p.dh_tm * p.dh_tn, r = u % tiles;
        w.kind = kVocabDh;
        w.split = u / tiles;
        w.m0 = r % p.dh_tm * bm;
        w.n0 = r / p.dh_tm * BN;
        w.kb0 = w.split * p.dh_kb;
        w.kb1 = min(w.kb0 + p.dh_kb, (p.g_vn + BK - 1) / BK);
        return true;
    }
    i -= mine;
    const int few = workers - rem;  // workers with one dH tile fewer (all of them where rem is 0: then dh_extra is 0)
    int u;
    if (worker >= rem && i < p.dh_extra) {
        u = worker - rem + i * few;
    } else {
        if (worker >= rem) i -= p.dh_extra;
        u = p.dh_extra * few + (worker >= rem ? worker - rem : worker + few) + i * workers;
    }
    w.split = 0;
    w.kb0 = 0;
    if (u < p.dw_items) {
        w.kind = kVocabDw;
        w.m0 = u / p.dw_tn * bm;
        w.n0 = u % p.dw_tn * BN;
        w.kb1 = (p.T + BK - 1) / BK;
        return true;
    }
    u -= p.dw_items;
    if (u >= p.z_items) return false;
    constexpr int GROUP = 16;
    const int group = u / (GROUP * p.z_tn), rows = min(GROUP, p.z_tm - group * GROUP), r = u - group * GROUP * p.z_tn;
    w.kind = p.z_kind;
    w.m0 = (group * GROUP + r % rows) * bm;
    w.n0 = r / rows * BN;
    w.kb1 = (p.D + BK - 1) / BK;
    return true;
}

__device__ __forceinline__ int segment_blocks(const VocabTileParams &p, int kind)
{
    return kind == kVocabDw || kind == kVocabDh ? p.seg_g : p.seg_z;
}

__device__ __forceinline__ int product_count(const VocabTileParams &p, int kind)
{
    return kind == kVocabDw ? p.products : p.f16_products;
}

// Parts of A and B in product i (0..5) of the six of three parts; fewer products are the last ones.
__device__ __forceinline__ int part_a(int i) { return (0x001102 >> (4 * i)) & 3; }
__device__ __forceinline__ int part_b(int i) { return (0x010120 >> (4 * i)) & 3; }

__device__ __forceinline__ float exp2_approx(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A warp's 32 rows x 128 columns leave through its staging area: rows of 128 bytes
// with the 128-byte swizzle (16-byte chunk j of row r at j ^ (r & 7)), so that each
// lane writes its own row without bank conflicts and one TMA store (or addition)
// per 128 bytes of columns takes them out in the background, clipped to the map.

// Take the staging area back from the copies that still read it.
__device__ __forceinline__ void stage_free(int lane)
{
    if (lane == 0) bulk_wait_read();
    __syncwarp();
}

// The staged block to columns x.., rows y.. of part z.
__device__ __forceinline__ void stage_send(const CUtensorMap *map, uint32_t stg, int lane, int x, int y, int z, bool add)
{
    fence_proxy_async();
    __syncwarp();
    if (lane == 0) {
        if (add)
            tma_add_3d(map, stg, x, y, z);
        else
            tma_store_3d(map, stg, x, y, z);
        bulk_commit();
    }
}

__device__ __forceinline__ void sts128(uint32_t addr, const uint32_t (&v)[4])
{
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3])
                 : "memory");
}

// alpha * FP32 columns, 32 per block. (Scaling here and not in dZ also lets the stores' groups of four registers be
// others than the accumulator's: without it the kernel spills 60 of them. As it is, a thread spills 44 and 28 bytes in the
// bfloat16 forms, single CTAs and pairs, 136 and 96 in the FP32 ones; between tiles and in their epilogue, where 128 of
// its 216 registers are the tile.)
__device__ __forceinline__ void send_f32(const CUtensorMap *map, const float (&acc)[COLS], uint32_t stg, int lane, int x,
                                         int y, int z, int cols, bool add, float alpha)
{
#pragma unroll
    for (int cb = 0; cb < COLS / 32; ++cb) {
        if (x + cb * 32 >= cols) break;
        stage_free(lane);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float *f = acc + cb * 32 + 4 * j;
            const uint32_t v[4] = {__float_as_uint(alpha * f[0]), __float_as_uint(alpha * f[1]),
                                   __float_as_uint(alpha * f[2]), __float_as_uint(alpha * f[3])};
            sts128(stg + lane * 128 + ((j ^ (lane & 7)) << 4), v);
        }
        stage_send(map, stg, lane, x + cb * 32, y, z, add);
    }
}

// alpha * columns as bfloat16, 64 per block, in parts: each but the last leaves its remainder (exact in FP32) to the
// next. blocks > 0: to a matrix in blocks of 64 columns, `blocks` of them per part.
__device__ __forceinline__ void send_bf16(const CUtensorMap *map, float (&acc)[COLS], uint32_t stg, int lane, int x,
                                          int y, int cols, int parts, int blocks, float alpha)
{
#pragma unroll
    for (int cb = 0; cb < COLS / 64; ++cb) {
        if (x + cb * 64 >= cols) break;
        for (int part = 0;;) {
            stage_free(lane);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                uint32_t v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float *f = acc + cb * 64 + 8 * j + 2 * i;
                    const __nv_bfloat162 y2 = __floats2bfloat162_rn(alpha * f[0], alpha * f[1]);
                    v[i] = *reinterpret_cast<const uint32_t *>(&y2);
                }
                sts128(stg + lane * 128 + ((j ^ (lane & 7)) << 4), v);
            }
            if (blocks > 0)
                stage_send(map, stg, lane, 0, y, part * blocks + x / 64 + cb, false);
            else
                stage_send(map, stg, lane, x + cb * 64, y, 0, false);
            if (++part == parts) break;
#pragma unroll
            for (int i = 0; i < 64; ++i) {  // (more than one part: dZ, whose alpha is 1)
                float &f = acc[cb * 64 + i];
                f -= __bfloat162float(__float2bfloat16_rn(f));
            }
        }
    }
}

// dZ for dH as two float16 parts, in blocks of 64 columns: columns times 2^15 factor[column] / most, which undoes the
// scaling of W's row against the largest such factor, so that nothing leaves float16's range (dZ is at most 1 here).
__device__ __forceinline__ void send_f16(const CUtensorMap *map, const float (&acc)[COLS],
                                         const float *factor, float most, uint32_t stg, int lane, int x, int y,
                                         int blocks)
{
    const float up = 1.0f / most;  // a power of two
#pragma unroll
    for (int cb = 0; cb < COLS / 64; ++cb) {
        const float4 *columns = reinterpret_cast<const float4 *>(factor + cb * 64);
#pragma unroll 1
        for (int part = 0; part < 2; ++part) {
            float4 next[2] = {columns[0], columns[1]};  // fetched one chunk ahead of its use
            stage_free(lane);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                uint32_t v[4];
                const float4 now[2] = {next[0], next[1]};
                if (j < 7) {
                    next[0] = columns[2 * j + 2];
                    next[1] = columns[2 * j + 3];
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float *f = acc + cb * 64 + 8 * j + 2 * i;
                    const float ux = i & 1 ? now[i / 2].z : now[i / 2].x, uy = i & 1 ? now[i / 2].w : now[i / 2].y;
                    const float a = f[0] * (ux * up * 32768.0f), b = f[1] * (uy * up * 32768.0f);
                    __half2 y2 = __floats2half2_rn(a, b);
                    if (part == 1) {
                        const float2 back = __half22float2(y2);
                        y2 = __floats2half2_rn(a - back.x, b - back.y);
                    }
                    v[i] = *reinterpret_cast<const uint32_t *>(&y2);
                }
                sts128(stg + lane * 128 + ((j ^ (lane & 7)) << 4), v);
            }
            stage_send(map, stg, lane, 0, y, part * blocks + x / 64 + cb, false);
        }
    }
}

// Rows that a TMA store cannot write (not 16-byte aligned), or that are added to (beta != 0), element by element or
// four at a time: 32 columns of FP32 staged, element (r, c) at 32 r + (c ^ r), then read back along rows.
template <typename E>
__device__ __forceinline__ void write_rows(const float (&acc)[COLS], float *stg, int lane, E *dst, long long ld, int rows,
                                           int cols, bool vec, float alpha, float beta)
{
#pragma unroll
    for (int cb = 0; cb < COLS / 32; ++cb) {
        stage_free(lane);
#pragma unroll
        for (int i = 0; i < 32; ++i) stg[lane * 32 + (i ^ lane)] = alpha * acc[cb * 32 + i];
        __syncwarp();
        if (vec) {  // 8 lanes per row
            const int sub = lane >> 3, c = 4 * (lane & 7);
            for (int k = 0; k < 8; ++k) {
                const int r = 4 * k + sub;
                float x[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] = stg[r * 32 + ((c + e) ^ r)];
                if (r >= rows || cb * 32 + c >= cols) continue;
                E *d = dst + r * ld + cb * 32 + c;
                if (cb * 32 + c + 3 < cols) {
                    if constexpr (sizeof(E) == 4) {
                        float4 y = beta != 0.0f ? *reinterpret_cast<const float4 *>(d) : make_float4(0, 0, 0, 0);
                        *reinterpret_cast<float4 *>(d) = make_float4(fmaf(beta, y.x, x[0]), fmaf(beta, y.y, x[1]),
                                                                     fmaf(beta, y.z, x[2]), fmaf(beta, y.w, x[3]));
                    } else {
                        __nv_bfloat162 *d2 = reinterpret_cast<__nv_bfloat162 *>(d);
                        const float2 y0 = beta != 0.0f ? __bfloat1622float2(d2[0]) : make_float2(0, 0);
                        const float2 y1 = beta != 0.0f ? __bfloat1622float2(d2[1]) : make_float2(0, 0);
                        d2[0] = __floats2bfloat162_rn(fmaf(beta, y0.x, x[0]), fmaf(beta, y0.y, x[1]));
                        d2[1] = __floats2bfloat162_rn(fmaf(beta, y1.x, x[2]), fmaf(beta, y1.y, x[3]));
                    }
                } else {
                    for (int e = 0; e < 4; ++e)
                        if (cb * 32 + c + e < cols)
                            d[e] = static_cast<E>(beta != 0.0f ? fmaf(beta, static_cast<float>(d[e]), x[e]) : x[e]);
                }
            }
        } else {  // 32 lanes along one row
            const int c = cb * 32 + lane;
#pragma unroll 4
            for (int r = 0; r < 32; ++r) {
                float x = stg[r * 32 + (lane ^ r)];
                if (r < rows && c < cols) {
                    E *d = dst + r * ld + c;
                    if (beta != 0.0f) x = fmaf(beta, static_cast<float>(*d), x);
                    *d = static_cast<E>(x);
                }
            }
        }
        __syncwarp();
    }
}

// Whether a token counts: it has a label, or a teacher's entry, in the vocabulary.
__device__ __forceinline__ bool is_used(const VocabTileParams &p, long long row)
{
    if (row >= p.T) return false;
    const long long y = p.t.labels != nullptr ? p.t.labels[row] : p.t.id[row * p.t.n];
    return p.t.labels != nullptr ? y >= 0 && y < p.V : y != kNoTarget;
}

// dloss of a token, 0 for a masked one.
__device__ __forceinline__ float load_dloss(const VocabTileParams &p, long long row)
{
    return is_used(p, row) ? p.dloss[row] : 0.0f;
}

// dZ of bfloat16 operands is kept divided by the significand of the first dloss that counts, a number in [1, 2), and dH and
// dW are multiplied by it. The losses' gradients are mostly one number, 1 / tokens, and the label's entry of dZ that number
// times p - 1: rounded as it is, all labels' entries would be off by much the same share; divided, it lies just below a
// power of two, where bfloat16 is densest (mean loss of an untrained head, dH off by 1.68e-3 of its norm, which is the
// result's own rounding; undivided 1.70e-3 over 1000 tokens, 1.99e-3 over 700, 2.43e-3 over 513). Masked tokens may hold
// anything, and a prompt is masked first: the warp looks past them, 256 tokens at a time, while the first tile's products
// run.
__device__ __forceinline__ float significand(const VocabTileParams &p, int lane)
{
    if (p.dloss == nullptr) return 1.0f;
    for (int t0 = 0; t0 < p.T; t0 += 256) {
        bool used[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) used[j] = is_used(p, t0 + 32 * j + lane);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const unsigned some = __ballot_sync(0xffffffffu, used[j]);
            if (some == 0) continue;
            const uint32_t bits = __float_as_uint(p.dloss[t0 + 32 * j + __ffs(some) - 1]), exponent = bits >> 23 & 255u;
            return exponent == 0 || exponent == 255 ? 1.0f : __uint_as_float((bits & 0x7fffffu) | 0x3f800000u);
        }
    }
    return 1.0f;
}

// What a thread needs to know of its row before the tile is there: fetched while the products run.
struct Row {
    int entry, id;   // the first target with an id of at least the tile's first column, and that id
    float q;
    float g, lse;    // dZ: the loss' gradient (0 for a masked token), log-sum-exp
    float scale;     // of the logits, with what undoes the scaling of H's row
    bool used;
};

__device__ __forceinline__ void load_target(const VocabTileParams &p, Row &r, long long row)
{
    r.id = kNoTarget;
    if (r.entry < p.t.n) {
        r.id = p.t.id[row * p.t.n + r.entry];
        r.q = p.t.q[row * p.t.n + r.entry];
    }
}

template <bool F16>
__device__ __forceinline__ Row load_row(const VocabTileParams &p, long long row, int c0, bool dz, float divide)
{
    Row r{};
    r.id = kNoTarget;
    r.scale = p.scale;
    if (row >= p.T) return r;
    if (F16) r.scale *= p.h_unscale[row];
    if (p.t.labels != nullptr) {
        const long long y = p.t.labels[row];
        r.used = y >= 0 && y < p.V;
        if (r.used && y >= c0) r.id = static_cast<int>(y);
        r.q = 1.0f;
    } else {
        const int *id = p.t.id + row * p.t.n;
        if (dz) r.used = id[0] != kNoTarget;
        int hi = p.t.n;
        while (r.entry < hi) {
            const int mid = (r.entry + hi) >> 1;
            if (id[mid] < c0)
                r.entry = mid + 1;
            else
                hi = mid;
        }
        load_target(p, r, row);
    }
    if (dz) {
        if (r.used) r.g = F16 ? p.dloss[row] : p.dloss[row] / divide;
        r.lse = p.lse[row];
    }
    return r;
}

// f(column - c0) for the row's targets in [c0, c0 + 128) one after the other; r.entry and r.q are the target's.
template <typename F>
__device__ __forceinline__ void for_targets(const VocabTileParams &p, Row &r, long long row, int c0, F f)
{
    while (r.id < c0 + COLS) {  // (kNoTarget, and V and above, are past every tile)
        f(r.id - c0);
        if (p.t.labels != nullptr) return;
        ++r.entry;
        load_target(p, r, row);
    }
}

// 32 of the thread's columns, as the TMEM loads take them.
__device__ __forceinline__ float (&columns(float (&acc)[COLS], int cb))[32]
{
    return reinterpret_cast<float(&)[32]>(acc[cb * 32]);
}

// Undo the scaling of W's rows (the same columns for every lane: broadcast loads; plain ones, here and in send_f16: the call's
// previous kernel wrote the factors while this one may already have been resident).
__device__ __forceinline__ void unscale_columns(const float *factor, float (&z)[COLS])
{
#pragma unroll
    for (int i = 0; i < COLS; i += 4) {
        const float4 f = *reinterpret_cast<const float4 *>(factor + i);
        z[i] *= f.x;
        z[i + 1] *= f.y;
        z[i + 2] *= f.z;
        z[i + 3] *= f.w;
    }
}

// Z tile of a loss call: the softmax statistics of the thread's columns, and the logits at its targets. z = scale * acc;
// the exponentials are powers of two, exp(z - m) = 2^(k acc - M) with k = scale log2(e) and M = k max(acc) rounded: M is
// what the pair holds, so its rounding costs nothing, until M's last bit is worth as much as the range of an exponential:
// from kHugeLog2 on the other products are rounded as M was, none of which is then above it.
__device__ __forceinline__ void leave_loss(const VocabTileParams &p, float (&z)[COLS], Row &r, long long row, int c0)
{
    const int cols = p.V - c0;  // columns of the vocabulary from c0 on
    if (cols < COLS) {
#pragma unroll
        for (int i = 0; i < COLS; ++i) z[i] = i < cols ? z[i] : -kInf;
    }
    float m[4] = {-kInf, -kInf, -kInf, -kInf};
#pragma unroll
    for (int i = 0; i < COLS; ++i) m[i & 3] = fmaxf(m[i & 3], z[i]);
    for_targets(p, r, row, c0, [&](int at) {
        float x = 0.0f;
#pragma unroll
        for (int i = 0; i < COLS; ++i) x = i == at ? z[i] : x;
        if (index_ok(row < p.T && r.entry >= 0 && r.entry < p.t.n, p.status, kWhereIdxVocabTarget))
            p.zt[row * p.t.n + r.entry] = r.scale * x;
    });
    // (not 0, which a tiny scale on a row of zeros would give: it must leave the columns past V at -infinity)
    float k = fmaxf(r.scale * kLog2e, kLeast);
    const float top = k * fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
    const float base = top == -kInf ? 0.0f : -top;
    if (fabsf(base) >= kHugeLog2) {  // products rounded as M was
#pragma unroll
        for (int i = 0; i < COLS; ++i) z[i] = __fmul_rn(k, z[i]);
        k = 1.0f;
    }
    const unsigned long long k2 = pack_f32x2(k, k), b2 = pack_f32x2(base, base);
    unsigned long long s2[4] = {};
#pragma unroll
    for (int i = 0; i < COLS; i += 2) {
        float x, y;
        unpack_f32x2(fma_f32x2(pack_f32x2(z[i], z[i + 1]), k2, b2), x, y);
        s2[i / 2 & 3] = add_f32x2(s2[i / 2 & 3], pack_f32x2(exp2_approx(x), exp2_approx(y)));
    }
    float x, y;
    unpack_f32x2(add_f32x2(add_f32x2(s2[0], s2[1]), add_f32x2(s2[2], s2[3])), x, y);
    if (row < p.T && index_ok(c0 / COLS < p.stat_cols, p.status, kWhereIdxVocabStat))
        p.part[static_cast<long long>(c0 / COLS) * p.T + row] = make_float2(top, x + y);
}

// Z tile of a gradient call, made into dZ / alpha = dloss (exp(z - lse) - q); for float16
// parts without dloss, which the sums over the vocabulary and the bfloat16 parts are multiplied by instead.
template <bool F16>
__device__ __forceinline__ void make_dz(const VocabTileParams &p, float (&z)[COLS], Row &r, long long row, int c0)
{
    // exp(z - lse) = 2^(k acc - L) 2^-l with L + l = lse log2(e), L rounded and l its remainder: l goes into the factor.
    // No probability is above 1: with a huge lse (1e9 is a multiple of 64) p, or l's factor, could leave the range of
    // FP32 or of dZ's parts. (A NaN logit has made lse NaN, and so l, which passes.)
    const float k = r.scale * kLog2e, L = r.lse * kLog2e;
    float l = fmaf(r.lse, kLog2e, -L) + r.lse * kLog2eLow;
    l = l > 100.0f ? 100.0f : l < -100.0f ? -100.0f : l;
    const float weight = F16 ? 1.0f : r.g, g = weight * exp2_approx(-l);
    const unsigned long long k2 = pack_f32x2(k, k), b2 = pack_f32x2(-L, -L), g2 = pack_f32x2(g, g);
#pragma unroll
    for (int i = 0; i < COLS; i += 2) {
        float x, y;
        unpack_f32x2(fma_f32x2(pack_f32x2(z[i], z[i + 1]), k2, b2), x, y);
        x = fminf(x, l);
        y = fminf(y, l);
        unpack_f32x2(mul_f32x2(pack_f32x2(exp2_approx(x), exp2_approx(y)), g2), z[i], z[i + 1]);
    }
    // a masked token's dZ is 0 whatever its logits are; so is dZ past the vocabulary, which the products do read
    const int cols = r.used ? p.V - c0 : 0;
    if (cols < COLS) {
#pragma unroll
        for (int i = 0; i < COLS; ++i) z[i] = i < cols ? z[i] : 0.0f;
    }
    int last = -1;
    for_targets(p, r, row, c0, [&](int at) {
        float keep = 1.0f, add = -weight * r.q;
        if (p.zt != nullptr && at != last) {  // a few tokens: p of the logit that the loss had (vocab_few.cu)
            keep = 0.0f;
            add += g * exp2_approx(fminf(fmaf(p.zt[row * p.t.n + r.entry], p.scale * kLog2e, -L), l));
            last = at;
        }
#pragma unroll
        for (int i = 0; i < COLS; ++i) z[i] = i == at ? fmaf(keep, z[i], add) : z[i];
    });
}

// Producer thread: this CTA's part of each stage, in boxes of 64 rows x 64 elements.
template <int CTAS>
__device__ __forceinline__ void produce(const VocabTileParams &p, Bars<Shape<CTAS>::STAGES> *bars, uint32_t a_base,
                                        uint32_t b_base, const VocabMaps &maps, uint32_t rank, int worker, int workers)
{
    using S = Shape<CTAS>;
    constexpr int STAGES = S::STAGES;
    constexpr bool PAIR = CTAS == 2;
    volatile int *abort_flag = &bars->abort_flag;
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    Item w;
    for (int i = 0; ok && item_at(p, i, worker, workers, S::BM, w); ++i) {
        const bool z = w.kind == kVocabLoss || w.kind == kVocabDz;
        const CUtensorMap *ta = z ? &maps.Hz : w.kind == kVocabDw ? &maps.G : &maps.Gz;
        const CUtensorMap *tb = w.kind == kVocabDw ? &maps.H : &maps.W;
        const bool a_k = w.kind != kVocabDw, b_k = z;  // K-major: K along the map's rows
        const int a_r = w.m0 + static_cast<int>(rank) * 128;
        const int b_r = w.n0 + static_cast<int>(rank) * S::CTA_N + (z ? p.z_v0 : 0);
        const int b_k0 = w.kind == kVocabDh ? p.g_v0 : 0;
        const int seg = segment_blocks(p, w.kind);
        for (int s0 = w.kb0; ok && s0 < w.kb1; s0 += seg) {
            const int s1 = min(s0 + seg, w.kb1);
            for (int pr = 6 - product_count(p, w.kind); ok && pr < 6; ++pr) {
                const int pa = part_a(pr), pb = part_b(pr);
                for (int kb = s0; kb < s1; ++kb) {
                    if (!mbar_wait_quiet<false>(smem_addr(&bars->empty[stage]), phase ^ 1u, abort_flag, p.timeout_ns)) {
                        raise_abort(bars, p, kTimeoutCode | kWhereProducerEmpty);
                        ok = false;
                        break;
                    }
                    const uint32_t a_dst = a_base + stage * S::A_BYTES;
                    const uint32_t b_dst = b_base + stage * S::B_BYTES;
                    if (rank == 0) mbar_arrive_expect_tx(smem_addr(&bars->full[stage]), CTAS * S::STAGE_BYTES);
                    uint32_t full = smem_addr(&bars->full[stage]);
                    if constexpr (PAIR) full = mapa_shared(full, 0);  // rank 0's barrier
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        // H: (k, token, part); dZ, in blocks of 64 entries: (entry, token, block of the part)
                        const int x = z ? kb * BK : 0;
                        const int y = a_k ? a_r + 64 * j : kb * BK;
                        const int b = z ? pa : pa * p.g_blocks + (a_k ? kb : a_r / 64 + j);
                        if constexpr (PAIR)
                            tma_load_3d_pair(a_dst + j * BOX_BYTES, ta, full, x, y, b);
                        else
                            tma_load_3d(a_dst + j * BOX_BYTES, ta, full, x, y, b);
                    }
#pragma unroll
                    for (int j = 0; j < S::CTA_N / 64; ++j) {
                        const int x = b_k ? kb * BK : b_r + 64 * j, y = b_k ? b_r + 64 * j : b_k0 + kb * BK;
                        if constexpr (PAIR)
                            tma_load_3d_pair(b_dst + j * BOX_BYTES, tb, full, x, y, pb);
                        else
                            tma_load_3d(b_dst + j * BOX_BYTES, tb, full, x, y, pb);
                    }
                    bars->issued[stage] = 2 | static_cast<int>(phase);
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
        }
    }
    pdl_trigger();  // every copy is issued: the call's next kernel may become resident
    // Drain, as in the TF32 kernel: every issued copy has landed (rank 0's barriers count both
    // CTAs'), and unless aborted the MMAs that read it have committed.
    for (int s = 0; s < STAGES; ++s) {
        const int rec = bars->issued[s];
        if (!(rec & 2)) continue;
        const uint32_t par = static_cast<uint32_t>(rec & 1);
        if (rank == 0 && !mbar_wait_quiet<true>(smem_addr(&bars->full[s]), par, nullptr, p.timeout_ns)) {
            report_status(p.status, kTimeoutCode | kWhereDrain);
            break;
        }
        if (!*abort_flag && !mbar_wait_quiet<false>(smem_addr(&bars->empty[s]), par, abort_flag, p.timeout_ns)) {
            report_status(p.status, kTimeoutCode | kWhereDrain);
            break;
        }
    }
}

// MMA thread (rank 0 of a pair): four K = 16 steps per slab, a commit per stage and per segment.
template <int CTAS, bool F16>
__device__ __forceinline__ void issue(const VocabTileParams &p, Bars<Shape<CTAS>::STAGES> *bars, uint32_t a_base,
                                      uint32_t b_base, uint32_t tmem, int worker, int workers)
{
    using S = Shape<CTAS>;
    constexpr int STAGES = S::STAGES;
    constexpr bool PAIR = CTAS == 2;
    volatile int *abort_flag = &bars->abort_flag;
    int stage = 0;
    uint32_t phase = 0;
    int it = 0;  // segments so far
    bool ok = true;
    Item w;
    for (int i = 0; ok && item_at(p, i, worker, workers, S::BM, w); ++i) {
        const bool a_mn = w.kind == kVocabDw, b_mn = w.kind == kVocabDw || w.kind == kVocabDh;
        const uint32_t idesc = idesc_16(S::BM, BN, a_mn, b_mn, F16 && w.kind != kVocabDw);
        const int seg = segment_blocks(p, w.kind);
        for (int s0 = w.kb0; ok && s0 < w.kb1; s0 += seg, ++it) {
            const int buf = it & 1;
            const uint32_t acc_phase = static_cast<uint32_t>(it >> 1) & 1u;
            if (!mbar_wait_quiet<true>(smem_addr(&bars->acc_empty[buf]), acc_phase ^ 1u, abort_flag,
                                           p.timeout_ns)) {
                raise_abort(bars, p, kTimeoutCode | kWhereAccum);
                ok = false;
                break;
            }
            tc_fence_after_sync();
            const uint32_t d_tmem = tmem + static_cast<uint32_t>(buf * BN);
            const int slabs = (min(s0 + seg, w.kb1) - s0) * product_count(p, w.kind);
            for (int j = 0; j < slabs; ++j) {
                if (!mbar_wait_quiet<true>(smem_addr(&bars->full[stage]), phase, abort_flag, p.timeout_ns)) {
                    raise_abort(bars, p, kTimeoutCode | kWhereMmaEmpty);
                    ok = false;
                    break;
                }
                tc_fence_after_sync();
                const uint32_t a_s = a_base + stage * S::A_BYTES;
                const uint32_t b_s = b_base + stage * S::B_BYTES;
#pragma unroll
                for (int k = 0; k < BK / MMA_K; ++k) {
                    // K-major: 16 elements = 32 bytes inside the swizzle row; MN-major: 16 K-rows of 128 bytes
                    const uint64_t a_desc = a_mn ? smem_desc_mn_sw128(a_s + k * MMA_K * 128, BOX_BYTES)
                                                 : smem_desc_k_sw128(a_s + k * MMA_K * 2);
                    const uint64_t b_desc = b_mn ? smem_desc_mn_sw128(b_s + k * MMA_K * 128, BOX_BYTES)
                                                 : smem_desc_k_sw128(b_s + k * MMA_K * 2);
                    const uint32_t accumulate = (j | k) != 0 ? 1u : 0u;
                    if constexpr (PAIR)
                        mma_16_pair(d_tmem, a_desc, b_desc, idesc, accumulate);
                    else
                        mma_16(d_tmem, a_desc, b_desc, idesc, accumulate);
                }
                if constexpr (PAIR)
                    mma_commit_pair_both(smem_addr(&bars->empty[stage]));
                else
                    mma_commit(smem_addr(&bars->empty[stage]));
                if (++stage == STAGES) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            if (!ok) break;
            if constexpr (PAIR)
                mma_commit_pair_both(smem_addr(&bars->acc_full[buf]));
            else
                mma_commit(smem_addr(&bars->acc_full[buf]));
        }
    }
    if constexpr (PAIR)
        mma_commit_pair_local(smem_addr(&bars->mma_done));
    else
        mma_commit(smem_addr(&bars->mma_done));
    if (!mbar_wait_quiet<false>(smem_addr(&bars->mma_done), 0u, nullptr, p.timeout_ns))
        report_status(p.status, kTimeoutCode | kWhereDrain);
}

// Epilogue warp: the segments of a tile added up in registers, then the tile left as its kind wants it.
template <int CTAS, bool F16>
__device__ __forceinline__ void leave_tiles(const VocabTileParams &p, Bars<Shape<CTAS>::STAGES> *bars,
                                            unsigned char *staging, const VocabMaps &maps, uint32_t tmem, uint32_t rank,
                                            int warp, int lane, int worker, int workers)
{
    using S = Shape<CTAS>;
    constexpr bool PAIR = CTAS == 2;
    volatile int *abort_flag = &bars->abort_flag;
    const int quarter = warp & 3, half = warp >> 3;
    unsigned char *area = staging + (warp - 4) * kWarpStaging;
    const uint32_t stg = smem_addr(area);
    const float divide = F16 ? 1.0f : significand(p, lane);
    int it = 0;
    bool ok = true;
    Item w;
    for (int i = 0; ok && item_at(p, i, worker, workers, S::BM, w); ++i) {
        float acc[COLS];
        const int seg = segment_blocks(p, w.kind);
        const int r0 = w.m0 + static_cast<int>(rank) * 128 + quarter * 32;  // the warp's first row
        const int c0 = w.n0 + half * COLS;
        Row r{};
        if (w.kind == kVocabLoss || w.kind == kVocabDz)
            r = load_row<F16>(p, r0 + lane, p.z_v0 + c0, w.kind == kVocabDz, divide);
        else if (F16 && w.kind == kVocabDh)
            r.g = load_dloss(p, r0 + lane);
        for (int s0 = w.kb0; s0 < w.kb1; s0 += seg, ++it) {
            const int buf = it & 1;
            const uint32_t acc_phase = static_cast<uint32_t>(it >> 1) & 1u;
            ok = mbar_wait_quiet<true>(smem_addr(&bars->acc_full[buf]), acc_phase, abort_flag, p.timeout_ns);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) {
                if (lane == 0) raise_abort(bars, p, kTimeoutCode | kWhereAccum);
                break;
            }
            tc_fence_after_sync();
            const uint32_t t = tmem + (static_cast<uint32_t>(quarter * 32) << 16) +
                               static_cast<uint32_t>(buf * BN + half * COLS);
            if (s0 == w.kb0) {
#pragma unroll
                for (int cb = 0; cb < COLS / 32; ++cb) tmem_ld_32(t + cb * 32, columns(acc, cb));
#pragma unroll
                for (int cb = 0; cb < COLS / 32; ++cb) tmem_wait_ld_32(columns(acc, cb));
            } else {
#pragma unroll
                for (int cb = 0; cb < COLS / 32; ++cb) {
                    float v[32];
                    tmem_ld_32(t + cb * 32, v);
                    tmem_wait_ld_32(v);
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        float *x = acc + cb * 32 + i;
                        unpack_f32x2(add_f32x2(pack_f32x2(x[0], x[1]), pack_f32x2(v[i], v[i + 1])), x[0], x[1]);
                    }
                }
            }
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                if constexpr (PAIR)
                    mbar_arrive_cluster(mapa_shared(smem_addr(&bars->acc_empty[buf]), 0));  // rank 0's
                else
                    mbar_arrive(smem_addr(&bars->acc_empty[buf]));
            }
        }
        if (!ok) break;
        if (F16 && (w.kind == kVocabLoss || w.kind == kVocabDz)) unscale_columns(p.w_unscale + p.z_v0 + c0, acc);
        if (w.kind == kVocabLoss) {
            leave_loss(p, acc, r, r0 + lane, p.z_v0 + c0);
            continue;
        }
        // the rest are rows of a matrix: rows from `row` and columns from c0 of the map, as FP32 or in bfloat16 parts
        const CUtensorMap *map = &maps.dW;
        const bool wide = w.kind == kVocabDh || (w.kind == kVocabDw && p.dtype == SGEMM_DTYPE_F32);
        int row = r0, cols = p.D, parts = 1, blocks = 0;
        float alpha = F16 ? p.alpha : p.alpha * divide;
        bool inside = r0 < p.T;
        if (w.kind == kVocabDz) {
            make_dz<F16>(p, acc, r, r0 + lane, p.z_v0 + c0);
            map = &maps.Gw;
            cols = p.g_blocks * 64;
            parts = F16 ? p.parts : 1;
            blocks = p.g_blocks;
            alpha = 1.0f;
            inside = inside && index_ok(c0 + COLS <= cols, p.status, kWhereIdxVocabDz);
            if (F16 && inside) {
                if (p.dh_tm > 0)
                    send_f16(&maps.Gzw, acc, p.w_unscale + p.z_v0 + c0, *p.w_most, stg, lane, c0, row, blocks);
                if (p.dw_tn == 0) continue;
#pragma unroll
                for (int i = 0; i < COLS; ++i) acc[i] *= r.g;
            }
        } else if (w.kind == kVocabDh) {
            map = &maps.acc;
            if (F16) alpha *= r.g * *p.w_most * (1.0f / 32768.0f);
            inside = inside && index_ok(w.split >= 0 && w.split < p.dh_splits, p.status, kWhereIdxVocabDh);
        } else {
            row = p.g_v0 + r0;
            inside = r0 < p.g_vn && index_ok(row < p.V && p.g_v0 + p.g_vn <= p.V, p.status, kWhereIdxVocabDw);
        }
        if (!inside) continue;
        if (w.kind == kVocabDw && !p.dw_tma) {
            const long long at = static_cast<long long>(row) * p.lddw + c0;
            if (wide)
                write_rows(acc, reinterpret_cast<float *>(area), lane, static_cast<float *>(p.dW) + at, p.lddw,
                           p.g_vn - r0, p.D - c0, p.dw_vec, alpha, p.beta);
            else
                write_rows(acc, reinterpret_cast<float *>(area), lane, static_cast<__nv_bfloat16 *>(p.dW) + at, p.lddw,
                           p.g_vn - r0, p.D - c0, p.dw_vec, alpha, p.beta);
        } else if (wide) {
            send_f32(map, acc, stg, lane, c0, row, w.split, cols, w.kind == kVocabDh && p.acc_add, alpha);
        } else {
            send_bf16(map, acc, stg, lane, c0, row, cols, parts, blocks, alpha);
        }
    }
    if (lane == 0) bulk_wait();  // the staging area is read and everything is written before the CTA ends
}

// F16: FP32 operands, whose Z and dH run on float16 parts (a kernel of its own: the code of the parts costs the other
// 2 %).
template <int CTAS, bool F16>
__global__ void __launch_bounds__(THREADS, 1)
vocab_kernel(const __grid_constant__ VocabMaps maps, const __grid_constant__ VocabTileParams p)
{
    using S = Shape<CTAS>;
    constexpr int STAGES = S::STAGES;
    constexpr bool PAIR = CTAS == 2;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    unsigned char *smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    const uint32_t a_base = smem_addr(smem);
    const uint32_t b_base = a_base + STAGES * S::A_BYTES;
    unsigned char *staging = smem + STAGES * S::STAGE_BYTES;
    Bars<STAGES> *bars = reinterpret_cast<Bars<STAGES> *>(staging + EPI_WARPS * kWarpStaging);
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    if (PAIR && cluster_size() != 2) {
        if (threadIdx.x == 0) report_status(p.status, kLayoutCode | kWherePairLayout);
        return;
    }
    const uint32_t rank = PAIR ? cluster_ctarank() : 0u;
    const int worker = PAIR ? static_cast<int>(cluster_id_x()) : static_cast<int>(blockIdx.x);
    const int workers = PAIR ? static_cast<int>(cluster_count_x()) : static_cast<int>(gridDim.x);

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(smem_addr(&bars->full[s]), 1);
            mbar_init(smem_addr(&bars->empty[s]), 1);
            bars->issued[s] = 0;
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_addr(&bars->acc_full[b]), 1);
            mbar_init(smem_addr(&bars->acc_empty[b]), EPI_WARPS * CTAS);
        }
        mbar_init(smem_addr(&bars->mma_done), 1);
        bars->abort_flag = 0;
        bars->ring_offset = a_base;
        fence_barrier_init();
        prefetch_tensormap(&maps.Hz);
        prefetch_tensormap(&maps.W);
        prefetch_tensormap(&maps.G);
    }
    if (warp == 0) {
        if constexpr (PAIR) {
            tmem_alloc_pair(smem_addr(&bars->tmem_base), TMEM_COLS);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(smem_addr(&bars->tmem_base), TMEM_COLS);
            tmem_relinquish();
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    if constexpr (PAIR) cluster_sync();  // both CTAs' barriers are initialised before any copy or arrive targets them
    tc_fence_after_sync();
    const uint32_t tmem = bars->tmem_base;
    bool same_layout = true;
    if constexpr (PAIR) {
        constexpr uint32_t kDescAddrMask = 0x3FFFFu;
        const uint32_t peer_ring = ld_shared_cluster_u32(mapa_shared(smem_addr(&bars->ring_offset), rank ^ 1u));
        same_layout = ((peer_ring ^ a_base) & kDescAddrMask) == 0;
        if (!same_layout && threadIdx.x == 0) raise_abort(bars, p, kLayoutCode | kWherePairLayout);
    }

    pdl_wait();  // the call's previous kernel is complete
    // Where the pair's layouts differ both CTAs see it: no copies, no MMAs.
    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_ISSUE));
        if (same_layout && warp == 0 && lane == 0)
            produce<CTAS>(p, bars, a_base, b_base, maps, rank, worker, workers);
        else if (same_layout && warp == 1 && lane == 0 && rank == 0)
            issue<CTAS, F16>(p, bars, a_base, b_base, tmem, worker, workers);
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_EPILOGUE));
        if (same_layout) leave_tiles<CTAS, F16>(p, bars, staging, maps, tmem, rank, warp, lane, worker, workers);
    }

    tc_fence_before_sync();
    __syncthreads();
    if constexpr (PAIR) cluster_sync();  // neither CTA leaves while the other may still use its barriers, stages or TMEM
    tc_fence_after_sync();
    if (warp == 0) {
        __syncwarp();
        if constexpr (PAIR)
            tmem_dealloc_pair(tmem, TMEM_COLS);
        else
            tmem_dealloc(tmem, TMEM_COLS);
    }
}

// bfloat16 rows at any stride -> rows on 128-byte lines. 64 threads per row, two elements each: 4-byte stores, and loads
// that need no alignment (50021 x 1531: 49 us, 6.3 TB/s).
__global__ void __launch_bounds__(256)
vocab_copy_kernel(const __nv_bfloat16 *__restrict__ src, long long ld, int rows, int cols,
                  __nv_bfloat16 *__restrict__ dst, long long ldd)
{
    pdl_wait();
    pdl_trigger();
    const long long r = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y;
    if (r >= rows) return;
    const __nv_bfloat16 *s = src + r * ld;
#pragma unroll 4
    for (int c = threadIdx.x * 2; c < ldd; c += 128) {
        const __nv_bfloat16 zero = __float2bfloat16_rn(0.0f);
        const __nv_bfloat162 y(c < cols ? __ldg(s + c) : zero, c + 1 < cols ? __ldg(s + c + 1) : zero);
        *reinterpret_cast<__nv_bfloat162 *>(dst + r * ldd + c) = y;
    }
}

// FP32 rows at any stride -> 16-bit parts in rows on 128-byte lines, a warp per row:
//   f16:  x 2^s = x0 + x1 in float16, s for each row such that its largest finite element lands in [2^14, 2^15);
//         2^-s is kept (2^-126 for rows without such an element and for those up to `padded`), and the largest of
//         them in *most; *clear is the next such word to set to 0. (The row is read a second time from the cache.)
//   BF parts in bfloat16: x = x0 + x1 (+ x2), each the remainder rounded to nearest; three hold all 24 bits. A value
//         that would round to infinity is truncated instead.
// Infinities and NaN stay in the first part. VEC: rows can be read 16 bytes at a time. (32768 x 2048, float16 parts: 106
// us, 5.1 TB/s.)
template <int BF, bool VEC>
__global__ void __launch_bounds__(256)
vocab_split_kernel(const float *__restrict__ src, long long ld, int rows, int cols, __half *__restrict__ f16,
                   float *__restrict__ unscale, int padded, float *__restrict__ most_scale, float *__restrict__ clear,
                   __nv_bfloat16 *__restrict__ bf, long long ldd)
{
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x;
    const long long r = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y;
    if (clear != nullptr && r == 0 && lane == 0) *clear = 0.0f;
    if (r >= rows) {
        if (r < padded && lane == 0) unscale[r] = scalbnf(1.0f, -126);
        return;
    }
    const float *s = src + r * ld;
    const long long part = rows * ldd;
    auto load = [&](int c, float (&x)[4]) {
        if (VEC && c + 4 <= cols) {
            const float4 v = __ldg(reinterpret_cast<const float4 *>(s + c));
            x[0] = v.x;
            x[1] = v.y;
            x[2] = v.z;
            x[3] = v.w;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = c + i < cols ? __ldg(s + c + i) : 0.0f;
        }
    };
    int e = 0;
    if (f16 != nullptr) {
        float most = 0.0f;
#pragma unroll 4
        for (int c = lane * 4; c < cols; c += 128) {
            float x[4];
            load(c, x);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float a = fabsf(x[i]);
                most = a < kInf ? fmaxf(most, a) : most;
            }
        }
        for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
        e = most > 0.0f ? min(14 - ilogbf(most), 126) : 126;
        if (lane == 0) {
            const float back = scalbnf(1.0f, -e);
            unscale[r] = back;
            // positive FP32 numbers are ordered as their bits are; nearly all rows see that they add nothing
            if (most_scale != nullptr && back > *static_cast<volatile float *>(most_scale))
                atomicMax(reinterpret_cast<int *>(most_scale), __float_as_int(back));
        }
    }
    const float up = scalbnf(1.0f, e / 2), up2 = scalbnf(1.0f, e - e / 2);  // 2^e itself may not be an FP32 number
#pragma unroll 4
    for (int c = lane * 4; c < ldd; c += 128) {
        float x[4];
        load(c, x);
        if (f16 != nullptr) {
            __half y[2][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float a = x[i] * up * up2;
                y[0][i] = __float2half_rn(a);
                y[1][i] = fabsf(a) < kInf ? __float2half_rn(a - __half2float(y[0][i])) : __float2half_rn(0.0f);
            }
            *reinterpret_cast<uint2 *>(f16 + r * ldd + c) = *reinterpret_cast<const uint2 *>(y[0]);
            *reinterpret_cast<uint2 *>(f16 + part + r * ldd + c) = *reinterpret_cast<const uint2 *>(y[1]);
        }
#pragma unroll
        for (int k = 0; k < BF; ++k) {
            __nv_bfloat16 y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const bool fine = fabsf(x[i]) < kInf;
                y[i] = __float2bfloat16_rn(x[i]);
                if (fine && __hisinf(y[i])) y[i] = __float2bfloat16_rz(x[i]);
                x[i] = fine ? x[i] - __bfloat162float(y[i]) : 0.0f;
            }
            *reinterpret_cast<uint2 *>(bf + k * part + r * ldd + c) = *reinterpret_cast<const uint2 *>(y);
        }
    }
}

template <int BF>
cudaError_t launch_split(const float *src, long long ld, int rows, int cols, __half *f16, float *unscale, int padded,
                         float *most, float *clear, __nv_bfloat16 *bf, long long ldd, bool dependent,
                         cudaStream_t stream)
{
    const bool vec = (reinterpret_cast<uintptr_t>(src) & 15) == 0 && ld % 4 == 0;
    return launch_kernel(dependent, vec ? vocab_split_kernel<BF, true> : vocab_split_kernel<BF, false>, dim3((padded + 7) / 8),
                         dim3(32, 8), 0, stream, src, ld, rows, cols, f16, unscale, padded, most, clear, bf, ldd);
}

template <int CTAS, bool F16>
cudaError_t set_attributes()
{
    cudaFuncAttributes a;
    const cudaError_t e = cudaFuncGetAttributes(&a, vocab_kernel<CTAS, F16>);
    if (e != cudaSuccess) return e;
    if (a.numRegs < REGS_LAUNCH) return cudaErrorInvalidConfiguration;  // the exchange of registers could not end
    return cudaFuncSetAttribute(vocab_kernel<CTAS, F16>, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<CTAS>::SMEM);
}

}  // namespace

cudaError_t vocab_set_attributes()
{
    for (cudaError_t e : {set_attributes<1, false>(), set_attributes<2, false>(), set_attributes<1, true>(),
                          set_attributes<2, true>()})
        if (e != cudaSuccess) return e;
    return cudaSuccess;
}

int vocab_max_pairs()
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = Shape<2>::SMEM;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int clusters = 0;
    if (cudaOccupancyMaxActiveClusters(&clusters, vocab_kernel<2, true>, &cfg) != cudaSuccess) {
        (void)cudaGetLastError();
        return 0;
    }
    return clusters;
}

cudaError_t launch_vocab_tiles(const VocabMaps &maps, const VocabTileParams &p, int ctas, int workers, bool dependent,
                               cudaStream_t stream)
{
    const int n = static_cast<int>(std::min<long long>(static_cast<long long>(p.dh_items) + p.dw_items + p.z_items, workers));
    if (ctas == 2)
        return launch_kernel_cluster(dependent, 2, p.f16 ? vocab_kernel<2, true> : vocab_kernel<2, false>, dim3(2 * n),
                                     dim3(THREADS), Shape<2>::SMEM, stream,
                                     maps, p);
    return launch_kernel(dependent, p.f16 ? vocab_kernel<1, true> : vocab_kernel<1, false>, dim3(n), dim3(THREADS),
                         Shape<1>::SMEM, stream, maps, p);
}

cudaError_t launch_vocab_copy(const void *src, long long ld, int rows, int cols, void *dst, long long ldd, bool dependent,
                              cudaStream_t stream)
{
    return launch_kernel(dependent, vocab_copy_kernel, dim3((rows + 3) / 4), dim3(64, 4), 0, stream,
                         static_cast<const __nv_bfloat16 *>(src), ld, rows, cols, static_cast<__nv_bfloat16 *>(dst), ldd);
}

cudaError_t launch_vocab_split(const void *src, long long ld, int rows, int cols, void *f16, float *unscale, int padded,
                               float *most, float *clear, void *bf, int parts, long long ldd, bool dependent,
                               cudaStream_t stream)
{
    const float *s = static_cast<const float *>(src);
    __half *f = static_cast<__half *>(f16);
    __nv_bfloat16 *b = static_cast<__nv_bfloat16 *>(bf);
    if (bf == nullptr)
        return launch_split<0>(s, ld, rows, cols, f, unscale, padded, most, clear, b, ldd, dependent, stream);
    return parts == 2 ? launch_split<2>(s, ld, rows, cols, f, unscale, padded, most, clear, b, ldd, dependent, stream)
                      : launch_split<3>(s, ld, rows, cols, f, unscale, padded, most, clear, b, ldd, dependent, stream);
}

}  // namespace sgemm_impl
