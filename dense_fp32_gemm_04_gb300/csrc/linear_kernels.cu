// Tile kernel of the linear layers on the 5th-generation tensor cores, 128 x 256 tiles
// per CTA or 256 x 256 tiles per CTA pair (Y's may be narrower), 16-bit operands, FP32 accumulation:
//   Y  = act(X W^T + b) + R   A = X (K-major), B = W (K-major)
//   dX = dZ W + beta dX       A = dZ (K-major), B = W (MN-major)
//   dW = dZ^T X + beta dW     A = dZ (MN-major), B = X (MN-major)
// Two forms of it. Persistent: as many CTAs or pairs as the machine holds, each taking
// tiles in turn, two accumulators, so the epilogue of a tile runs beside the products
// of the next; dX and dW in one launch, so one's tiles fill the last round of the other's. Split: where there are
// too few tiles for that, a cluster of 2 to 8 CTAs shares a tile, each a part of its K range, and adds the parts
// in distributed shared memory, in rank order; one launch and no workspace.
//
// FP32 operands are sums of two float16 parts (22 bits) of rows or columns scaled by
// powers of two, a product of them three products of parts, small ones first: the
// same loop over more slabs. What is scaled is never the sum's index: X and W by rows
// for Y; for dX dZ by rows, with W's row factors put into it first; for dW dZ and X
// by columns. An element far below its row's or column's largest has fewer bits: it is
// held to 2^-39 of that one, which shows where the other operand is 0, or as small, in
// the largest one's place. (Three bfloat16 parts, which need no scaling, took six products: a training
// step of 2047 x 3001 x 1531 438 us.) The tensor core truncates its accumulator and the
// products next to it at every K = 16 step (8e-6 of a sum of alike terms at K = 4096, all
// toward zero), which FP32 results would show: their K range is cut into segments that
// the epilogue warps add in registers, rounded to nearest, while the next ones run.
// Results that are rounded to bfloat16 are one segment: K = 65536 loses 3.4e-4, a tenth
// of that rounding.
//
// Warps of a CTA (five warpgroups): 0 TMA producer, 1 MMA issuer (rank 0 of a pair),
// 2 and 3 idle; 4..19 epilogue: warp w reads TMEM lanes 32 (w % 4) and the columns of
// its side (w / 4 - 1) of the accumulator, a part of one row per thread: 64 columns, which is what the
// FP32 forms' segments add up to in registers. (Eight warps of 128 columns and a sixth ring stage: 2047 x 3001 x
// 1531 in FP32 with activation and residual 182 us, 136 with sixteen; 512 x 4096 x 4096 in bfloat16, split, 29 and 24;
// 2048 x 8192 x 2048 in bfloat16, whole, 52.0 and 51.4.) Ring and accumulator
// barriers: full / empty per stage, acc_full / acc_empty per accumulator, all waits
// bounded. The epilogue works on 64 bytes of columns at a time: accumulator to
// registers, bias, activation, slope, what is added; results leave through swizzled
// staging and TMA stores in the background (rows off 16-byte boundaries: element by element, along rows).
//
// What bounds whole tiles: an SM takes its operands from the L2 at 32 KB per 512 cycles of the tensor core, all that its
// port gives, so what a tile's epilogue moves beside them adds to its time (2048 x 8192 x 2048, four rounds: 50 us, 6 more
// for GELU, 10 for slopes, a second result of its size). In FP32 the tensor cores wait for a tile's epilogue, whose sums are in
// registers: 2047 x 3001 x 1531 with residual and slopes at odd strides 81 us (93 with its operands' parts), two tiles of 20 us a pair and
// their epilogues. In bfloat16 4096 x 16384 x 4096 takes 315 us from a cool start, 1.75 PFLOP/s, and 356 at the power limit.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "device_ptx.cuh"
#include "linear_act.cuh"
#include "linear_internal.h"
#include "sgemm_internal.h"
#include "tcgen05_ptx.cuh"

namespace sgemm_impl {
namespace {

using namespace sgemm_dev;

constexpr int kTimeoutCode = 5 << 16;
constexpr int kLayoutCode = 7 << 16;
constexpr int BK = kLinearBK;  // 64 bfloat16 = 128 bytes, one swizzle row
constexpr int MMA_K = 16;
constexpr int BOX_BYTES = 64 * 64 * 2;  // every copy: 64 rows of 64 elements
constexpr uint32_t TMEM_COLS = 512;
constexpr int STRIP = 64;                   // bytes of columns that the epilogue works on at a time
constexpr int kStripBytes = 32 * STRIP;     // of a warp's 32 rows
constexpr int kWarpStaging = 2 * kStripBytes;  // the result's strip twice, or the result's and the slope's

// A form of the kernel. CTAS: per tile of up to 256 columns, or 1 and tiles of BN = 128 columns (split ones). A split tile is not
// staged, but lies where the ring was.
template <int CTAS_, int BN_, bool F32, bool SPLIT_>
struct Shape {
    typedef typename std::conditional<F32, float, __nv_bfloat16>::type E;
    static constexpr bool PAIR = CTAS_ == 2, SPLIT = SPLIT_, SUMS = F32 || SPLIT;  // SUMS: a tile's segments meet in registers
    static constexpr int CTAS = CTAS_, BM = 128 * CTAS, BN = BN_;
    static constexpr int CTA_N = BN / CTAS;  // columns of B staged per CTA
    static constexpr int EPI_WARPS = 16, THREADS = 128 + 32 * EPI_WARPS;
    static constexpr int COLS = BN / (EPI_WARPS / 4);  // accumulator columns of one epilogue thread
    static constexpr int STAGES = SPLIT ? (BN == 128 ? 6 : 4) : CTAS == 2 ? 5 : 3;
    static constexpr int TILE_STRIDE = BN + 4;  // floats of a row of a split tile: 16 bytes more than its columns, so that
                                                // rows next to each other start in other banks
    static constexpr int A_BYTES = 128 * BK * 2;
    static constexpr int B_BYTES = CTA_N * BK * 2;
    static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
    static constexpr int STAGING_BYTES = SPLIT ? 0 : EPI_WARPS * kWarpStaging;
    static constexpr int SMEM = 1024 + STAGES * STAGE_BYTES + STAGING_BYTES + 512;
    // Registers per thread: at launch (the most that so many threads can have), and after the warpgroups' exchange.
    static constexpr int REGS_LAUNCH = 96, REGS_ISSUE = 56, REGS_EPILOGUE = 104;
    static_assert(REGS_ISSUE + EPI_WARPS / 4 * REGS_EPILOGUE <= THREADS / 128 * REGS_LAUNCH,
                  "an exchange above the launch's registers never ends");
    static_assert(!SPLIT || CTAS == 1, "a cluster is a pair or shares a tile");
    static_assert(SPLIT || BN == kLinearBN, "whole tiles have up to 256 columns");
    static_assert(SMEM <= 227 * 1024, "shared memory per CTA");
    static_assert(!SPLIT || 128 * TILE_STRIDE * 4 <= STAGES * STAGE_BYTES, "a split tile lies where the ring was");
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
__device__ __forceinline__ void raise_abort(Bars<STAGES> *b, const LinearParams &p, int code)
{
    volatile int *f = &b->abort_flag;
    if (!*f) {
        *f = 1;
        report_status(p.status, code);
    }
}

// One tile of a launch: of product t, rows from m0, columns from n0, k-blocks [kb0, kb1).
struct Item {
    int t, m0, n0, kb0, kb1;
};

// Tile u of a product: in groups of 16 tile rows, along them first: they share their columns of B, and the group's rows
// of A stay in the L2.
__device__ __forceinline__ void place_tile(const LinearProduct &t, int u, int bm, int bn, Item &w)
{
    constexpr int GROUP = 16;
    const int group = u / (GROUP * t.tiles_n), rows = min(GROUP, t.tiles_m - group * GROUP), r = u - group * GROUP * t.tiles_n;
    w.m0 = (group * GROUP + r % rows) * bm;
    w.n0 = r / rows * bn;
}

// Item i of a worker. Persistent: first its tiles of t[0], the longer ones, dealt in turn; workers that get one fewer take
// `extra` of t[1] in its place; then the others in turn. Split: one tile a cluster, a part of its K range each.
template <bool SPLIT>
__device__ __forceinline__ bool item_at(const LinearParams &p, int i, int worker, int workers, int bm, int bn, int rank, Item &w)
{
    const int a = p.t[0].tiles_m * p.t[0].tiles_n;
    int u;
    if constexpr (SPLIT) {
        if (i > 0) return false;
        w.t = worker >= a;
        u = worker - (w.t ? a : 0);
    } else {
        const int turns = a / workers, rem = a - turns * workers, mine = turns + (worker < rem ? 1 : 0);
        if (i < mine) {
            w.t = 0;
            u = worker + i * workers;
        } else {
            i -= mine;
            const int few = workers - rem;  // workers with one tile fewer (all where rem is 0: then extra is 0)
            w.t = 1;
            if (worker >= rem && i < p.extra) {
                u = worker - rem + i * few;
            } else {
                if (worker >= rem) i -= p.extra;
                u = p.extra * few + (worker >= rem ? worker - rem : worker + few) + i * workers;
            }
        }
    }
    if (w.t >= p.products_of_launch) return false;
    const LinearProduct &t = p.t[w.t];
    if (u >= t.tiles_m * t.tiles_n) return false;
    place_tile(t, u, bm, bn, w);
    w.kb0 = 0;
    w.kb1 = t.kblocks;
    if constexpr (SPLIT) {
        w.kb0 = static_cast<int>(static_cast<long long>(t.kblocks) * rank / p.splits);
        w.kb1 = static_cast<int>(static_cast<long long>(t.kblocks) * (rank + 1) / p.splits);
    }
    return true;
}

// Parts of A and B in product i of three: low high, high low, high high; bfloat16 operands have the last one.
__device__ __forceinline__ int part_a(int i) { return i == 0; }
__device__ __forceinline__ int part_b(int i) { return i == 1; }

__device__ __forceinline__ void sts128(uint32_t addr, const uint32_t (&v)[4])
{
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3])
                 : "memory");
}

__device__ __forceinline__ void lds128(uint32_t addr, uint32_t (&v)[4])
{
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(addr) : "memory");
}

// Wait until at most N of this thread's bulk groups still read shared memory.
template <int N>
__device__ __forceinline__ void bulk_wait_read_but()
{
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}

// ---------------------------------------------------------------------------
// Epilogue. A strip: 32 rows of STRIP bytes, row r's 16-byte chunk j at j ^ (r / 2 % 4), the 64-byte swizzle.

template <typename E>
constexpr int kStripCols = STRIP / static_cast<int>(sizeof(E));

__device__ __forceinline__ uint32_t chunk_at(uint32_t strip, int row, int j) { return strip + row * STRIP + ((j ^ (row >> 1 & 3)) << 4); }

// Element e (of T) of a strip's row.
template <typename T>
__device__ __forceinline__ T *element_at(unsigned char *strip, int row, int e)
{
    constexpr int PER = 16 / sizeof(T);
    return reinterpret_cast<T *>(strip + row * STRIP + (((e / PER) ^ (row >> 1 & 3)) << 4)) + e % PER;
}

// A strip of rows that 16-byte accesses cannot take: neighbouring lanes take neighbouring elements of a row, ROWS rows at a
// time, COUNT times.
template <typename T>
struct Ragged {
    static constexpr int C = STRIP / sizeof(T), ROWS = 32 / C > 0 ? 32 / C : 1, COUNT = 32 / ROWS;

    // (a whole strip has no branch at every element)
    static __device__ __forceinline__ void fetch(T (&v)[COUNT], const T *m, long long ld, int rows, int cols, int lane)
    {
        const T *from = m + lane / C * ld + lane % C;  // (plain loads: what is added may be the result's own rows)
        const long long step = ROWS * ld;
        if (rows >= 32 && cols >= C) {
#pragma unroll
            for (int i = 0; i < COUNT; ++i, from += step) v[i] = *from;
        } else {
#pragma unroll
            for (int i = 0; i < COUNT; ++i, from += step) v[i] = i * ROWS + lane / C < rows && lane % C < cols ? *from : T{};
        }
    }
    static __device__ __forceinline__ void put(const T (&v)[COUNT], unsigned char *strip, int lane)
    {
#pragma unroll
        for (int i = 0; i < COUNT; ++i) *element_at<T>(strip, i * ROWS + lane / C, lane % C) = v[i];
    }
    static __device__ __forceinline__ void store(unsigned char *strip, T *m, long long ld, int rows, int cols, int lane)
    {
        T *to = m + lane / C * ld + lane % C;
        const long long step = ROWS * ld;
        if (rows >= 32 && cols >= C) {
#pragma unroll
            for (int i = 0; i < COUNT; ++i, to += step) *to = *element_at<T>(strip, i * ROWS + lane / C, lane % C);
        } else {
#pragma unroll
            for (int i = 0; i < COUNT; ++i, to += step) {
                const T x = *element_at<T>(strip, i * ROWS + lane / C, lane % C);
                if (i * ROWS + lane / C < rows && lane % C < cols) *to = x;
            }
        }
    }
};

template <typename E>
__device__ __forceinline__ void open16(const uint32_t (&v)[4], float *x)
{
    if constexpr (sizeof(E) == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = __uint_as_float(v[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(v[i] << 16);
            x[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
        }
    }
}

template <typename E>
__device__ __forceinline__ void close16(const float *x, uint32_t (&v)[4])
{
    if constexpr (sizeof(E) == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __float_as_uint(x[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 y = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            v[i] = *reinterpret_cast<const uint32_t *>(&y);
        }
    }
}

// 16 bytes of slopes.
template <typename E>
__device__ __forceinline__ void close_slope(const float *s, uint32_t (&v)[4])
{
    if constexpr (sizeof(E) == 4) {
        close16<float>(s, v);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[i] = static_cast<uint16_t>(slope_close(s[2 * i])) | static_cast<uint32_t>(static_cast<uint16_t>(slope_close(s[2 * i + 1]))) << 16;
    }
}

// N columns of this thread's TMEM lane.
template <int N>
__device__ __forceinline__ void tmem_load(uint32_t taddr, float (&v)[N])
{
    if constexpr (N == 8)
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
                     "tcgen05.wait::ld.sync.aligned;"
                     : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
                     : "r"(taddr)
                     : "memory");
    else
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];\n\t"
                     "tcgen05.wait::ld.sync.aligned;"
                     : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
                     : "r"(taddr)
                     : "memory");
}

// A 16-byte chunk of a strip's row: y = act(v) + gamma * what stands there (if add), act'(v) at `slopes`.
template <typename E>
constexpr int kChunk = 16 / static_cast<int>(sizeof(E));

template <typename E, int ACT, bool SLOPE>
__device__ __forceinline__ void make_chunk(const float (&v)[kChunk<E>], bool add, float gamma, uint32_t to, uint32_t slopes)
{
    constexpr int PER = kChunk<E>;
    float y[PER], s[PER];
    uint32_t packed[4];
#pragma unroll
    for (int i = 0; i < PER; ++i) activate<ACT, sizeof(E) == 4>(v[i], y[i], s[i]);
    if (add) {
        float r[PER];
        lds128(to, packed);
        open16<E>(packed, r);
#pragma unroll
        for (int i = 0; i < PER; ++i) y[i] = fmaf(gamma, r[i], y[i]);
    }
    close16<E>(y, packed);
    sts128(to, packed);
    if constexpr (SLOPE) {
        close_slope<E>(s, packed);
        sts128(slopes, packed);
    }
}

template <typename E, bool SLOPE>
__device__ __forceinline__ void make_chunk_by(int act, const float (&v)[kChunk<E>], bool add, float gamma, uint32_t to, uint32_t slopes)
{
    switch (act) {
    case SGEMM_ACT_RELU: make_chunk<E, SGEMM_ACT_RELU, SLOPE>(v, add, gamma, to, slopes); break;
    case SGEMM_ACT_GELU: make_chunk<E, SGEMM_ACT_GELU, SLOPE>(v, add, gamma, to, slopes); break;
    case SGEMM_ACT_GELU_TANH: make_chunk<E, SGEMM_ACT_GELU_TANH, SLOPE>(v, add, gamma, to, slopes); break;
    case SGEMM_ACT_SILU: make_chunk<E, SGEMM_ACT_SILU, SLOPE>(v, add, gamma, to, slopes); break;
    default: make_chunk<E, SGEMM_ACT_NONE, SLOPE>(v, add, gamma, to, slopes);
    }
}

// Bias of a chunk's columns, `cols` of which exist. vec: it starts on a 16-byte boundary.
template <typename E>
__device__ __forceinline__ void add_bias(const E *bias, bool vec, int cols, float (&v)[kChunk<E>])
{
    constexpr int PER = kChunk<E>;
    if (vec && cols >= PER) {
        const uint4 b = __ldg(reinterpret_cast<const uint4 *>(bias));
        const uint32_t w[4] = {b.x, b.y, b.z, b.w};
        float x[PER];
        open16<E>(w, x);
#pragma unroll
        for (int i = 0; i < PER; ++i) v[i] += x[i];
    } else {
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (i < cols) v[i] += static_cast<float>(__ldg(bias + i));
    }
}

// What a tile in FP32 multiplies and adds, asked for before its sums are there: the root of a row's factor, and of a warp's (up to
// 64) columns each lane's two, of factors' roots and bias. (With the factors and the bias loaded where they are used, a tile of 2048 x 2432
// x 1536 left in 14 us, and its products take 20.)
struct Scales {
    float row, col[2], bias[2];
};

// (plain loads of factors: the call's previous kernels wrote them)
__device__ __forceinline__ void fetch_scales(const LinearProduct &q, const float *bias, int row, int c0, int width, int lane, Scales &s)
{
    s.row = row + lane < q.rows ? q.row_unscale[row + lane] : 1.0f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int c = 32 * h + lane;
        const bool there = c < width && c0 + c < q.cols;
        s.col[h] = there && q.col_unscale != nullptr ? q.col_unscale[c0 + c] : 1.0f;
        s.bias[h] = there && bias != nullptr ? __ldg(bias + c0 + c) : 0.0f;
    }
}

// Rows of what will be added, on their way to the L2 while the products are made.
template <typename E>
__device__ __forceinline__ void ask_for_added(const LinearProduct &q, int row, int c0, int width, int lane)
{
    const int cols = min(width, q.cols - c0);
    if (q.add == nullptr || cols <= 0 || row + lane >= q.rows) return;
    const E *a = static_cast<const E *>(q.add) + static_cast<long long>(row + lane) * q.ldadd + c0;
    for (int c = 0; c < cols; c += 128 / static_cast<int>(sizeof(E))) asm volatile("prefetch.global.L2 [%0];" ::"l"(a + c));
    asm volatile("prefetch.global.L2 [%0];" ::"l"(a + cols - 1));
}

// 32 rows x `width` columns of a tile from the accumulator at `t` or the sums acc: rows from `row`, columns from c0 of the product.
template <class Sh>
__device__ __forceinline__ void leave_tile(const LinearParams &p, const LinearMaps &maps, const LinearProduct &q, int which,
                                           uint32_t t, float (&acc)[Sh::SUMS ? Sh::COLS : 1], const Scales &scales, unsigned char *area, int lane,
                                           int row, int c0, int width, int &strips)
{
    typedef typename Sh::E E;
    typedef typename std::conditional<sizeof(E) == 4, float, short>::type S;
    constexpr int C = kStripCols<E>;
    const uint32_t stg = smem_addr(area);
    const bool first = q.kind == kLinearY, slope = first && p.slope != nullptr;
    const int act = first ? p.act : SGEMM_ACT_NONE;
    const int rows = q.rows - row;  // that exist
    // What is added to a strip: pieces of 16 bytes, four lanes to a row, or (FP32) ragged elements, fetched while the strip before it
    // is made, or ragged ones when it is. (With a row to a lane, 2048 x 8192 x 2048 in bfloat16 with a residual 57.0 us for 52.9.)
    uint32_t next[16];
    static_assert(sizeof(E) == 2 || Ragged<E>::COUNT == 16, "as many as a row's strip has");
    auto whole = [&](int c) { return q.add_tma && q.cols - c >= C; };
    auto added = [&](int c) { return static_cast<const E *>(q.add) + static_cast<long long>(row) * q.ldadd + c; };
    auto fetch = [&](int c) {
        if (q.add == nullptr) return;
        if (whole(c)) {  // four lanes to a row's 64 bytes
            const E *a = added(c) + lane % 4 * (16 / sizeof(E));
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = 8 * j + lane / 4;
                const uint4 x = r < rows ? *reinterpret_cast<const uint4 *>(a + r * q.ldadd) : make_uint4(0, 0, 0, 0);
                next[4 * j] = x.x, next[4 * j + 1] = x.y, next[4 * j + 2] = x.z, next[4 * j + 3] = x.w;
            }
        } else if constexpr (sizeof(E) == 4) {
            Ragged<uint32_t>::fetch(next, reinterpret_cast<const uint32_t *>(added(c)), q.ldadd, rows, q.cols - c, lane);
        }
    };
    if (rows <= 0 || width <= 0) return;
    static_assert(sizeof(E) == 2 || (C == 16 && Sh::COLS <= 64), "two columns of scales a lane");
    const E *bias = first ? static_cast<const E *>(p.bias) : nullptr;
    const bool bias_vec = (reinterpret_cast<uintptr_t>(bias) & 15) == 0;
    fetch(c0);
#pragma unroll 1
    for (int cb = 0; cb * C < width; ++cb) {
        const int c = c0 + cb * C, cols = q.cols - c;
        if (cols <= 0) break;
        const int buf = slope ? 0 : strips++ & 1;
        const uint32_t to = stg + buf * kStripBytes;
        if (lane == 0) {  // the staging is free again
            if (slope)
                bulk_wait_read_but<0>();
            else
                bulk_wait_read_but<1>();
        }
        __syncwarp();
        if (q.add != nullptr) {  // where the result will stand
            if (whole(c)) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t x[4] = {next[4 * j], next[4 * j + 1], next[4 * j + 2], next[4 * j + 3]};
                    sts128(chunk_at(to, 8 * j + lane / 4, lane % 4), x);
                }
                __syncwarp();
                if ((cb + 1) * C < width) fetch(c + C);
            } else if constexpr (sizeof(E) == 4) {
                Ragged<uint32_t>::put(next, area + buf * kStripBytes, lane);
                __syncwarp();
                if ((cb + 1) * C < width) fetch(c + C);
            } else {
                E ragged[Ragged<E>::COUNT];
                Ragged<E>::fetch(ragged, added(c), q.ldadd, rows, cols, lane);
                Ragged<E>::put(ragged, area + buf * kStripBytes, lane);
                __syncwarp();
            }
        }
        // The chunks' columns: from the accumulator, or FP32 sums from registers, from which the accumulator has long been
        // given back. FP32's activations are long, so their loops are not unrolled; what a turn takes lies in the first
        // registers, and the others move up.
        constexpr int PER = kChunk<E>, UNROLL = sizeof(E) == 4 ? 1 : 4;
        float sums[4 * PER];
        if constexpr (Sh::SUMS) {
#pragma unroll
            for (int i = 0; i < 4 * PER; ++i) sums[i] = acc[i];
#pragma unroll
            for (int i = 0; i < Sh::COLS - 4 * PER; ++i) acc[i] = acc[i + 4 * PER];
        }
        auto chunk = [&](int j, float (&v)[PER], int act) {
            if constexpr (sizeof(E) == 4) {  // what undoes the scaling of the operands' rows and columns, and the bias
                const float col = cb < 2 ? scales.col[0] : scales.col[1], b = cb < 2 ? scales.bias[0] : scales.bias[1];
                const int from = (cb & 1) * C + j * PER;
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    const float root = scales.row * __shfl_sync(0xffffffffu, col, from + i);
                    v[i] = fmaf(v[i] * root, root, __shfl_sync(0xffffffffu, b, from + i));
                }
            }
            if (sizeof(E) == 2 && bias != nullptr) add_bias(bias + c + j * PER, bias_vec, cols - j * PER, v);
            const uint32_t at = chunk_at(to, lane, j);
            if (slope)
                make_chunk_by<E, true>(act, v, q.add != nullptr, q.gamma, at, chunk_at(stg + kStripBytes, lane, j));
            else
                make_chunk_by<E, false>(act, v, q.add != nullptr, q.gamma, at, 0);
        };
        if (Sh::SUMS && act == SGEMM_ACT_NONE && !slope) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float v[PER];
#pragma unroll
                for (int i = 0; i < PER; ++i) v[i] = sums[j * PER + i];
                chunk(j, v, SGEMM_ACT_NONE);
            }
        } else {
#pragma unroll UNROLL
            for (int j = 0; j < 4; ++j) {
                float v[PER];
                if constexpr (Sh::SUMS) {
#pragma unroll
                    for (int i = 0; i < PER; ++i) v[i] = sums[i];
#pragma unroll
                    for (int i = 0; i < 3 * PER; ++i) sums[i] = sums[i + PER];
                } else {
                    tmem_load(t + cb * C + j * PER, v);
                }
                chunk(j, v, act);
            }
        }
        if (!index_ok(row < q.rows && c < q.cols, p.status, kWhereIdxLinear)) break;
        // a TMA store writes whole 16-byte pieces: a row that ends inside one would lose what follows it
        const bool pieces = cols >= C || cols * sizeof(E) % 16 == 0, out_tma = q.out_tma && pieces;
        const bool slope_tma = slope && p.slope_tma && pieces;
        if (out_tma || slope_tma) fence_proxy_async();
        __syncwarp();
        if (out_tma) {
            if (lane == 0) tma_store_3d(&maps.out[which], to, c, row, 0);
        } else {
            Ragged<E>::store(area + buf * kStripBytes, static_cast<E *>(q.out) + row * q.ldo + c, q.ldo, rows, cols, lane);
        }
        if (slope) {
            if (slope_tma) {
                if (lane == 0) tma_store_3d(&maps.slope, stg + kStripBytes, c, row, 0);
            } else {
                Ragged<S>::store(area + kStripBytes, static_cast<S *>(p.slope) + row * p.lds + c, p.lds, rows, cols, lane);
            }
        }
        if (lane == 0) bulk_commit();
        __syncwarp();
    }
}

// Four neighbouring elements of a result, from the sum of a split tile's parts.
template <typename E>
__device__ __forceinline__ void leave_four(const LinearParams &p, const LinearProduct &q, int row, int c, float (&x)[4])
{
    typedef typename std::conditional<sizeof(E) == 4, float, short>::type S;
    const bool first = q.kind == kLinearY, slope = first && p.slope != nullptr;
    const int act = first ? p.act : SGEMM_ACT_NONE, n = min(4, q.cols - c);
    if (!index_ok(row < q.rows && n > 0, p.status, kWhereIdxLinear)) return;
    typedef typename std::conditional<sizeof(E) == 4, uint4, uint2>::type Four;  // four elements as one access
    if constexpr (sizeof(E) == 4) {
        const float f = q.row_unscale[row];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float root = f * (q.col_unscale != nullptr && i < n ? q.col_unscale[c + i] : 1.0f);
            x[i] = x[i] * root * root;
        }
    }
    E b[4] = {}, r[4] = {};
    if (first && p.bias != nullptr) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < n) b[i] = __ldg(static_cast<const E *>(p.bias) + c + i);
    }
    if (q.add != nullptr) {
        const E *a = static_cast<const E *>(q.add) + row * q.ldadd + c;
        if (q.add_vec && n == 4) {
            const Four f = *reinterpret_cast<const Four *>(a);
            memcpy(r, &f, sizeof(f));
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < n) r[i] = a[i];
        }
    }
    E y[4];
    S s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float v, d;
        activate_by<sizeof(E) == 4>(act, x[i] + static_cast<float>(b[i]), v, d);
        y[i] = static_cast<E>(fmaf(q.gamma, static_cast<float>(r[i]), v));
        if constexpr (sizeof(E) == 4)
            s[i] = d;
        else
            s[i] = slope_close(d);
    }
    E *o = static_cast<E *>(q.out) + row * q.ldo + c;
    if (q.out_vec && n == 4) {
        Four f;
        memcpy(&f, y, sizeof(f));
        *reinterpret_cast<Four *>(o) = f;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < n) o[i] = y[i];
    }
    if (!slope) return;
    S *so = static_cast<S *>(p.slope) + row * p.lds + c;
    if (p.slope_vec && n == 4) {
        Four f;
        memcpy(&f, s, sizeof(f));
        *reinterpret_cast<Four *>(so) = f;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < n) so[i] = s[i];
    }
}

// ---------------------------------------------------------------------------

// Producer thread: this CTA's part of each stage, in boxes of 64 rows x 64 elements.
template <class S>
__device__ __forceinline__ void produce(const LinearParams &p, Bars<S::STAGES> *bars, uint32_t a_base,
                                        uint32_t b_base, const LinearMaps &maps, uint32_t rank, int worker, int workers)
{
    constexpr int STAGES = S::STAGES;
    constexpr bool PAIR = S::PAIR;
    volatile int *abort_flag = &bars->abort_flag;
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    Item w;
    for (int i = 0; ok && item_at<S::SPLIT>(p, i, worker, workers, S::BM, p.bn, rank, w); ++i) {
        const int kind = p.t[w.t].kind;
        const CUtensorMap *ta = &maps.a[w.t], *tb = &maps.b[w.t];
        const bool a_k = kind != kLinearDw, b_k = kind == kLinearY;  // K-major: K along the map's rows
        const int half = PAIR ? static_cast<int>(rank) : 0, cta_n = p.bn / S::CTAS;
        const int a_r = w.m0 + half * 128, b_r = w.n0 + half * cta_n;
        // Y's columns of B come in one box of as many rows as a CTA has of the tile, others in boxes of 64
        const uint32_t bytes = S::CTAS * (S::A_BYTES + static_cast<uint32_t>(cta_n) * BK * 2);
        for (int s0 = w.kb0; ok && s0 < w.kb1; s0 += p.segment) {
            const int s1 = min(s0 + p.segment, w.kb1);
            for (int pr = 3 - p.products; ok && pr < 3; ++pr) {
                const int pa = part_a(pr), pb = part_b(pr);
                for (int kb = s0; kb < s1; ++kb) {
                    if (!mbar_wait_quiet<false>(smem_addr(&bars->empty[stage]), phase ^ 1u, abort_flag, p.timeout_ns)) {
                        raise_abort(bars, p, kTimeoutCode | kWhereProducerEmpty);
                        ok = false;
                        break;
                    }
                    const uint32_t a_dst = a_base + stage * S::A_BYTES;
                    const uint32_t b_dst = b_base + stage * S::B_BYTES;
                    if (!PAIR || rank == 0) mbar_arrive_expect_tx(smem_addr(&bars->full[stage]), bytes);
                    uint32_t full = smem_addr(&bars->full[stage]);
                    if constexpr (PAIR) full = mapa_shared(full, 0);  // rank 0's barrier
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int x = a_k ? kb * BK : a_r + 64 * j, y = a_k ? a_r + 64 * j : kb * BK;
                        if constexpr (PAIR)
                            tma_load_3d_pair(a_dst + j * BOX_BYTES, ta, full, x, y, pa);
                        else
                            tma_load_3d(a_dst + j * BOX_BYTES, ta, full, x, y, pa);
                    }
                    for (int j = 0; j < (b_k ? 1 : S::CTA_N / 64); ++j) {
                        const int x = b_k ? kb * BK : b_r + 64 * j, y = b_k ? b_r : kb * BK;
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
    // Drain: every issued copy has landed (rank 0's barriers count both CTAs'), and unless aborted the MMAs that read it
    // have committed.
    for (int s = 0; s < STAGES; ++s) {
        const int rec = bars->issued[s];
        if (!(rec & 2)) continue;
        const uint32_t par = static_cast<uint32_t>(rec & 1);
        if ((!PAIR || rank == 0) && !mbar_wait_quiet<true>(smem_addr(&bars->full[s]), par, nullptr, p.timeout_ns)) {
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
template <class S>
__device__ __forceinline__ void issue(const LinearParams &p, Bars<S::STAGES> *bars, uint32_t a_base,
                                      uint32_t b_base, uint32_t tmem, uint32_t rank, int worker, int workers)
{
    constexpr int STAGES = S::STAGES;
    constexpr bool PAIR = S::PAIR;
    volatile int *abort_flag = &bars->abort_flag;
    int stage = 0;
    uint32_t phase = 0;
    int it = 0;  // segments so far
    bool ok = true;
    Item w;
    for (int i = 0; ok && item_at<S::SPLIT>(p, i, worker, workers, S::BM, p.bn, rank, w); ++i) {
        const int kind = p.t[w.t].kind;
        const bool a_mn = kind == kLinearDw, b_mn = kind != kLinearY;
        const uint32_t idesc = idesc_16(S::BM, p.bn, a_mn, b_mn, p.dtype == SGEMM_DTYPE_F32);
        for (int s0 = w.kb0; ok && s0 < w.kb1; s0 += p.segment, ++it) {
            const int buf = it & 1;
            const uint32_t acc_phase = static_cast<uint32_t>(it >> 1) & 1u;
            if (!mbar_wait_quiet<true>(smem_addr(&bars->acc_empty[buf]), acc_phase ^ 1u, abort_flag, p.timeout_ns)) {
                raise_abort(bars, p, kTimeoutCode | kWhereAccum);
                ok = false;
                break;
            }
            tc_fence_after_sync();
            const uint32_t d_tmem = tmem + static_cast<uint32_t>(buf * S::BN);
            const int slabs = (min(s0 + p.segment, w.kb1) - s0) * p.products;
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

// Epilogue warp: the segments of a tile added up (FP32 operands, split tiles: in registers), the tile
// left as its product wants it, or as a part of a split tile in shared memory.
template <class S>
__device__ __forceinline__ void leave_tiles(const LinearParams &p, Bars<S::STAGES> *bars, unsigned char *ring,
                                            unsigned char *staging, const LinearMaps &maps, uint32_t tmem, uint32_t rank,
                                            int warp, int lane, int worker, int workers)
{
    constexpr bool PAIR = S::PAIR;
    constexpr int COLS = S::COLS;
    volatile int *abort_flag = &bars->abort_flag;
    const int quarter = warp & 3, side = (warp - 4) >> 2;
    unsigned char *area = staging + (warp - 4) * kWarpStaging;
    int it = 0, strips = 0;
    bool ok = true;
    Item w;
    auto release = [&](int buf) {
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) {
            if constexpr (PAIR)
                mbar_arrive_cluster(mapa_shared(smem_addr(&bars->acc_empty[buf]), 0));  // rank 0's
            else
                mbar_arrive(smem_addr(&bars->acc_empty[buf]));
        }
    };
    for (int i = 0; ok && item_at<S::SPLIT>(p, i, worker, workers, S::BM, p.bn, rank, w); ++i) {
        const LinearProduct &q = p.t[w.t];
        const int row = w.m0 + (PAIR ? static_cast<int>(rank) * 128 : 0) + quarter * 32;  // the warp's first
        // (FP32 in narrow tiles: strips dealt evenly, or one side's warps would have nothing and another's four)
        const int span = S::SUMS && !S::SPLIT ? (p.bn / 16 + 3) / 4 * 16 : COLS, c0 = w.n0 + side * span, width = min(span, p.bn - side * span);
        Scales scales;
        if constexpr (S::SUMS && !S::SPLIT)
            fetch_scales(q, q.kind == kLinearY ? static_cast<const float *>(p.bias) : nullptr, row, c0, width, lane, scales);
        if constexpr (!S::SPLIT) ask_for_added<typename S::E>(q, row, c0, width, lane);
        float acc[S::SUMS ? COLS : 1];
        if constexpr (S::SUMS) {
#pragma unroll
            for (int j = 0; j < COLS; ++j) acc[j] = 0.0f;
        }
        for (int s0 = w.kb0; s0 < w.kb1; s0 += p.segment, ++it) {
            const int buf = it & 1;
            ok = mbar_wait_quiet<true>(smem_addr(&bars->acc_full[buf]), static_cast<uint32_t>(it >> 1) & 1u, abort_flag,
                                       p.timeout_ns);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) {
                if (lane == 0) raise_abort(bars, p, kTimeoutCode | kWhereAccum);
                break;
            }
            tc_fence_after_sync();
            const uint32_t t = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(buf * S::BN + side * span);
            if constexpr (S::SUMS) {
#pragma unroll
                for (int cb = 0; cb < COLS / 16; ++cb) {
                    if (cb * 16 >= width) break;
                    uint32_t v[16];
                    tmem_ld_16(t + cb * 16, v);
                    tmem_wait_ld(v);
#pragma unroll
                    for (int j = 0; j < 16; j += 2) {
                        float *x = acc + cb * 16 + j;
                        unpack_f32x2(add_f32x2(pack_f32x2(x[0], x[1]), pack_f32x2(__uint_as_float(v[j]), __uint_as_float(v[j + 1]))), x[0],
                                     x[1]);
                    }
                }
            } else {
                leave_tile<S>(p, maps, q, w.t, t, acc, scales, area, lane, row, c0, width, strips);
            }
            release(buf);
        }
        if constexpr (S::SUMS && !S::SPLIT) {
            if (ok) leave_tile<S>(p, maps, q, w.t, 0, acc, scales, area, lane, row, c0, width, strips);
        }
        if constexpr (S::SPLIT) {
            if (!ok) break;
            // the ring is idle: its last copies have been read by products that have completed
            float *tile = reinterpret_cast<float *>(ring);
            const int r = quarter * 32 + lane;
            if (w.m0 + r < q.rows) {
#pragma unroll
                for (int j = 0; j < COLS; j += 4)
                    *reinterpret_cast<float4 *>(tile + r * S::TILE_STRIDE + side * COLS + j) =
                        make_float4(acc[j], acc[j + 1], acc[j + 2], acc[j + 3]);
            }
        }
    }
    if constexpr (!S::SPLIT) {
        if (lane == 0) bulk_wait();  // the staging is read and everything is written before the CTA ends
    }
}

// A split tile put together: the parts of all CTAs in rank order, four columns a thread at a time.
template <class S>
__device__ __forceinline__ void join_tile(const LinearParams &p, unsigned char *ring, uint32_t rank, int worker, int tid)
{
    Item w;
    if (!item_at<true>(p, 0, worker, 0, S::BM, p.bn, static_cast<int>(rank), w)) return;
    const LinearProduct &q = p.t[w.t];
    const int rows = min(128, q.rows - w.m0), groups = (min(p.bn, q.cols - w.n0) + 3) / 4;
    const uint32_t base = smem_addr(ring);
    for (int g = static_cast<int>(rank) * 32 * S::EPI_WARPS + tid; g < rows * groups; g += p.splits * 32 * S::EPI_WARPS) {
        const int r = g / groups, c = (g - r * groups) * 4;
        const uint32_t at = base + static_cast<uint32_t>(r * S::TILE_STRIDE + c) * 4;
        float x[4] = {};
        for (int s = 0; s < p.splits; ++s) {
            const float4 v = ld_shared_cluster_v4(mapa_shared(at, s));
            x[0] += v.x;
            x[1] += v.y;
            x[2] += v.z;
            x[3] += v.w;
        }
        leave_four<typename S::E>(p, q, w.m0 + r, w.n0 + c, x);
    }
}

template <class S>
__global__ void __launch_bounds__(S::THREADS, 1)
linear_kernel(const __grid_constant__ LinearMaps maps, const __grid_constant__ LinearParams p)
{
    constexpr int STAGES = S::STAGES;
    constexpr bool PAIR = S::PAIR, SPLIT = S::SPLIT;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    unsigned char *smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    const uint32_t a_base = smem_addr(smem);
    const uint32_t b_base = a_base + STAGES * S::A_BYTES;
    unsigned char *staging = smem + STAGES * S::STAGE_BYTES;
    Bars<STAGES> *bars = reinterpret_cast<Bars<STAGES> *>(staging + S::STAGING_BYTES);
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    if ((PAIR && cluster_size() != 2) || (SPLIT && static_cast<int>(cluster_size()) != p.splits)) {
        if (threadIdx.x == 0) report_status(p.status, kLayoutCode | (PAIR ? kWherePairLayout : kWhereLinearCluster));
        return;
    }
    const uint32_t rank = PAIR || SPLIT ? cluster_ctarank() : 0u;
    const int worker = PAIR || SPLIT ? static_cast<int>(cluster_id_x()) : static_cast<int>(blockIdx.x);
    const int workers = PAIR || SPLIT ? static_cast<int>(cluster_count_x()) : static_cast<int>(gridDim.x);

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(smem_addr(&bars->full[s]), 1);
            mbar_init(smem_addr(&bars->empty[s]), 1);
            bars->issued[s] = 0;
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_addr(&bars->acc_full[b]), 1);
            mbar_init(smem_addr(&bars->acc_empty[b]), S::EPI_WARPS * S::CTAS);
        }
        mbar_init(smem_addr(&bars->mma_done), 1);
        bars->abort_flag = 0;
        bars->ring_offset = a_base;
        fence_barrier_init();
        prefetch_tensormap(&maps.a[0]);
        prefetch_tensormap(&maps.b[0]);
        prefetch_tensormap(&maps.out[0]);
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
    if constexpr (PAIR || SPLIT) cluster_sync();  // the CTAs' barriers are initialised before any copy or arrive targets them
    tc_fence_after_sync();
    const uint32_t tmem = bars->tmem_base;
    bool same_layout = true;
    if constexpr (PAIR || SPLIT) {
        constexpr uint32_t kDescAddrMask = 0x3FFFFu;
        for (uint32_t r = 0; r < (PAIR ? 2u : static_cast<uint32_t>(p.splits)); ++r) {
            const uint32_t other = ld_shared_cluster_u32(mapa_shared(smem_addr(&bars->ring_offset), r));
            same_layout = same_layout && ((other ^ a_base) & kDescAddrMask) == 0;
        }
        if (!same_layout && threadIdx.x == 0) raise_abort(bars, p, kLayoutCode | (PAIR ? kWherePairLayout : kWhereLinearCluster));
    }

    pdl_wait();  // the call's previous kernel is complete
    // Where the CTAs' layouts differ all of them see it: no copies, no MMAs.
    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::REGS_ISSUE));
        if (same_layout && warp == 0 && lane == 0)
            produce<S>(p, bars, a_base, b_base, maps, rank, worker, workers);
        else if (same_layout && warp == 1 && lane == 0 && (!PAIR || rank == 0))
            issue<S>(p, bars, a_base, b_base, tmem, rank, worker, workers);
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(S::REGS_EPILOGUE));
        if (same_layout) leave_tiles<S>(p, bars, smem, staging, maps, tmem, rank, warp, lane, worker, workers);
    }
    if constexpr (SPLIT) {
        __syncwarp();
        cluster_sync();  // every CTA's part is there
        if (same_layout && warp >= 4 && !*static_cast<volatile int *>(&bars->abort_flag))
            join_tile<S>(p, smem, rank, worker, threadIdx.x - 128);
    }

    tc_fence_before_sync();
    __syncthreads();
    if constexpr (PAIR || SPLIT) cluster_sync();  // no CTA leaves while another may still use its barriers, memory or TMEM
    tc_fence_after_sync();
    if (warp == 0) {
        __syncwarp();
        if constexpr (PAIR)
            tmem_dealloc_pair(tmem, TMEM_COLS);
        else
            tmem_dealloc(tmem, TMEM_COLS);
    }
}

template <class S>
cudaError_t set_attributes()
{
    cudaFuncAttributes a;
    const cudaError_t e = cudaFuncGetAttributes(&a, linear_kernel<S>);
    if (e != cudaSuccess) return e;
    if (a.numRegs < S::REGS_LAUNCH) return cudaErrorInvalidConfiguration;  // the exchange of registers could not end
    return cudaFuncSetAttribute(linear_kernel<S>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
}

template <class S>
int max_clusters(int ctas)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(S::THREADS);
    cfg.dynamicSmemBytes = S::SMEM;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ctas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int clusters = 0;
    if (cudaOccupancyMaxActiveClusters(&clusters, linear_kernel<S>, &cfg) != cudaSuccess) {
        (void)cudaGetLastError();
        return 0;
    }
    return clusters;
}

// clusters of `cluster` CTAs, `grid` CTAs in all
template <class S>
cudaError_t launch(const LinearMaps &maps, const LinearParams &p, long long grid, int cluster, bool dependent, cudaStream_t stream)
{
    return launch_kernel_cluster(dependent, cluster, linear_kernel<S>, dim3(static_cast<unsigned>(grid)), dim3(S::THREADS), S::SMEM,
                                 stream, maps, p);
}

template <bool F32>
cudaError_t launch_typed(const LinearMaps &maps, const LinearParams &p, int ctas, long long tiles, int workers, bool dependent,
                         cudaStream_t stream)
{
    if (p.splits > 0)
        return p.bn == 128 ? launch<Shape<1, 128, F32, true>>(maps, p, tiles * p.splits, p.splits, dependent, stream)
                           : launch<Shape<1, 256, F32, true>>(maps, p, tiles * p.splits, p.splits, dependent, stream);
    const long long n = std::min<long long>(tiles, workers);
    return ctas == 2 ? launch<Shape<2, 256, F32, false>>(maps, p, 2 * n, 2, dependent, stream)
                     : launch<Shape<1, 256, F32, false>>(maps, p, n, 1, dependent, stream);
}

template <bool F32>
cudaError_t set_typed()
{
    for (cudaError_t e : {set_attributes<Shape<1, 256, F32, false>>(), set_attributes<Shape<2, 256, F32, false>>(),
                          set_attributes<Shape<1, 128, F32, true>>(), set_attributes<Shape<1, 256, F32, true>>()})
        if (e != cudaSuccess) return e;
    return cudaSuccess;
}

}  // namespace

cudaError_t linear_set_attributes()
{
    const cudaError_t e = set_typed<false>();
    return e != cudaSuccess ? e : set_typed<true>();
}

int linear_max_pairs() { return max_clusters<Shape<2, 256, true, false>>(2); }

void linear_max_clusters(int *clusters)
{
    for (int c = 1; c <= kLinearMaxSplits; ++c) clusters[c - 1] = max_clusters<Shape<1, 256, true, true>>(c);
}

cudaError_t launch_linear_tiles(const LinearMaps &maps, const LinearParams &p, int ctas, int workers, bool dependent,
                                cudaStream_t stream)
{
    long long tiles = 0;
    for (int i = 0; i < p.products_of_launch; ++i) tiles += static_cast<long long>(p.t[i].tiles_m) * p.t[i].tiles_n;
    return p.dtype == SGEMM_DTYPE_F32 ? launch_typed<true>(maps, p, ctas, tiles, workers, dependent, stream)
                                      : launch_typed<false>(maps, p, ctas, tiles, workers, dependent, stream);
}

}  // namespace sgemm_impl
