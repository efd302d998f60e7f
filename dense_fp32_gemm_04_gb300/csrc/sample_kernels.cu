// One token per row of logits. Contract: include/sgemm_sample.h.
//
// A cluster of 1 to 8 CTAs takes a row, each a run of it that stays in shared memory
// (where it fits), so the logits are read from memory once. What the row needs of
// other CTAs goes through distributed shared memory; a call is one launch without
// workspace.
//
// Weights are integers. A token is a whole number, and sums rounded in an order of
// their own would give another one where u S lies next to a border: with V = 131072
// entries of a flat row, FP32 sums would be wrong in one row of ten. So
// w = exp((l - m) / T) is computed in pairs of FP32 numbers to about 2^-45 of the
// largest weight (FP64 units are too few: 2 operations a clock and SM), rounded to a
// multiple of 2^-44, and added in 64-bit integers, which is exact in any order, with
// atomics too. That is Weigh, some 60 instructions an entry. Rough takes a third of them
// and is off by up to 1.5 * 2^-22 of the weight: sums of those decide nearly every row,
// since what they can be off by is known; where u S or a cut's share lies within that of
// a border, the sums are taken again with Weigh. What a row gives is the same either way.
//
// Every filter keeps a beginning of the order (logit descending, index ascending), so
// what is kept is one cut in it, a (logit, index) pair as a 64-bit number. The cut of a
// count (top-k) or of a mass (top-p) is looked for in a histogram over the distance
// from the largest logit: 2048 bins of T / 128, counts only, in 32 bits. Weights in a
// bin differ by 0.8 %, so the counts say in which few bins a cut of a mass lies; one
// pass adds up the weights above them and all of them, and the entries of those bins are
// sorted in one CTA. Where they are more than it sorts (many equal logits, flat rows),
// further histograms narrow the range, and equal entries are counted in order of the
// index (refine()). Where everything that is kept is among the sorted entries, that CTA
// draws from them (finish()); else find() walks what is kept in order of the index: sums
// of blocks of 256 entries, then the one block that the target lies in.
//
// What bounds it: not memory (64 rows of 131072 in FP32 are read in 5 us), but a chain of
// passes over shared memory with meetings of the cluster between them, 1 to 2 us each, and
// the instructions of the passes. Measured, in us:
//                                  greedy  unfiltered  top 50  top 50 and p  top-p  min-p
//   1 x 32768, bfloat16              3.7       7.8      15.5       17.3       23.2    9.1
//   64 x 131072, FP32               10.7      33        46         49         91      34
//   512 x 50021, FP32               28        67       117        126        198      81
// (all weights by Weigh: unfiltered 512 x 50021 100, top-p 292).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "device_ptx.cuh"
#include "sample_internal.h"

namespace sgemm_impl {
namespace {

using namespace sgemm_dev;
typedef unsigned long long u64;

constexpr int BLOCK = kSampleBlock;
constexpr int BINS = 2048;
constexpr int WIDE_BINS = 1024;  // of 64 bits, in the same memory
constexpr int SORT = 1024;       // entries that one CTA sorts, there too
constexpr int LIST = 512;        // and that a CTA collects (1024 would leave three CTAs less of L1: loads then take 33 us for 28)
constexpr int MAX_CTAS = 8, MAX_WARPS = 16;
constexpr int SLOTS = 192;       // (a row takes 162 at most)
constexpr int Q = 44;            // weights are multiples of 2^-Q
constexpr float kInf = __builtin_huge_valf();

// 2^(i / 1024) as a sum of two FP32 numbers, from the exponential series.
struct Powers {
    float2 at[1024];
};
constexpr Powers make_powers()
{
    Powers p{};
    for (int i = 0; i < 1024; ++i) {
        const double x = i * (0.693147180559945309417 / 1024.0);
        double term = 1.0, sum = 0.0;
        for (int k = 1; k < 24; ++k) {
            sum += term;
            term *= x / k;
        }
        p.at[i].x = static_cast<float>(sum);
        p.at[i].y = static_cast<float>(sum - static_cast<double>(p.at[i].x));
    }
    return p;
}
__device__ const Powers kPowers = make_powers();

struct Shared {
    union {
        unsigned bins[BINS];
        u64 wide[WIDE_BINS];
        u64 sorted[SORT];
    };
    u64 list[LIST];
    u64 pub[SLOTS];       // what this CTA says to the others, each slot once per row
    u64 all[4][MAX_CTAS]; // what all said
    u64 red[2 * MAX_WARPS];
    u64 found[2];
    unsigned lo, hi;
    int n, pad;
};
static_assert(sizeof(Shared) % 16 == 0, "what follows starts on a 16-byte boundary");

__device__ __forceinline__ u64 ld_cluster_u64(uint32_t addr)
{
    u64 v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
    return v;
}

// The sum over the cluster's CTAs of the number at this address in each (all loads on their way together).
template <typename T>
__device__ __forceinline__ T cluster_sum(uint32_t addr, int ctas)
{
    T x[MAX_CTAS];
#pragma unroll
    for (int c = 0; c < MAX_CTAS; ++c) {
        x[c] = 0;
        if (c >= ctas) continue;
        if constexpr (sizeof(T) == 8)
            x[c] = ld_cluster_u64(mapa_shared(addr, c));
        else
            x[c] = ld_shared_cluster_u32(mapa_shared(addr, c));
    }
    T sum = 0;
#pragma unroll
    for (int c = 0; c < MAX_CTAS; ++c) sum += x[c];
    return sum;
}

// FP32 numbers in their order as unsigned ones (-0 is 0).
__device__ __forceinline__ unsigned ordered(float x)
{
    const unsigned b = __float_as_uint(x + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float unordered(unsigned k)
{
    return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}
// (l descending, index ascending) as a descending number.
__device__ __forceinline__ u64 place(float l, int i) { return static_cast<u64>(ordered(l)) << 32 | ~static_cast<unsigned>(i); }

// A cut in that order: what is at it or above.
struct Cut {
    float l;
    int i;
    __device__ __forceinline__ bool keeps(float x, int at) const { return x > l || (x == l && at <= i); }
};
__device__ __forceinline__ Cut cut_at(u64 p) { return Cut{unordered(static_cast<unsigned>(p >> 32)), static_cast<int>(~static_cast<unsigned>(p))}; }

// w = exp((l - m) / T) as a multiple of 2^-(Q - drop), two of them at a time with packed FP32 (a scalar one costs the same
// number of instructions).
struct Weigh {
    float top, ch, cl;  // m; log2(e) / T in two parts
    int drop;

    __device__ __forceinline__ void two(float l0, float l1, u64 &w0, u64 &w1) const
    {
        typedef unsigned long long f2;
        auto both = [](float x) { return pack_f32x2(x, x); };
        // d = l - m exactly, t = d log2(e) / T, both in two parts
        const f2 l = pack_f32x2(l0, l1), less = both(-1.0f), c = both(ch);
        const f2 dh = add_f32x2(l, both(-top)), back = fma_f32x2(l, less, dh), rest1 = fma_f32x2(back, less, dh);
        const f2 dl = add_f32x2(fma_f32x2(rest1, less, l), fma_f32x2(back, less, both(-top)));
        const f2 tm = mul_f32x2(dh, both(-ch));  // -t
        const f2 tl = add_f32x2(fma_f32x2(dh, c, tm), fma_f32x2(dh, both(cl), mul_f32x2(dl, c)));
        // Below 2^-(60 - drop) (and where l is -infinity or NaN) the bits of w are shifted out, whatever they are: by 60, as a
        // shift by 64 would leave them all.
        float t0, t1;
        unpack_f32x2(tm, t0, t1);
        const float far = static_cast<float>(drop - 60);
        const f2 th = pack_f32x2(fmaxf(-t0, far), fmaxf(-t1, far));
        // t = k / 1024 + r, r at most 2^-11 and a little
        constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23: its neighbours are 1 apart, k stands in its low bits
        constexpr int kBits = 0x4b400000;
        const f2 kf = fma_f32x2(th, both(1024.0f), both(kMagic));
        const f2 r0 = fma_f32x2(add_f32x2(kf, both(-kMagic)), both(-1.0f / 1024.0f), th);
        const f2 r = add_f32x2(r0, tl), rl = add_f32x2(fma_f32x2(r, less, r0), tl);
        // 2^r = 1 + x + x^2 / 2 + x^3 / 6 with x = r log(2); the next term is 2^-50
        constexpr float kLn2 = 0.693147180559945309417, kLn2Low = 0.693147180559945309417 - static_cast<double>(kLn2);
        const f2 xh = mul_f32x2(r, both(kLn2)), xm = mul_f32x2(r, both(-kLn2));
        const f2 xl = add_f32x2(fma_f32x2(r, both(kLn2), xm), fma_f32x2(r, both(kLn2Low), mul_f32x2(rl, both(kLn2))));
        const f2 x = add_f32x2(xh, xl);
        const f2 more = fma_f32x2(mul_f32x2(x, x), fma_f32x2(x, both(1.0f / 6.0f), both(0.5f)), xl);
        float k0, k1;
        unpack_f32x2(kf, k0, k1);
        const int i0 = __float_as_int(k0), i1 = __float_as_int(k1);
        const float2 p0 = __ldg(&kPowers.at[i0 & 1023]), p1 = __ldg(&kPowers.at[i1 & 1023]);
        const f2 px = pack_f32x2(p0.x, p1.x), py = pack_f32x2(p0.y, p1.y);
        // 2^t = 2^(k / 1024) (p.x + ph + low); p.x holds 24 bits, ph * 2^32 and the rest * 2^44 are below 2^22
        const f2 ph = mul_f32x2(px, xh), pm = mul_f32x2(px, xm);
        const f2 low = add_f32x2(fma_f32x2(px, xh, pm), fma_f32x2(px, more, py));
        const f2 af = fma_f32x2(ph, both(4294967296.0f), both(kMagic));
        const f2 left = add_f32x2(fma_f32x2(add_f32x2(af, both(-kMagic)), both(-1.0f / 4294967296.0f), ph), low);
        const f2 bf = fma_f32x2(left, both(17592186044416.0f), both(kMagic));
        float a0, a1, b0, b1;
        unpack_f32x2(af, a0, a1);
        unpack_f32x2(bf, b0, b1);
        auto close = [&](int k, float p, float a, float b) -> u64 {
            // twice what there is, so that the last bit rounds; 64 bits hold it whatever the floats are
            const int m = (__float_as_int(p) & 0x7fffff) | 0x800000;
            long long w = static_cast<long long>(m) * (1 << 22) - (static_cast<long long>(kBits) * (1 << 13) + static_cast<long long>(kBits) * 2);
            w += static_cast<long long>(__float_as_int(a)) * (1 << 13);
            w += static_cast<long long>(__float_as_int(b)) * 2;
            return ((static_cast<u64>(w) >> ((drop + (kBits >> 10) - (k >> 10)) & 63)) + 1) >> 1;
        };
        w0 = close(i0, p0.x, a0, b0);
        w1 = close(i1, p1.x, a1, b1);
    }

    __device__ __forceinline__ u64 operator()(float l) const
    {
        u64 w0, w1;
        two(l, l, w0, w1);
        return w0;
    }
};

// w in one FP32 exponential. l log2(e) / T = k + r with k whole and r at most a half in size, and the same of m; then
// w = 2^(k - k_m) 2^(r - r_m). Each r is off by 0.75 * 2^-24 at most, their difference so by 2.5 * 2^-24, and ex2.approx by
// 2^-22 of itself, so that w is off by less than 1.5 * 2^-22 of itself, and by half a unit of 2^-(Q - drop) as all are; the largest
// logit has exactly 1, for its r is r_m. Only where |m| log2(e) / T is below 2^20, and temperatures are no extremes (rough_can).
__device__ __forceinline__ bool rough_can(float tau, float top, float scale)
{
    return tau > 1e-30f && tau < 1e30f && fabsf(top) < 1e30f && fabsf(top) * scale < 1048576.0f;
}

// By how much a sum up to about `goal` and a goal that is a share of another such sum can be off against each other.
__device__ __forceinline__ u64 rough_doubt(u64 goal, int entries) { return (goal >> 21) + (goal >> 22) + 2 * static_cast<u64>(entries); }

// A sum of a few (512 at most) such weights as an integer, in two parts of 22 bits (a conversion to 64 bits runs on the FP64 units):
// the numbers a and b below are 1.5 * 2^23 + x for whole x, so x stands in the low bits of the float, and plain adds sum it up.
struct Parts {
    static constexpr int kBits = 0x4b400000;
    int a = 0, b = 0, n = 0;
    __device__ __forceinline__ void add(int a0, int b0)
    {
        a += a0;
        b += b0;
        ++n;
    }
    __device__ __forceinline__ u64 sum() const
    {
        const unsigned off = static_cast<unsigned>(n) * kBits;
        return (static_cast<u64>(static_cast<unsigned>(a) - off) << 22) +
               static_cast<u64>(static_cast<long long>(static_cast<int>(static_cast<unsigned>(b) - off)));
    }
};

struct Rough {
    typedef unsigned long long f2;
    static constexpr float kMagic = 12582912.0f;
    float ch, cl, r_top, least;  // log2(e) / T in two parts, r_m; logits below least (2^-60), and NaN, are taken as it
    int exponent;                // Q - drop - k_m, for the exponent's bits

    __device__ __forceinline__ Rough(float top, float scale, float scale_low, int drop) : ch(scale), cl(scale_low)
    {
        least = top - 60.0f / scale;
        const float kf = fmaf(top, ch, kMagic), km = fmaf(kf, -1.0f, kMagic);
        r_top = fmaf(top, cl, fmaf(top, ch, km));
        exponent = (Q - drop + static_cast<int>(km)) << 23;
    }
    // The weights, in units of 2^-(Q - drop).
    __device__ __forceinline__ f2 two(float l0, float l1) const
    {
        auto both = [](float x) { return pack_f32x2(x, x); };
        const f2 l = pack_f32x2(fmaxf(l0, least), fmaxf(l1, least)), c = both(ch);
        const f2 kf = fma_f32x2(l, c, both(kMagic)), km = fma_f32x2(kf, both(-1.0f), both(kMagic));  // -k
        const f2 r = add_f32x2(fma_f32x2(l, both(cl), fma_f32x2(l, c, km)), both(-r_top));
        float r0, r1, k0, k1;
        unpack_f32x2(r, r0, r1);
        unpack_f32x2(kf, k0, k1);
        auto power = [&](float x, float k) {  // (k stands in the low bits of its float)
            float y;
            asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
            return __int_as_float(__float_as_int(y) + (__float_as_int(k) << 23) + exponent);
        };
        return pack_f32x2(power(r0, k0), power(r1, k1));
    }
    static __device__ __forceinline__ void split(f2 y, int &a0, int &b0, int &a1, int &b1)
    {
        auto both = [](float x) { return pack_f32x2(x, x); };
        const f2 af = fma_f32x2(y, both(1.0f / 4194304.0f), both(kMagic));
        const f2 bf = add_f32x2(fma_f32x2(add_f32x2(af, both(-kMagic)), both(-4194304.0f), y), both(kMagic));
        float x0, x1, y0, y1;
        unpack_f32x2(af, x0, x1);
        unpack_f32x2(bf, y0, y1);
        a0 = __float_as_int(x0);
        a1 = __float_as_int(x1);
        b0 = __float_as_int(y0);
        b1 = __float_as_int(y1);
    }
    static __device__ __forceinline__ void add(f2 y, Parts &to)
    {
        int a0, b0, a1, b1;
        split(y, a0, b0, a1, b1);
        to.add(a0, b0);
        to.add(a1, b1);
    }
};

// A row as one CTA of its cluster sees it: `n` positions, an even number, position p being entry first + p. In shared memory
// they start on a 16-byte boundary of the row, and positions that are no entries of this CTA's hold -infinity.
template <typename E>
struct Run {
    const E *shared;  // NULL: read from memory
    const E *global;  // position 0 (shared == NULL)
    int n, first;
    int end;          // positions that there are in memory
    bool infinite;    // the largest logit is +infinity (shared == NULL; else the run itself has been changed)

    __device__ __forceinline__ float far(int p) const
    {
        const float l = p < end ? static_cast<float>(global[p]) : -kInf;
        return infinite ? l == kInf ? 0.0f : -kInf : l;
    }
    // (NaN stays NaN: it is above no cut and in no bin, and has no weight)
    __device__ __forceinline__ void two(int p, float &l0, float &l1) const
    {
        if (shared != nullptr) {
            if constexpr (sizeof(E) == 4) {
                const float2 l = *reinterpret_cast<const float2 *>(shared + p);
                l0 = l.x;
                l1 = l.y;
            } else {
                const uint32_t l = *reinterpret_cast<const uint32_t *>(shared + p);
                l0 = __uint_as_float(l << 16);
                l1 = __uint_as_float(l & 0xffff0000u);
            }
        } else {
            l0 = far(p);
            l1 = far(p + 1);
        }
    }
};

__device__ __forceinline__ u64 warp_sum(u64 x)
{
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

__device__ __forceinline__ u64 warp_max(u64 x)
{
    for (int o = 16; o > 0; o >>= 1) x = max(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}

// One row at work: what the functions below share.
template <typename E, int THREADS>
struct Team {
    static constexpr int WARPS = THREADS / 32;
    Shared *s;
    u64 *blocks;  // sums of blocks of the run
    Run<E> run;
    int ctas, rank, tid;
    int entries;  // of the row
    float top, per_bin, tau;
    int slot = 0;  // the next free one

    // The CTAs meet; the numbers that thread 0 put into the next `count` slots of each are then in s->all.
    __device__ __forceinline__ void meet(int count)
    {
        cluster_sync();
        if (tid < ctas * count)
            s->all[tid / ctas][tid % ctas] = ld_cluster_u64(mapa_shared(smem_addr(&s->pub[slot + tid / ctas]), tid % ctas));
        slot += count;
        __syncthreads();
    }
    __device__ __forceinline__ u64 from(int cta, int at) const { return ld_cluster_u64(mapa_shared(smem_addr(&s->pub[at]), cta)); }
    __device__ __forceinline__ u64 sum(int which) const
    {
        u64 x = 0;
        for (int c = 0; c < ctas; ++c) x += s->all[which][c];
        return x;
    }
    // The CTA that `target` (below the sum of all) lies in, and what is before it.
    __device__ __forceinline__ int owner(u64 target, u64 &before) const
    {
        before = 0;
        for (int c = 0; c + 1 < ctas; ++c) {
            if (target < before + s->all[0][c]) return c;
            before += s->all[0][c];
        }
        return ctas - 1;
    }

    // The sum over the block, in thread 0.
    __device__ __forceinline__ u64 block_sum(u64 x)
    {
        x = warp_sum(x);
        __syncthreads();
        if ((tid & 31) == 0) s->red[tid >> 5] = x;
        __syncthreads();
        x = 0;
        if (tid == 0)
            for (int w = 0; w < WARPS; ++w) x += s->red[w];
        return x;
    }

    __device__ __forceinline__ void block_sums(u64 &x, u64 &y)
    {
        x = warp_sum(x);
        y = warp_sum(y);
        __syncthreads();
        if ((tid & 31) == 0) {
            s->red[tid >> 5] = x;
            s->red[WARPS + (tid >> 5)] = y;
        }
        __syncthreads();
        x = y = 0;
        if (tid == 0)
            for (int w = 0; w < WARPS; ++w) {
                x += s->red[w];
                y += s->red[WARPS + w];
            }
    }

    // Exclusive sum over the block's threads, and the total.
    __device__ __forceinline__ u64 scan(u64 x, u64 &total)
    {
        const int lane = tid & 31, warp = tid >> 5;
        u64 in = x;
        for (int o = 1; o < 32; o <<= 1) {
            const u64 y = __shfl_up_sync(0xffffffffu, in, o);
            if (lane >= o) in += y;
        }
        __syncthreads();
        if (lane == 31) s->red[warp] = in;
        __syncthreads();
        u64 before = 0;
        total = 0;
        for (int w = 0; w < WARPS; ++w) {
            const u64 y = s->red[w];
            if (w < warp) before += y;
            total += y;
        }
        return before + in - x;
    }
    __device__ __forceinline__ float scan(float x, float &total)
    {
        const int lane = tid & 31, warp = tid >> 5;
        float in = x;
        for (int o = 1; o < 32; o <<= 1) {
            const float y = __shfl_up_sync(0xffffffffu, in, o);
            if (lane >= o) in += y;
        }
        __syncthreads();
        if (lane == 31) s->red[warp] = __float_as_uint(in);
        __syncthreads();
        float before = 0.0f;
        total = 0.0f;
        for (int w = 0; w < WARPS; ++w) {
            const float y = __uint_as_float(static_cast<unsigned>(s->red[w]));
            if (w < warp) before += y;
            total += y;
        }
        return before + in - x;
    }

    // f(l0, l1, p) for this thread's pairs of positions; all lanes of a warp take part in every call.
    // (after(): when it has been called for a few of them)
    template <typename F, typename G>
    __device__ __forceinline__ void pairs(F f, G after) const
    {
        constexpr int AHEAD = 4;  // (run.n is a multiple of 64: a warp's pairs exist or do not)
        for (int p0 = (tid & ~31) * 2; p0 < run.n; p0 += 2 * THREADS * AHEAD) {
            float l0[AHEAD], l1[AHEAD];
#pragma unroll
            for (int j = 0; j < AHEAD; ++j)
                if (p0 + 2 * THREADS * j < run.n) run.two(p0 + 2 * THREADS * j + (tid & 31) * 2, l0[j], l1[j]);
#pragma unroll
            for (int j = 0; j < AHEAD; ++j)
                if (p0 + 2 * THREADS * j < run.n) f(l0[j], l1[j], p0 + 2 * THREADS * j + (tid & 31) * 2);
            after();
        }
    }
    template <typename F>
    __device__ __forceinline__ void pairs(F f) const
    {
        pairs(f, [] {});
    }

    // The distance from the largest logit in bins; an entry's bin is its whole part, at most BINS - 1.
    __device__ __forceinline__ float bins_from(float l) const { return (top - l) * per_bin; }
    __device__ __forceinline__ float capped(float l) const { return fminf(bins_from(l), BINS - 1); }
    __device__ __forceinline__ int bin_of(float l) const { return static_cast<int>(capped(l)); }
};

// In order of the index, the entry at which the cumulative weight passes target(sum of all): its index and weight, in every
// CTA, or (LAST: nothing of the row follows) in the CTA that has it, the others left as they were.
// sums(l0, l1, i, w0, w1): the weights of entries i and i + 1 that sums are made of, weights(...) those in the block
// where the target lies; all lanes of a warp call them together. ROUGH: sums(l0, l1, i) are those of Rough; false where the entry
// is not sure (in every CTA alike; not with LAST).
template <bool LAST, bool ROUGH, typename E, int THREADS, typename R, typename W, typename F>
__device__ __forceinline__ bool find(Team<E, THREADS> &t, const R &sums, const W &weights, const F &target, int &index, u64 &w,
                                     u64 &all)
{
    static_assert(!LAST || !ROUGH, "the others have to learn whether it is sure");
    Shared *s = t.s;
    const Run<E> &run = t.run;
    const int lane = t.tid & 31, warp = t.tid >> 5, count = (run.n + BLOCK - 1) / BLOCK;
    __syncthreads();
    for (int b = warp; b < count; b += t.WARPS) {
        const int to = min((b + 1) * BLOCK, run.n);
        u64 sum = 0;
        Parts parts;
        // (to is a multiple of 64; several pairs at a time, or their latency would be most of the time)
        constexpr int AHEAD = 4;
        for (int p0 = b * BLOCK; p0 < to; p0 += 64 * AHEAD) {
            float l0[AHEAD], l1[AHEAD];
#pragma unroll
            for (int j = 0; j < AHEAD; ++j)
                if (p0 + 64 * j < to) run.two(p0 + 64 * j + 2 * lane, l0[j], l1[j]);
#pragma unroll
            for (int j = 0; j < AHEAD; ++j) {
                if (p0 + 64 * j >= to) break;
                const int i = run.first + p0 + 64 * j + 2 * lane;
                if constexpr (ROUGH) {
                    Rough::add(sums(l0[j], l1[j], i), parts);
                } else {
                    u64 w0, w1;
                    sums(l0[j], l1[j], i, w0, w1);
                    sum += w0 + w1;
                }
            }
        }
        sum = warp_sum(ROUGH ? parts.sum() : sum);
        if (lane == 0) t.blocks[b] = sum;
    }
    __syncthreads();
    if (warp == 0) {
        u64 mine = 0;
        for (int b = lane; b < count; b += 32) mine += t.blocks[b];
        mine = warp_sum(mine);
        if (lane == 0) s->pub[t.slot] = mine;
    }
    t.meet(1);
    if constexpr (LAST) cluster_arrive();  // nobody reads another CTA's memory from here on
    all = t.sum(0);
    index = -1;
    w = 0;
    if (all == 0) return true;
    u64 goal = target(all), before;
    const int own = t.owner(goal, before), at = t.slot;
    t.slot += 3;
    // what the cumulative weight and the target can be off by against each other
    const u64 off = ROUGH ? rough_doubt(goal, t.entries) : 0;
    const u64 whole = goal;
    if (own == t.rank) {
        goal -= before;
        if (t.tid == 0) s->pub[at + 2] = 0;
        if (warp == 0) {
            u64 passed = 0;
            for (int b0 = 0; b0 < count; b0 += 32) {
                const u64 x = b0 + lane < count ? t.blocks[b0 + lane] : 0;
                u64 in = x;
                for (int o = 1; o < 32; o <<= 1) {
                    const u64 y = __shfl_up_sync(0xffffffffu, in, o);
                    if (lane >= o) in += y;
                }
                const bool here = goal >= passed + in - x && goal < passed + in;
                if (here) {
                    s->found[0] = b0 + lane;
                    s->found[1] = passed + in - x;
                }
                passed += __shfl_sync(0xffffffffu, in, 31);
                if (__any_sync(0xffffffffu, here)) break;
            }
        }
        __syncthreads();
        const int from = static_cast<int>(s->found[0]) * BLOCK;
        goal -= s->found[1];
        constexpr int PER = 2;  // (the other threads have none)
        u64 x[PER], part = 0, total;
#pragma unroll
        for (int j = 0; j < PER; j += 2) {
            const int p = from + t.tid * PER + j;
            float l0 = -kInf, l1 = -kInf;
            if (p < run.n && p < from + BLOCK) run.two(p, l0, l1);
            weights(l0, l1, run.first + p, x[j], x[j + 1]);
            part += x[j] + x[j + 1];
        }
        u64 sum = t.scan(part, total);
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            if (goal >= sum && goal < sum + x[j]) {
                s->pub[at] = static_cast<unsigned>(run.first + from + t.tid * PER + j);
                s->pub[at + 1] = x[j];
                // (before the first entry of weight nothing can be off)
                s->pub[at + 2] = !ROUGH || ((whole == goal - sum || goal - sum >= off) && sum + x[j] - goal > off);
                if constexpr (LAST) {
                    index = run.first + from + t.tid * PER + j;
                    w = x[j];
                }
            }
            sum += x[j];
        }
    }
    if constexpr (LAST) return true;
    cluster_sync();
    index = static_cast<int>(t.from(own, at));
    w = t.from(own, at + 1);
    return !ROUGH || t.from(own, at + 2) != 0;
}

// The entries of a range, at or above a cut: linear bins [ba, bb] and ordered() in [lo, hi].
struct Range {
    int ba, bb;
    unsigned lo, hi;
};

// The smallest and the largest ordered() that a thread has collected.
struct Span {
    unsigned lo = 0xffffffffu, hi = 0;
};

// Adds the entries that `take` says of a pair to the CTA's list (as far as there is room) and counts them.
template <typename E, int THREADS>
__device__ __forceinline__ void collect(Team<E, THREADS> &t, Span &span, float l0, float l1, int i, bool take0, bool take1)
{
    Shared *s = t.s;
    const unsigned some0 = __ballot_sync(0xffffffffu, take0), some1 = __ballot_sync(0xffffffffu, take1);
    if ((some0 | some1) == 0) return;
    const int lane = t.tid & 31;
    int at = 0;
    if (lane == 0) at = atomicAdd(&s->n, __popc(some0) + __popc(some1));
    at = __shfl_sync(0xffffffffu, at, 0);
    const unsigned before = (1u << lane) - 1u;
    auto put = [&](float l, int k, int to) {
        const u64 at = place(l, k);
        if (to < LIST) s->list[to] = at;
        span.lo = min(span.lo, static_cast<unsigned>(at >> 32));
        span.hi = max(span.hi, static_cast<unsigned>(at >> 32));
    };
    if (take0) put(l0, i, at + __popc(some0 & before));
    if (take1) put(l1, i + 1, at + __popc(some0) + __popc(some1 & before));
}

template <typename E, int THREADS>
__device__ __forceinline__ void collect_start(Team<E, THREADS> &t)
{
    __syncthreads();
    if (t.tid == 0) {
        t.s->n = 0;
        t.s->lo = 0xffffffffu;
        t.s->hi = 0;
    }
    __syncthreads();
}

// x[0, size) in descending order, size a power of two from 128 to SORT; what is there before and after stands behind barriers.
// Bitonic, four neighbours to a thread: steps over 1 and 2 stay in its registers, those up to 64 in its warp, and only those from
// 128 on go through shared memory (with all of them through it, the top 50 of 512 rows of 50021 took 143 us, now 117, sort and finish()).
template <int THREADS>
__device__ __forceinline__ void sort_descending(u64 *x, int size, int tid)
{
    constexpr int PER = 4;
    static_assert(THREADS * PER >= SORT, "a thread has four");
    const int base = tid * PER;
    const bool has = base < size;  // (of whole warps)
    u64 v[PER];
    auto load = [&](int from) {
        const ulonglong2 a = *reinterpret_cast<const ulonglong2 *>(x + from), b = *reinterpret_cast<const ulonglong2 *>(x + from + 2);
        v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
    };
    auto store = [&] {
        *reinterpret_cast<ulonglong2 *>(x + base) = make_ulonglong2(v[0], v[1]);
        *reinterpret_cast<ulonglong2 *>(x + base + 2) = make_ulonglong2(v[2], v[3]);
    };
    auto order = [](u64 &a, u64 &b, bool down) {
        const u64 high = max(a, b), low = min(a, b);
        a = down ? high : low;
        b = down ? low : high;
    };
    if (has) {
        load(base);
        order(v[0], v[1], true);
        order(v[2], v[3], false);
    }
    for (int k = 4; k <= size; k <<= 1) {
        const bool down = (base & k) == 0;
        int j = k >> 1;
        for (; j >= 32 * PER; j >>= 1) {
            u64 mine[PER];
            if (has) store();
#pragma unroll
            for (int e = 0; e < PER; ++e) mine[e] = v[e];
            __syncthreads();
            if (has) {
                load(base ^ j);
#pragma unroll
                for (int e = 0; e < PER; ++e) v[e] = ((base & j) == 0) == down ? max(mine[e], v[e]) : min(mine[e], v[e]);
            }
            __syncthreads();
        }
        if (!has) continue;
        for (; j >= PER; j >>= 1) {
            const bool larger = ((base & j) == 0) == down;
#pragma unroll
            for (int e = 0; e < PER; ++e) {
                const u64 other = __shfl_xor_sync(0xffffffffu, v[e], j / PER);
                v[e] = larger ? max(v[e], other) : min(v[e], other);
            }
        }
        order(v[0], v[2], down);
        order(v[1], v[3], down);
        order(v[0], v[1], down);
        order(v[2], v[3], down);
    }
    if (has) store();
    __syncthreads();
}

__device__ __forceinline__ int sorted_size(int n) { return n <= 128 ? 128 : 1 << (32 - __clz(n - 1)); }

// All CTAs' lists, in rank 0's `sorted` and in order. Returns the number of entries (in every CTA); -1 if they do not fit. Then
// nothing is sorted and range has the entries' ordered(). SUMS: x and y, in thread 0 its CTA's, become the cluster's in every one.
template <bool SUMS, typename E, int THREADS>
__device__ __forceinline__ int gather(Team<E, THREADS> &t, const Span &span, Range &range, u64 &x, u64 &y)
{
    Shared *s = t.s;
    const unsigned warp_lo = __reduce_min_sync(0xffffffffu, span.lo), warp_hi = __reduce_max_sync(0xffffffffu, span.hi);
    if ((t.tid & 31) == 0) {
        atomicMin(&s->lo, warp_lo);
        atomicMax(&s->hi, warp_hi);
    }
    __syncthreads();
    if (t.tid == 0) {
        s->pub[t.slot] = static_cast<unsigned>(s->n);
        s->pub[t.slot + 1] = static_cast<u64>(s->hi) << 32 | s->lo;
        if (SUMS) {
            s->pub[t.slot + 2] = x;
            s->pub[t.slot + 3] = y;
        }
    }
    t.meet(SUMS ? 4 : 2);
    if (SUMS) {
        x = t.sum(2);
        y = t.sum(3);
    }
    long long n = 0;
    bool fits = true;
    unsigned lo = 0xffffffffu, hi = 0;
    for (int c = 0; c < t.ctas; ++c) {
        n += static_cast<long long>(s->all[0][c]);
        fits = fits && s->all[0][c] <= LIST;
        lo = min(lo, static_cast<unsigned>(s->all[1][c]));
        hi = max(hi, static_cast<unsigned>(s->all[1][c] >> 32));
    }
    if (!fits || n > SORT) {
        range.lo = lo;
        range.hi = hi;
        return -1;
    }
    if (t.rank == 0) {
        const int size = sorted_size(static_cast<int>(n));
        for (int i = t.tid; i < size; i += THREADS) {
            u64 e = 0;
            int c = 0, k = i;
            while (c < t.ctas && k >= static_cast<int>(s->all[0][c])) k -= static_cast<int>(s->all[0][c++]);
            if (c < t.ctas) e = ld_cluster_u64(mapa_shared(smem_addr(&s->list[k]), c));
            s->sorted[i] = e;
        }
        __syncthreads();
        sort_descending<THREADS>(s->sorted, size, t.tid);
    }
    return static_cast<int>(n);
}

template <typename E, int THREADS>
__device__ __forceinline__ int gather(Team<E, THREADS> &t, const Span &span, Range &range)
{
    u64 none = 0;
    return gather<false>(t, span, range, none, none);
}

// Rank 0: the entry of the n sorted ones at which the sum of value reaches goal >= 1 (the last one if it does not), into slot
// `at`; into the next one whether it is that whatever the goal is off by, up to `off` (first: nothing is before the sorted ones).
template <typename E, int THREADS, typename W>
__device__ __forceinline__ void resolve(Team<E, THREADS> &t, int n, u64 goal, const W &value, int at, u64 off = 0, bool first = false)
{
    Shared *s = t.s;
    constexpr int PER = SORT / THREADS;
    u64 v[PER], sum = 0, whole;
    for (int j = 0; j < PER; ++j) {
        const int i = t.tid * PER + j;
        v[j] = i < n ? value(unordered(static_cast<unsigned>(s->sorted[i] >> 32))) : 0;
        sum += v[j];
    }
    u64 passed = t.scan(sum, whole);
    const bool there = goal <= whole;
    goal = max(min(goal, whole), 1ull);
    if (whole == 0 && t.tid == 0) {  // (no call comes here: the cut has weight)
        s->pub[at] = s->sorted[0];
        s->pub[at + 1] = 0;
    }
    for (int j = 0; j < PER; ++j) {
        if (passed < goal && goal <= passed + v[j]) {
            s->pub[at] = s->sorted[t.tid * PER + j];
            s->pub[at + 1] = there && ((first && passed == 0) || goal - passed > off) && passed + v[j] - goal >= off;
        }
        passed += v[j];
    }
}

// Rank 0, where all that is kept stands among its n sorted entries (down to `cut`, of weight `least` or more): they are sorted by
// index, and the entry is found as in find(): the thread that has it gets its index and weight, all get the sum.
template <typename E, int THREADS, typename F>
__device__ __forceinline__ void finish(Team<E, THREADS> &t, int n, u64 cut, u64 least, const Weigh &weigh, const F &target, int &index,
                                       u64 &w, u64 &all)
{
    Shared *s = t.s;
    constexpr int PER = SORT / THREADS;
    const int size = sorted_size(n);
    for (int i = t.tid; i < size; i += THREADS) {
        const u64 e = i < n ? s->sorted[i] : 0;
        const bool keep = e != 0 && e >= cut && weigh(unordered(static_cast<unsigned>(e >> 32))) >= least;
        s->sorted[i] = keep ? e >> 32 | e << 32 : 0;  // ~index first
    }
    __syncthreads();
    sort_descending<THREADS>(s->sorted, size, t.tid);
    u64 e[PER], v[PER], sum = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int i = t.tid * PER + j;
        e[j] = i < n ? s->sorted[i] : 0;
        v[j] = e[j] != 0 ? weigh(unordered(static_cast<unsigned>(e[j]))) : 0;
        sum += v[j];
    }
    u64 passed = t.scan(sum, all);
    const u64 goal = target(all);
    index = -1;
    w = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        if (goal >= passed && goal < passed + v[j]) {
            index = static_cast<int>(~static_cast<unsigned>(e[j] >> 32));
            w = v[j];
        }
        passed += v[j];
    }
}

// The bin of `wide` (all CTAs' together) in which the sum reaches goal, which is then counted from that bin on; -1 if all are 0.
template <typename E, int THREADS>
__device__ __forceinline__ int pick_wide(Team<E, THREADS> &t, u64 &goal)
{
    Shared *s = t.s;
    cluster_sync();
    // this CTA's part of the bins, summed over all CTAs
    const int part = WIDE_BINS / t.ctas, per = (part + THREADS - 1) / THREADS;
    u64 x[WIDE_BINS / THREADS] = {}, mine = 0, total;
    if (t.tid * per < part) {
#pragma unroll
        for (int j = 0; j < WIDE_BINS / THREADS; ++j) {
            if (j >= per) break;
            x[j] = cluster_sum<u64>(smem_addr(&s->wide[t.rank * part + t.tid * per + j]), t.ctas);
            mine += x[j];
        }
    }
    u64 before = t.scan(mine, total), earlier;
    if (t.tid == 0) s->pub[t.slot] = total;
    t.meet(1);
    if (t.sum(0) == 0) return -1;
    goal = min(goal, t.sum(0));
    const int own = t.owner(goal - 1, earlier), at = t.slot;
    t.slot += 2;
    if (own == t.rank) {
        before += earlier;
#pragma unroll
        for (int j = 0; j < WIDE_BINS / THREADS; ++j) {
            if (before < goal && goal <= before + x[j]) {
                s->pub[at] = static_cast<unsigned>(t.rank * part + t.tid * per + j);
                s->pub[at + 1] = before;
            }
            before += x[j];
        }
    }
    cluster_sync();
    goal -= t.from(own, at + 1);
    return static_cast<int>(t.from(own, at));
}

// Collects a range's entries at or above the cut.
template <typename E, int THREADS>
__device__ __forceinline__ Span collect_range(Team<E, THREADS> &t, const Cut &cut, const Range &range)
{
    Span span;
    collect_start(t);
    const float from = static_cast<float>(range.ba), to = static_cast<float>(range.bb + 1);
    t.pairs([&](float l0, float l1, int p) {
        auto in = [&](float l, int i) {
            const float b = t.capped(l);
            if (!(l > -kInf) || !(b >= from) || !(b < to) || !cut.keeps(l, i)) return false;
            const unsigned k = ordered(l);
            return k >= range.lo && k <= range.hi;
        };
        const int i = t.run.first + p;
        const bool in0 = in(l0, i), in1 = in(l1, i + 1);
        if (__any_sync(0xffffffffu, in0 || in1)) collect(t, span, l0, l1, i, in0, in1);
    });
    return span;
}

// The cut at which the sum of value over the range's entries (at or above `cut`), in order, reaches goal >= 1; the caller has
// collected them, in vain: there are more than are sorted.
template <typename E, int THREADS, typename W>
__device__ __forceinline__ u64 refine(Team<E, THREADS> &t, const Cut &cut, Range range, u64 goal, const W &value)
{
    Shared *s = t.s;
    for (int level = 0; level < 8; ++level) {  // (two over the bins, four over the 32 bits are the most)
        if (range.lo == range.hi) {  // equal logits: the cut is at one of them
            const float l = unordered(range.lo);
            const u64 each = max(value(l), 1ull);
            int index;
            u64 w, all;
            const auto equal = [&](float l0, float l1, int i, u64 &w0, u64 &w1) {
                w0 = l0 == l && cut.keeps(l0, i);
                w1 = l1 == l && cut.keeps(l1, i + 1);
            };
            find<false, false>(t, equal, equal, [&](u64 sum) { return min((goal - 1) / each, sum - 1); }, index, w, all);
            return place(l, index);
        }
        // a histogram of value: over the linear bins while there are several, then over ordered()
        const bool linear = range.ba < range.bb;
        const unsigned span = linear ? range.bb - range.ba : range.hi - range.lo;
        const int shift = max(0, 22 - __clz(span));  // span >> shift is below WIDE_BINS
        auto member = [&](float l, int i) {
            if (!(l > -kInf) || !cut.keeps(l, i)) return -1;
            const unsigned k = ordered(l);
            const int b = t.bin_of(l);
            if (k < range.lo || k > range.hi || b < range.ba || b > range.bb) return -1;
            return static_cast<int>((linear ? static_cast<unsigned>(b - range.ba) : range.hi - k) >> shift);
        };
        __syncthreads();
        for (int b = t.tid; b < WIDE_BINS; b += THREADS) s->wide[b] = 0;
        __syncthreads();
        t.pairs([&](float l0, float l1, int p) {
            const int b0 = member(l0, t.run.first + p), b1 = member(l1, t.run.first + p + 1);
            if (b0 >= 0) atomicAdd(&s->wide[b0], value(l0));
            if (b1 >= 0) atomicAdd(&s->wide[b1], value(l1));
        });
        const int bin = pick_wide(t, goal);
        if (bin < 0) break;  // (no call comes here)
        if (linear) {
            const int base = range.ba;
            range.ba = base + (bin << shift);
            range.bb = min(range.bb, base + ((bin + 1) << shift) - 1);
        } else {
            const unsigned top = range.hi;
            range.hi = top - (static_cast<unsigned>(bin) << shift);
            range.lo = max(static_cast<long long>(range.lo), static_cast<long long>(top) - static_cast<long long>(((static_cast<u64>(bin) + 1) << shift) - 1));
        }
        const int n = gather(t, collect_range(t, cut, range), range);
        if (n >= 0) {
            const int at3 = t.slot;
            t.slot += 2;
            if (t.rank == 0) resolve(t, n, goal, value, at3);
            cluster_sync();
            return t.from(0, at3);
        }
    }
    return 0;
}

// How many entries at or above the cut each linear bin has: this CTA's part of the bins, `per` of them a thread, summed over
// all CTAs.
template <bool CUT, typename E, int THREADS>
__device__ __forceinline__ int count_bins(Team<E, THREADS> &t, const Cut &cut, unsigned (&x)[BINS / THREADS])
{
    Shared *s = t.s;
    __syncthreads();
    for (int b = t.tid; b < BINS; b += THREADS) s->bins[b] = 0;
    __syncthreads();
    unsigned far = 0;  // the last bin can hold nearly all: counted apart
    t.pairs([&](float l0, float l1, int p) {
        auto count = [&](float l, int i) {
            const float x = t.bins_from(l);
            if (CUT && !cut.keeps(l, i)) return;
            if (x < static_cast<float>(BINS - 1))
                atomicAdd(&s->bins[static_cast<int>(x)], 1u);
            else
                far += l > -kInf;
        };
        count(l0, t.run.first + p);
        count(l1, t.run.first + p + 1);
    });
    far = __reduce_add_sync(0xffffffffu, far);
    if ((t.tid & 31) == 0 && far > 0) atomicAdd(&s->bins[BINS - 1], far);
    cluster_sync();
    const int part = BINS / t.ctas, per = (part + THREADS - 1) / THREADS;
#pragma unroll
    for (int j = 0; j < BINS / THREADS; ++j) x[j] = 0;
    if (t.tid * per < part)
#pragma unroll
        for (int j = 0; j < BINS / THREADS; ++j) {
            if (j >= per) break;
            x[j] = cluster_sum<unsigned>(smem_addr(&s->bins[t.rank * part + t.tid * per + j]), t.ctas);
        }
    return per;
}

// floor(x * n) for 0 <= x < 1, and whether something was cut off.
__device__ __forceinline__ u64 share_of(float x, u64 n, bool &more)
{
    const u64 f = static_cast<u64>(x * 4294967296.0f * 4294967296.0f);  // x 2^64: a whole number, or x is below 2^-40
    more = f * n != 0;
    return __umul64hi(f, n);
}

// The smallest mass that the share p of `all` asks for: that of the first entry at least.
__device__ __forceinline__ u64 goal_of(float p, u64 all)
{
    bool more;
    const u64 f = share_of(p, all, more);
    return max(f + more, 1ull);
}

// The cut of top-k. Where all down to it is sorted, done is the number of those entries (in every CTA); only rank 0 then has the
// cut, that of top-p too.
template <typename E, int THREADS>
__device__ __forceinline__ u64 select_count(Team<E, THREADS> &t, unsigned k, float top_p, const Weigh &weigh, int &done)
{
    Shared *s = t.s;
    const Cut all{-kInf, 0x7fffffff};
    unsigned x[BINS / THREADS];
    const int per = count_bins<false>(t, all, x);
    u64 mine = 0, total, earlier;
#pragma unroll
    for (int j = 0; j < BINS / THREADS; ++j) mine += x[j];
    u64 before = t.scan(mine, total);
    if (t.tid == 0) s->pub[t.slot] = total;
    t.meet(1);
    if (k >= t.sum(0)) return 0;
    const int own = t.owner(k - 1, earlier), at = t.slot;
    t.slot += 3;
    if (own == t.rank) {
        before += earlier;
#pragma unroll
        for (int j = 0; j < BINS / THREADS; ++j) {
            if (before < k && k <= before + x[j]) {
                s->pub[at] = static_cast<unsigned>(t.rank * (BINS / t.ctas) + t.tid * per + j);
                s->pub[at + 1] = before;
                s->pub[at + 2] = before + x[j];
            }
            before += x[j];
        }
    }
    cluster_sync();
    const int bin = static_cast<int>(t.from(own, at));
    before = t.from(own, at + 1);
    const bool whole = t.from(own, at + 2) <= (t.ctas > 2 ? SORT : LIST);  // all down to the cut's bin, or that bin alone
    if (whole) before = 0;
    Span span;
    collect_start(t);
    const float from = whole ? 0.0f : static_cast<float>(bin), to = static_cast<float>(bin + 1);
    t.pairs([&](float l0, float l1, int p) {
        auto in = [&](float l) {
            const float b = t.capped(l);
            return l > -kInf && b < to && b >= from;
        };
        const bool in0 = in(l0), in1 = in(l1);
        if (__any_sync(0xffffffffu, in0 || in1)) collect(t, span, l0, l1, t.run.first + p, in0, in1);
    });
    Range range{whole ? 0 : bin, bin, 0, 0xffffffffu};
    const int n = gather(t, span, range);
    const u64 goal = k - before;
    const auto one = [](float) { return 1ull; };
    if (n < 0) return refine(t, all, range, goal, one);  // (all that it meets are above -infinity)
    const int at3 = t.slot;
    t.slot += 2;
    if (whole) {
        done = n;
        if (t.rank != 0 || !(top_p < 1.0f)) return t.rank == 0 ? s->sorted[k - 1] : 1;
        u64 sum = 0;  // of the first k entries
        for (int i = t.tid; i < static_cast<int>(k); i += THREADS) sum += weigh(unordered(static_cast<unsigned>(s->sorted[i] >> 32)));
        sum = t.block_sum(sum);
        if (t.tid == 0) s->found[0] = sum;
        __syncthreads();
        resolve(t, static_cast<int>(k), goal_of(top_p, s->found[0]), weigh, at3);
        __syncthreads();
        return s->pub[at3];
    }
    if (t.rank == 0) resolve(t, n, goal, one, at3);
    cluster_sync();
    return t.from(0, at3);
}

// The cut of top-p among the entries at or above `cut`, or (not cutting) among all, with sums of the weights that `sums` gives.
// ROUGH: they are off by as much as Rough; false where the cut is not sure. done: as for select_count.
template <bool ROUGH, typename E, int THREADS, typename R>
__device__ __forceinline__ bool select_mass(Team<E, THREADS> &t, bool cutting, const Cut &cut, float top_p, const R &sums,
                                            const Weigh &weigh, u64 &found, int &done)
{
    Shared *s = t.s;
    unsigned x[BINS / THREADS];
    const int per = cutting ? count_bins<true>(t, cut, x) : count_bins<false>(t, cut, x), b0 = t.rank * (BINS / t.ctas) + t.tid * per;
    // Bounds of the mass: an entry of bin b weighs between exp(-(b + 1) / 128) and exp(-b / 128), but for roundings of the
    // bins and of these sums far below 2^-12; of the last bin, and where T is so small that bins are wider, only the upper
    // bound holds.
    // ROUGH takes the mean weight of a bin and a tenth of a percent for both: a range some bins wide that hardly ever misses the
    // cut, and the sums below tell when it does.
    constexpr float kSlack = ROUGH ? 1.0f / 1024.0f : 1.0f / 4096.0f;
    const bool narrow = t.tau > 1e-28f;
    float lo[BINS / THREADS], hi[BINS / THREADS], lo_sum = 0.0f, hi_sum = 0.0f, lo_all, hi_all;
#pragma unroll
    for (int j = 0; j < BINS / THREADS; ++j) {
        const float w = exp2f(-1.44269504f / 128.0f * static_cast<float>(b0 + j)), n = static_cast<float>(x[j]);
        hi[j] = n * w * (ROUGH ? b0 + j < BINS - 1 ? 0.996101f : 0.5f : 1.0f);  // 128 (1 - exp(-1 / 128))
        lo[j] = ROUGH ? hi[j] : narrow && b0 + j < BINS - 1 ? n * w * 0.992217938f : 0.0f;  // exp(-1 / 128)
        lo_sum += lo[j];
        hi_sum += hi[j];
    }
    float lo_before = t.scan(lo_sum, lo_all), hi_before = t.scan(hi_sum, hi_all);
    if (t.tid == 0) {
        s->pub[t.slot] = __float_as_uint(lo_all);
        s->pub[t.slot + 1] = __float_as_uint(hi_all);
    }
    t.meet(2);
    lo_all = hi_all = 0.0f;
    for (int c = 0; c < t.ctas; ++c) {
        const float l = __uint_as_float(static_cast<unsigned>(s->all[0][c])), h = __uint_as_float(static_cast<unsigned>(s->all[1][c]));
        if (c < t.rank) {
            lo_before += l;
            hi_before += h;
        }
        lo_all += l;
        hi_all += h;
    }
    // bins that are surely above the cut, and bins that are not surely below it
    const float sure = top_p * lo_all * (1.0f - kSlack), maybe = top_p * hi_all * (1.0f + kSlack);
    u64 bounds = 0;  // these two, and the number of entries down to the latter
#pragma unroll
    for (int j = 0; j < BINS / THREADS; ++j) {
        if (j >= per || t.tid * per >= BINS / t.ctas) break;
        bounds += lo_before < maybe ? x[j] : 0;
        hi_before += hi[j];
        lo_before += lo[j];
        bounds += static_cast<u64>(hi_before < sure) << 52 | static_cast<u64>(lo_before < maybe) << 40;
    }
    bounds = t.block_sum(bounds);
    if (t.tid == 0) s->pub[t.slot] = bounds;
    t.meet(1);
    bounds = t.sum(0);
    Range range{min(static_cast<int>(bounds >> 52), BINS - 1), min(static_cast<int>(bounds >> 40 & 0xfff), BINS - 1), 0, 0xffffffffu};
    range.bb = max(range.bb, range.ba);
    if (ROUGH && (bounds & 0xffffffffffull) <= LIST) range.ba = 0;  // so few that all are sorted
    // the exact mass of all and of what is above the range; the range's entries
    collect_start(t);
    const float from = static_cast<float>(range.ba), to = static_cast<float>(range.bb + 1);
    const int shift = max(0, 22 - __clz(static_cast<unsigned>(range.bb - range.ba)));  // the range in WIDE_BINS bins
    if (!ROUGH)
        for (int b = t.tid; b < WIDE_BINS; b += THREADS) s->wide[b] = 0;  // (the counts have been read: the CTAs have met)
    __syncthreads();
    u64 all = 0, over = 0;
    Parts some, some_over;
    Span span;
    t.pairs([&](float l0, float l1, int p) {
        const int i = t.run.first + p;
        const bool in0 = !cutting || cut.keeps(l0, i), in1 = !cutting || cut.keeps(l1, i + 1);
        if (cutting && !__any_sync(0xffffffffu, in0 || in1)) return;
        u64 w0 = 0, w1 = 0;
        const float c0 = t.capped(l0), c1 = t.capped(l1);
        if constexpr (ROUGH) {
            int a0, a1, b0, b1;
            Rough::split(sums.two(l0, l1), a0, b0, a1, b1);
            if (in0) some.add(a0, b0);
            if (in1) some.add(a1, b1);
            if (in0 && c0 < from) some_over.add(a0, b0);
            if (in1 && c1 < from) some_over.add(a1, b1);
        } else {
            sums.two(l0, l1, w0, w1);
            w0 = in0 ? w0 : 0;
            w1 = in1 ? w1 : 0;
            all += w0 + w1;
            over += (c0 < from ? w0 : 0) + (c1 < from ? w1 : 0);
        }
        const bool take0 = in0 && l0 > -kInf && c0 >= from && c0 < to, take1 = in1 && l1 > -kInf && c1 >= from && c1 < to;
        if (__any_sync(0xffffffffu, take0 || take1)) {
            if (!ROUGH && take0) atomicAdd(&s->wide[(static_cast<int>(c0) - range.ba) >> shift], w0);
            if (!ROUGH && take1) atomicAdd(&s->wide[(static_cast<int>(c1) - range.ba) >> shift], w1);
            collect(t, span, l0, l1, i, take0, take1);
        }
    }, [&] {
        if constexpr (ROUGH) {
            all += some.sum();
            over += some_over.sum();
            some = some_over = Parts();
        }
    });
    t.block_sums(all, over);
    int n = gather<true>(t, span, range, all, over);
    const u64 goal_all = goal_of(top_p, all), passed = over;
    u64 goal = goal_all > passed ? goal_all - passed : 1;
    const u64 off = ROUGH ? rough_doubt(goal_all, t.entries) : 0;
    if constexpr (ROUGH) {
        if (n < 0) return false;
        bool there = false;
        if (passed == 0 || goal_all > passed + off) {
            const int at = t.slot;
            t.slot += 2;
            if (t.rank == 0) resolve(t, n, goal, weigh, at, off, passed == 0);
            cluster_sync();
            found = t.from(0, at);
            there = t.from(0, at + 1) != 0;
        }
        if (!there) {  // the exact sums, and the same entries again
            all = over = 0;
            t.pairs([&](float l0, float l1, int p) {
                const int i = t.run.first + p;
                const bool in0 = !cutting || cut.keeps(l0, i), in1 = !cutting || cut.keeps(l1, i + 1);
                if (cutting && !__any_sync(0xffffffffu, in0 || in1)) return;
                u64 w0, w1;
                weigh.two(l0, l1, w0, w1);
                all += (in0 ? w0 : 0) + (in1 ? w1 : 0);
                over += (in0 && t.capped(l0) < from ? w0 : 0) + (in1 && t.capped(l1) < from ? w1 : 0);
            });
            t.block_sums(all, over);
            if (t.tid == 0) {
                s->pub[t.slot] = all;
                s->pub[t.slot + 1] = over;
            }
            t.meet(2);
            const u64 wanted = goal_of(top_p, t.sum(0)), before = t.sum(1);
            if (wanted <= before) return false;
            const int at = t.slot;
            t.slot += 2;
            if (t.rank == 0) resolve(t, n, wanted - before, weigh, at);
            cluster_sync();
            found = t.from(0, at);
            there = t.from(0, at + 1) != 0;
        }
        done = there && range.ba == 0 ? n : 0;
        return there;
    }
    if (n < 0) {  // too many: those of the one bin
        const int bin = pick_wide(t, goal);
        if (bin >= 0) {
            range.ba += bin << shift;
            range.bb = min(range.bb, range.ba + (1 << shift) - 1);
        }
        n = gather(t, collect_range(t, cut, range), range);
        if (n < 0) {
            found = refine(t, cut, range, goal, weigh);
            return true;
        }
    }
    const int at = t.slot;
    t.slot += 2;
    if (t.rank == 0) resolve(t, n, goal, weigh, at);
    cluster_sync();
    found = t.from(0, at);
    return true;
}

// BLOCKS: CTAs that an SM holds at once.
template <typename E, int THREADS, int BLOCKS>
__global__ void __launch_bounds__(THREADS, BLOCKS)
sample_kernel(const SampleParams p)
{
    extern __shared__ __align__(16) unsigned char raw[];
    typedef Team<E, THREADS> T;
    Shared *s = reinterpret_cast<Shared *>(raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long r = blockIdx.x / p.ctas;
    T t;
    t.s = s;
    t.blocks = reinterpret_cast<u64 *>(raw + sizeof(Shared));
    t.ctas = p.ctas;
    t.rank = static_cast<int>(cluster_ctarank());
    t.tid = tid;
    t.entries = p.V;
    E *slice = reinterpret_cast<E *>(t.blocks + (p.share + 2) / 2 * 2);  // on a 16-byte boundary
    const int count = (p.V + BLOCK - 1) / BLOCK;  // blocks of the row, shared out evenly
    const int first = static_cast<int>(static_cast<long long>(count) * t.rank / p.ctas) * BLOCK;
    const int last = min(p.V, static_cast<int>(static_cast<long long>(count) * (t.rank + 1) / p.ctas) * BLOCK);
    const E *src = static_cast<const E *>(p.logits) + r * p.ldl + first;
    const int n = max(0, last - first);
    constexpr int VEC = 16 / sizeof(E);

    const float tau0 = p.how.temperatures != nullptr ? p.how.temperatures[r] : p.how.temperature;
    const int k = p.how.top_ks != nullptr ? p.how.top_ks[r] : p.how.top_k;
    const float top_p = p.how.top_ps != nullptr ? p.how.top_ps[r] : p.how.top_p;
    const float min_p0 = p.how.min_ps != nullptr ? p.how.min_ps[r] : p.how.min_p;
    const float u = p.u[r];
    t.tau = tau0 > 0.0f ? fminf(tau0, 3.402823466e38f) : 0.0f;  // (0 times infinity would be no weight at all)
    // log2(e) / T in two parts (below 2^-127 a temperature counts as that: logits that differ by less than 1e-37 would show it)
    constexpr float kLog2e = 1.4426950408889634f, kLog2eLow = 1.4426950408889634 - static_cast<double>(kLog2e);
    const float divide = t.tau > 0.0f ? fmaxf(t.tau, 5e-39f) : 1.0f;
    const float scale = kLog2e / divide, scale_low = (fmaf(-scale, divide, kLog2e) + kLog2eLow) / divide;
    t.per_bin = fminf(128.0f / divide, 1e30f);
    // the run into shared memory, and the largest entry with the first index it has, on the way
    u64 best = 0;
    t.run.infinite = false;
    if (p.resident) {
        const int head = static_cast<int>(reinterpret_cast<uintptr_t>(src) / sizeof(E) % VEC);  // entries past a boundary
        const int lead = min(n, (VEC - head) % VEC), body = (n - lead) / VEC;
        t.run.shared = slice;
        t.run.global = nullptr;
        t.run.n = (head + n + 63) / 64 * 64;
        t.run.first = first - head;
        t.run.end = 0;
        E *dst = slice + head;
        const E least = static_cast<E>(-kInf);
        if (tid < head) slice[tid] = least;
        if (tid < 64 && head + n + tid < t.run.n) slice[head + n + tid] = least;
        const uint4 *from = reinterpret_cast<const uint4 *>(src + lead);
        uint4 *to = reinterpret_cast<uint4 *>(dst + lead);
        float high = -kInf;
        int at = -1;
        constexpr int AHEAD = 8;  // accesses that a thread has in flight
        for (int i0 = tid; i0 < body; i0 += AHEAD * THREADS) {
            uint4 v[AHEAD];
#pragma unroll
            for (int a = 0; a < AHEAD; ++a)
                if (i0 + a * THREADS < body) v[a] = __ldg(from + i0 + a * THREADS);
#pragma unroll
            for (int a = 0; a < AHEAD; ++a) {
                const int i = i0 + a * THREADS;
                if (i >= body) break;
                to[i] = v[a];
                const uint32_t w[4] = {v[a].x, v[a].y, v[a].z, v[a].w};
                float m = -kInf;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if constexpr (sizeof(E) == 4)
                        m = fmaxf(m, __uint_as_float(w[j]));
                    else
                        m = fmaxf(m, fmaxf(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xffff0000u)));
                }
                if (m > high) {
                    high = m;
                    at = i;
                }
            }
        }
        if (at >= 0) {
#pragma unroll
            for (int j = VEC - 1; j >= 0; --j) {
                const int q = lead + at * VEC + j;
                if (static_cast<float>(dst[q]) == high) best = place(high, first + q);
            }
        }
        for (int q = tid; q < n; q += THREADS) {  // the ends
            if (q >= lead && q < lead + body * VEC) {
                q += (lead + body * VEC - 1 - q) / THREADS * THREADS;
                continue;
            }
            dst[q] = src[q];
            best = max(best, place(fmaxf(static_cast<float>(src[q]), -kInf), first + q));
        }
    } else {
        t.run.shared = nullptr;
        t.run.global = src;
        t.run.n = (n + 63) / 64 * 64;
        t.run.first = first;
        t.run.end = n;
        for (int q = tid; q < n; q += THREADS) best = max(best, place(fmaxf(static_cast<float>(src[q]), -kInf), first + q));
    }
    best = warp_max(best);
    if (lane == 0) s->red[warp] = best;
    __syncthreads();
    best = warp == 0 ? warp_max(lane < T::WARPS ? s->red[lane] : 0) : 0;
    if (tid == 0) s->pub[t.slot] = best;
    t.meet(1);
    best = 0;
    for (int c = 0; c < p.ctas; ++c) best = max(best, s->all[0][c]);
    t.top = best == 0 ? -kInf : unordered(static_cast<unsigned>(best >> 32));
    int index = static_cast<int>(~static_cast<unsigned>(best));
    float logp = 0.0f;
    bool mine = tid == 0 && t.rank == 0, arrived = false;  // the thread that has the answer
    if (t.top == -kInf) {
        index = -1;
        logp = -kInf;
    } else if (t.tau > 0.0f) {
        if (t.top == kInf) {  // infinities alone have weight, 1 each
            t.top = 0.0f;
            best = place(0.0f, index);
            t.run.infinite = t.run.shared == nullptr;
            if (t.run.shared != nullptr) {
                __syncthreads();
                for (int q = tid; q < t.run.n; q += THREADS)
                    slice[q] = static_cast<E>(static_cast<float>(slice[q]) == kInf ? 0.0f : -kInf);
                __syncthreads();
            }
        }
        const Weigh weigh{t.top, scale, scale_low, p.drop};
        const bool fast = rough_can(t.tau, t.top, scale);
        const Rough rough(t.top, scale, scale_low, p.drop);
        const u64 one = 1ull << (Q - p.drop);
        u64 cut = 0, least = 1;
        int done = 0;
        if (top_p <= 0.0f) {
            cut = best;
        } else {
            if (k > 0 && k < p.V) cut = select_count(t, static_cast<unsigned>(k), top_p, weigh, done);
            if (top_p < 1.0f && done == 0) {
                const Cut from = cut != 0 ? cut_at(cut) : Cut{-kInf, 0x7fffffff};
                const bool cutting = cut != 0;
                if (!fast || !select_mass<true>(t, cutting, from, top_p, rough, weigh, cut, done))
                    select_mass<false>(t, cutting, from, top_p, weigh, weigh, cut, done);
            }
        }
        if (min_p0 > 0.0f) {
            bool more = false;
            least = min_p0 < 1.0f ? share_of(min_p0, one, more) : one;
            least += more;
        }
        auto target = [&](u64 sum) {
            bool more;
            return u > 0.0f ? u < 1.0f ? share_of(u, sum, more) : sum - 1 : 0;
        };
        u64 w = 0, all = 0;
        bool sure = false;
        if (done != 0) {
            __syncwarp();
            cluster_arrive();  // nobody reads another CTA's memory from here on
            index = -1;
            if (t.rank == 0) finish(t, done, cut, least, weigh, target, index, w, all);
        } else if (cut == 0 && least <= 1) {
            const auto exact = [&](float l0, float l1, int, u64 &w0, u64 &w1) { weigh.two(l0, l1, w0, w1); };
            const auto quick = [&](float l0, float l1, int) { return rough.two(l0, l1); };
            sure = fast && find<false, true>(t, quick, exact, target, index, w, all);
            if (!sure) find<true, false>(t, exact, exact, target, index, w, all);
        } else {
            const Cut kept = cut != 0 ? cut_at(cut) : Cut{-kInf, 0x7fffffff};
            // a rough weight may be on the other side of min_p (and least is rounded here)
            const float border = static_cast<float>(least), doubt = border * (1.0f / 1048576.0f) + 2.0f;
            const auto exact = [&](float l0, float l1, int i, u64 &w0, u64 &w1) {
                w0 = w1 = 0;
                if (!__any_sync(0xffffffffu, l0 >= kept.l || l1 >= kept.l)) return;
                u64 x0, x1;
                weigh.two(l0, l1, x0, x1);
                w0 = kept.keeps(l0, i) && x0 >= least ? x0 : 0;
                w1 = kept.keeps(l1, i + 1) && x1 >= least ? x1 : 0;
            };
            const auto quick = [&](float l0, float l1, int i) -> u64 {
                if (!__any_sync(0xffffffffu, l0 >= kept.l || l1 >= kept.l)) return 0;
                float y0, y1;
                unpack_f32x2(rough.two(l0, l1), y0, y1);
                bool in0 = kept.keeps(l0, i), in1 = kept.keeps(l1, i + 1);
                if (least > 1) {
                    bool most0 = y0 >= border, most1 = y1 >= border;
                    if (__any_sync(0xffffffffu, fabsf(y0 - border) <= doubt || fabsf(y1 - border) <= doubt)) {
                        u64 x0, x1;
                        weigh.two(l0, l1, x0, x1);
                        most0 = x0 >= least;
                        most1 = x1 >= least;
                    }
                    in0 = in0 && most0;
                    in1 = in1 && most1;
                }
                return pack_f32x2(in0 ? y0 : 0.0f, in1 ? y1 : 0.0f);
            };
            sure = fast && find<false, true>(t, quick, exact, target, index, w, all);
            if (!sure) find<true, false>(t, exact, exact, target, index, w, all);
        }
        if (sure) {  // every CTA knows
            index = mine ? index : -1;
            __syncwarp();
            cluster_arrive();
        }
        arrived = true;
        mine = index >= 0 || (all == 0 && mine);
        // (in FP32, whose functions take a tenth of the time; of a token that has most of the mass from the rest's share)
        if (mine && p.logp != nullptr)
            logp = all == 0 ? -kInf
                   : 2 * w > all ? log1pf(-static_cast<float>(all - w) / static_cast<float>(all))
                                 : logf(static_cast<float>(w) / static_cast<float>(all));
    }
    if (mine) {
        p.ids[r] = index;
        if (p.logp != nullptr) p.logp[r] = logp;
    }
    __syncwarp();
    if (!arrived) cluster_arrive();
    cluster_wait();  // no CTA leaves while another may read its shared memory
}

// Shared memory of a CTA's share of a row: small ones are taken by 256 threads, three CTAs to an SM, others by 512 (64 rows of
// 131072 in FP32, eight CTAs of 64 KB, 512 threads against 256: top-p 114 and 131 us, top 50 46 and 46, unfiltered 36 and 35).
constexpr int kSmallBytes = 53 << 10, kMostBytes = 192 << 10;
constexpr size_t kSmBytes = 228 << 10;  // of an SM, 1 KB of which each CTA on it takes besides its own

template <typename E, int THREADS, int BLOCKS>
cudaError_t launch(const SampleParams &p, size_t smem, cudaStream_t stream)
{
    // (always the same value: two handles may be at it at once)
    constexpr int kResident = kMostBytes + (kMostBytes / (BLOCK * sizeof(E)) + 2) * sizeof(u64);
    constexpr int kFar = (SGEMM_SAMPLE_MAX_VOCAB / BLOCK / MAX_CTAS + 2) * sizeof(u64);
    constexpr int kMostSmem = sizeof(Shared) + (kResident > kFar ? kResident : kFar);
    static_assert(kMostSmem <= 227 * 1024, "shared memory per CTA");
    const cudaError_t e = cudaFuncSetAttribute(sample_kernel<E, THREADS, BLOCKS>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostSmem);
    if (e != cudaSuccess) return e;
    return launch_kernel_cluster(false, p.ctas, sample_kernel<E, THREADS, BLOCKS>, dim3(static_cast<unsigned>(p.T) * p.ctas), dim3(THREADS),
                                 smem, stream, p);
}

template <typename E>
cudaError_t launch_typed(SampleParams p, int num_sms, cudaStream_t stream)
{
    const int count = (p.V + BLOCK - 1) / BLOCK;
    const long long bytes = static_cast<long long>(p.V) * sizeof(E);
    // Clusters as large as a row's shared memory asks for, and larger where there are few rows (32768 in bfloat16 with top-k and
    // top-p, in us, by 1 / 2 / 4 / 8 CTAs: 1 row 24.7 / 24.3 / 19.1 / 17.1, 16 rows 24.7 / 24.5 / 19.5 / 18.1, 64 rows 25.0 /
    // 24.7 / 21.5 / 33.5, 128 rows 25.2 / 27.5 / 38.0 / 50.1).
    p.ctas = 1;
    while (p.ctas < MAX_CTAS && p.ctas < count &&
           (bytes > static_cast<long long>(kSmallBytes) * p.ctas || 2LL * p.T * p.ctas <= num_sms))
        p.ctas *= 2;
    p.share = (count + p.ctas - 1) / p.ctas;
    const long long share_bytes = (static_cast<long long>(p.share) * BLOCK + 64 + 16 / sizeof(E)) * sizeof(E);
    p.resident = share_bytes <= kMostBytes;
    p.drop = 0;
    for (long long most = 1LL << 18; most < p.V; most <<= 1) ++p.drop;
    const size_t smem = sizeof(Shared) + static_cast<size_t>(p.share + 2) / 2 * 16 + (p.resident ? share_bytes : 0);
    if (share_bytes > kSmallBytes + 1024) return launch<E, 512, 2>(p, smem, stream);
    // Four to an SM, on 64 registers instead of 80, where that spares a round of them: 64 rows of 131072 in bfloat16, 512 CTAs of 32 KB,
    // top 50 43 -> 34 us, top-p 102 -> 79; where it spares none the spilled registers cost 3 to 8 % (512 rows of 50021 in
    // FP32, top 50 117 and 121 us).
    const long long all = static_cast<long long>(p.T) * p.ctas;
    const bool four = all > 3LL * num_sms && all <= 4LL * num_sms && 4 * (smem + 1024) <= kSmBytes;
    return four ? launch<E, 256, 4>(p, smem, stream) : launch<E, 256, 3>(p, smem, stream);
}

}  // namespace

cudaError_t launch_sample(SampleParams p, int dtype, int num_sms, cudaStream_t stream)
{
    return dtype == SGEMM_DTYPE_BF16 ? launch_typed<__nv_bfloat16>(p, num_sms, stream) : launch_typed<float>(p, num_sms, stream);
}

}  // namespace sgemm_impl
