// C ABI of the global norm and clipping: argument checks, the tensors' tables,
// launches. Declarations and contracts: include/sgemm_clip.h.
#include <algorithm>
#include <cstdint>
#include <new>
#include <vector>

#include <cuda_runtime.h>

#include "clip_internal.h"
#include "handle.h"
#include "sgemm_internal.h"

using namespace sgemm_impl;

namespace {

// Of the 129 MB of L2, what is read last in the first kernel and first in the second (bfloat16 with outputs, in us, keeping 0 / 40 /
// 80 / 110 MB: 38 MB 22.4 / 20.8 / 20.9 / 20.9, 114 MB 61.6 / 57.7 / 59.8 / 63.0, 476 MB 242.5 / 240.1 / 240.8 / 242.8).
constexpr long long kKeptBytes = 40LL << 20;

bool aligned(const void *p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

int check(const sgemm_tensor_t &t)
{
    if (t.dtype != SGEMM_DTYPE_F32 && t.dtype != SGEMM_DTYPE_BF16) return SGEMM_ERR_INVALID_VALUE;
    if (t.rows < 0 || t.cols < 0) return SGEMM_ERR_INVALID_VALUE;
    if (t.rows == 0 || t.cols == 0) return SGEMM_OK;
    const unsigned size = t.dtype == SGEMM_DTYPE_BF16 ? 2 : 4;
    if (t.data == nullptr || !aligned(t.data, size) || !aligned(t.out, size)) return SGEMM_ERR_INVALID_VALUE;
    if (t.rows > 1 && (t.ld < t.cols || (t.out != nullptr && t.ld_out < t.cols))) return SGEMM_ERR_INVALID_VALUE;
    if (t.out == t.data && t.rows > 1 && t.ld_out != t.ld) return SGEMM_ERR_INVALID_VALUE;  // rows over each other
    // every offset counts in 64 bits
    const long long most = 1LL << 60, ld = std::max(t.ld, t.out != nullptr ? t.ld_out : 0);
    if (t.cols > most || (t.rows > 1 && (ld > most || t.rows > most / ld))) return SGEMM_ERR_INVALID_VALUE;
    return SGEMM_OK;
}

// A tensor as the kernels take it, but for its chunks.
ClipTensor describe(const sgemm_tensor_t &t)
{
    ClipTensor d{};
    const unsigned size = t.dtype == SGEMM_DTYPE_BF16 ? 2 : 4;
    d.data = t.data;
    d.in_place = t.out == nullptr;
    d.out = d.in_place ? const_cast<void *>(t.data) : t.out;
    d.rows = t.rows;
    d.cols = t.cols;
    d.ld = t.rows > 1 ? t.ld : t.cols;
    d.ld_out = t.rows <= 1 ? t.cols : d.in_place ? t.ld : t.ld_out;
    if (t.rows > 1 && d.ld == t.cols && d.ld_out == t.cols) {  // packed: one long row
        d.cols = t.rows * t.cols;
        d.rows = 1;
        d.ld = d.ld_out = d.cols;
    }
    d.dtype = static_cast<short>(t.dtype);
    const long long group = 16 / size;
    d.vec = aligned(d.data, 16) && aligned(d.out, 16) && d.cols % group == 0 &&
            (d.rows == 1 || (d.ld % group == 0 && d.ld_out % group == 0));
    return d;
}

// Its chunks of `chunk` elements; more than there can be where they do not count in 32 bits.
long long cut(ClipTensor *d, int chunk)
{
    const long long row_chunks = (d->cols + chunk - 1) / chunk;
    if (row_chunks > 1 << 30) return 1LL << 40;
    d->chunk_rows = row_chunks > 1 ? 1 : static_cast<int>(std::min<long long>(chunk / d->cols, d->rows));
    d->row_chunks = static_cast<int>(row_chunks);
    return row_chunks > 1 ? d->rows * row_chunks : (d->rows + d->chunk_rows - 1) / d->chunk_rows;
}

// All tables of a call, N tensors in each, through both kernels.
template <int N>
int run(sgemm_handle_t h, const std::vector<ClipTensor> &all, const std::vector<int> &chunks, int chunk, float max_norm,
        float *norm, cudaStream_t stream)
{
    double *part = static_cast<double *>(h->workspace);
    const int count = static_cast<int>(all.size()), tables = std::max(1, (count + N - 1) / N);
    const int most = kClipBlocks * h->num_sms;
    std::vector<int> blocks(tables);
    ClipTable<N> table;
    auto fill = [&](int i) {
        table.count = std::min(N, count - i * N);
        table.chunks = 0;
        table.chunk = chunk;
        long long kept = kKeptBytes;
        for (int j = 0; j < table.count; ++j) {
            table.t[j] = all[i * N + j];
            table.t[j].first = table.chunks;
            table.chunks += chunks[i * N + j];
        }
        table.stream = table.chunks;  // the last kKeptBytes stay in the L2 (of the last table; of earlier ones what fits)
        for (int j = table.count - 1; j >= 0 && kept > 0; --j) {
            const int size = table.t[j].dtype == SGEMM_DTYPE_BF16 ? 2 : 4;
            const long long n = chunks[i * N + j], each = std::max(1LL, table.t[j].rows * table.t[j].cols * size / n);
            const long long some = std::min(n, kept / each + 1);
            table.stream -= static_cast<int>(some);
            kept -= some * each;
        }
    };
    int parts = 0;
    for (int i = 0; i < tables; ++i) {
        fill(i);
        if (table.count == 0) break;  // no elements at all
        blocks[i] = std::min(table.chunks, most);
        if (launch_clip_norm<N>(table, blocks[i], part + parts, stream) != cudaSuccess) return SGEMM_ERR_LAUNCH;
        parts += blocks[i];
    }
    for (int i = tables - 1; i >= 0; --i) {
        if (tables > 1) fill(i);
        if (launch_clip_scale<N>(table, std::max(1, blocks[i]), part, parts, max_norm, i == 0 ? norm : nullptr,
                                 parts > 0 && i == tables - 1, stream) != cudaSuccess)
            return SGEMM_ERR_LAUNCH;
    }
    return SGEMM_OK;
}

}  // namespace

extern "C" {

int sgemm_clip_workspace(int count, long long *bytes)
{
    if (count < 0 || bytes == nullptr) return SGEMM_ERR_INVALID_VALUE;
    // one sum per block and table, on a machine of up to 256 SMs
    const long long tables = std::max(1, (count + kClipMany - 1) / kClipMany);
    *bytes = tables * kClipBlocks * 256 * static_cast<long long>(sizeof(double));
    return SGEMM_OK;
}

int sgemm_clip(sgemm_handle_s *h, int count, const sgemm_tensor_t *tensors, float max_norm, float *norm, CUstream_st *stream)
{
    if (h == nullptr || count < 0 || (count > 0 && tensors == nullptr) || norm == nullptr || !elem_aligned(norm) ||
        !(max_norm >= 0.0f))
        return SGEMM_ERR_INVALID_VALUE;
    for (int i = 0; i < count; ++i) {
        const int rc = check(tensors[i]);
        if (rc != SGEMM_OK) return rc;
    }
    try {
        std::vector<ClipTensor> all;
        std::vector<int> chunks;
        std::vector<const void *> firsts;  // first elements of tensors and of outputs of their own
        double elements = 0.0;
        for (int i = 0; i < count; ++i) {
            const sgemm_tensor_t &t = tensors[i];
            if (t.rows == 0 || t.cols == 0) continue;
            all.push_back(describe(t));
            firsts.push_back(t.data);
            if (all.back().out != t.data) firsts.push_back(all.back().out);
            elements += static_cast<double>(t.rows) * static_cast<double>(t.cols);
        }
        int chunk = kClipMost;
        while (chunk > kClipLeast && elements < static_cast<double>(chunk) * kClipBlocks * h->num_sms) chunk /= 2;
        long long total = 0;
        for (ClipTensor &d : all) {
            const long long n = cut(&d, chunk);
            total += n;
            if (total > 1LL << 30) return SGEMM_ERR_NOT_SUPPORTED;  // chunks are counted in 32 bits
            chunks.push_back(static_cast<int>(n));
        }
        std::sort(firsts.begin(), firsts.end());
        if (std::adjacent_find(firsts.begin(), firsts.end()) != firsts.end()) return SGEMM_ERR_INVALID_VALUE;
        DeviceGuard g(h->device);
        if (!g.ok) return SGEMM_ERR_CUDA;
        long long bytes = 0;
        sgemm_clip_workspace(static_cast<int>(all.size()), &bytes);
        const int rc = ensure_workspace(h, static_cast<size_t>(bytes), stream);
        if (rc != SGEMM_OK) return rc;
        return all.size() <= kClipFew ? run<kClipFew>(h, all, chunks, chunk, max_norm, norm, stream)
                                      : run<kClipMany>(h, all, chunks, chunk, max_norm, norm, stream);
    } catch (const std::bad_alloc &) {
        return SGEMM_ERR_ALLOC;
    }
}

}  // extern "C"
