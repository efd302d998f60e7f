// The library's host code (handle, planning, entry points) with a CUDA runtime and
// kernels that only pretend: for tests of what the host does when a part of the
// machine is not as on a GB300, without a GPU. Built and run by
// tests/test_vocab_host.py. Memory "on the device" is host memory that nobody reads.
#include <cstdio>
#include <cstdlib>
#include <cstring>

#include "../dense_fp32_gemm_04_gb300/csrc/handle.h"
#include "../dense_fp32_gemm_04_gb300/csrc/sgemm_internal.h"
#include "../dense_fp32_gemm_04_gb300/csrc/vocab_internal.h"

static int g_sms = 152, g_pairs = 76;
static cudaError_t g_attributes = cudaSuccess;
static size_t g_largest = 0, g_limit = 0;
static int g_launches = 0;

extern "C" {
cudaError_t cudaGetDeviceCount(int *n) { return *n = 1, cudaSuccess; }
cudaError_t cudaGetDevice(int *d) { return *d = 0, cudaSuccess; }
cudaError_t cudaSetDevice(int) { return cudaSuccess; }
cudaError_t cudaGetLastError() { return cudaSuccess; }
cudaError_t cudaDeviceSynchronize() { return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int *v, cudaDeviceAttr a, int)
{
    *v = a == cudaDevAttrComputeCapabilityMajor ? 10 : a == cudaDevAttrComputeCapabilityMinor ? 3 : g_sms;
    return cudaSuccess;
}
cudaError_t cudaMalloc(void **p, size_t bytes)
{
    static char somewhere[1024];
    if (g_limit > 0 && bytes > g_limit) return cudaErrorMemoryAllocation;
    if (bytes > g_largest) g_largest = bytes;
    *p = somewhere;
    return cudaSuccess;
}
cudaError_t cudaFree(void *) { return cudaSuccess; }
cudaError_t cudaMemset(void *, int, size_t) { return cudaSuccess; }
cudaError_t cudaMemcpy(void *, const void *, size_t, cudaMemcpyKind) { return cudaSuccess; }
cudaError_t cudaMemcpy2DAsync(void *, size_t, const void *, size_t, size_t, size_t, cudaMemcpyKind, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaStreamIsCapturing(cudaStream_t, cudaStreamCaptureStatus *s) { return *s = cudaStreamCaptureStatusNone, cudaSuccess; }
cudaError_t cudaStreamCreateWithFlags(cudaStream_t *s, unsigned) { return *s = nullptr, cudaSuccess; }
cudaError_t cudaStreamDestroy(cudaStream_t) { return cudaSuccess; }
cudaError_t cudaStreamSynchronize(cudaStream_t) { return cudaSuccess; }
cudaError_t cudaStreamWaitEvent(cudaStream_t, cudaEvent_t, unsigned) { return cudaSuccess; }
cudaError_t cudaEventCreateWithFlags(cudaEvent_t *e, unsigned) { return *e = nullptr, cudaSuccess; }
cudaError_t cudaEventDestroy(cudaEvent_t) { return cudaSuccess; }
cudaError_t cudaEventRecord(cudaEvent_t, cudaStream_t) { return cudaSuccess; }
static CUresult encode(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                       const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                       CUtensorMapL2promotion, CUtensorMapFloatOOBfill)
{
    return CUDA_SUCCESS;
}
cudaError_t cudaGetDriverEntryPointByVersion(const char *, void **f, unsigned, unsigned long long,
                                             cudaDriverEntryPointQueryResult *r)
{
    *f = reinterpret_cast<void *>(&encode);
    if (r != nullptr) *r = cudaDriverEntryPointSuccess;
    return cudaSuccess;
}
}

namespace sgemm_impl {
cudaError_t ffma_set_attributes() { return cudaSuccess; }
cudaError_t tf32_set_attributes() { return cudaSuccess; }
int tf32_pair_max_pairs() { return g_pairs; }
size_t min2_candidate_bytes(int) { return 64; }
cudaError_t vocab_set_attributes() { return g_attributes; }
int vocab_max_pairs() { return g_pairs; }
int vocab_few_warps(int T, int num_sms) { return (T > 4 ? 8 : 16) * num_sms; }
static cudaError_t launched() { return ++g_launches, cudaSuccess; }
cudaError_t launch_scale(int, int, float, float *, long long, int, cudaStream_t) { return launched(); }
// (the GEMM's other kernels, for the linker)
cudaError_t launch_ffma(int, int, const CUtensorMap &, const CUtensorMap &, const FfmaParams &, int, cudaStream_t, bool) { return launched(); }
cudaError_t launch_tf32(const CUtensorMap &, const CUtensorMap &, const Tf32Params &, int, cudaStream_t, bool) { return launched(); }
cudaError_t launch_tf32_pair(const CUtensorMap &, const CUtensorMap &, const Tf32Params &, int, cudaStream_t, bool) { return launched(); }
cudaError_t launch_ladder(int, int, int, int, float, const float *, const float *, float, float *, cudaStream_t) { return launched(); }
cudaError_t launch_min2(const float *, long long, int, int, void *, int, float *, int *, cudaStream_t) { return launched(); }
cudaError_t launch_prep(const float *, long long, float *, long long, int, int, bool, const float *, long long, float *,
                        long long, int, int, int, cudaStream_t)
{
    return launched();
}
cudaError_t launch_repack(const float *, long long, float *, long long, int, int, int, cudaStream_t) { return launched(); }
cudaError_t launch_sk_reduce(const FfmaParams &, int, int, int, cudaStream_t) { return launched(); }
cudaError_t launch_splitk_reduce(const float *, long long, long long, int, int, int, float, float, float *, long long, int,
                                 int, cudaStream_t, long long, int *)
{
    return launched();
}
cudaError_t launch_transpose(const float *, long long, float *, long long, int, int, cudaStream_t) { return launched(); }
cudaError_t launch_vocab_targets(int, int, int, const long long *, const float *, long long, float, int *, float *, float *,
                                 bool, cudaStream_t)
{
    return launched();
}
cudaError_t launch_vocab_combine(int, int, const VocabTargets &, const float2 *, int, const float *, float, float *, float *,
                                 cudaStream_t)
{
    return launched();
}
cudaError_t launch_vocab_finish(int, int, const float *, long long, long long, int, float, void *, long long, int, bool,
                                cudaStream_t)
{
    return launched();
}
// What the debug build's checks hold the few-token kernels to is what they write: a launch that says otherwise fails.
cudaError_t launch_vocab_few(VocabFewParams p, int, bool, int num_sms, bool, cudaStream_t)
{
    const bool good = p.stat_rows == vocab_few_warps(p.T, num_sms) && p.targets == p.T * p.t.n;
    return good ? launched() : cudaErrorInvalidValue;
}
cudaError_t launch_vocab_few_targets(const VocabFewParams &p, int, bool, bool, cudaStream_t)
{
    return p.targets == p.T * p.t.n ? launched() : cudaErrorInvalidValue;
}
cudaError_t launch_vocab_tiles(const VocabMaps &, const VocabTileParams &, int, int, bool, cudaStream_t) { return launched(); }
cudaError_t launch_vocab_copy(const void *, long long, int, int, void *, long long, bool, cudaStream_t) { return launched(); }
cudaError_t launch_vocab_split(const void *, long long, int, int, void *, float *, int, float *, float *, void *, int,
                               long long, bool, cudaStream_t)
{
    return launched();
}
}  // namespace sgemm_impl

// workspace PAIRS T V D DTYPE GRADS: on a machine where PAIRS CTA pairs are resident at once, what a call still allocates
// once the plan's bytes are reserved, and the plan's and the call's launches. attributes: the status of making a handle, of a GEMM without work, of a loss and of a gradient
// where the vocabulary kernels cannot run.
int main(int argc, char **argv)
{
    if (argc > 1 && std::strcmp(argv[1], "attributes") == 0) g_attributes = cudaErrorInvalidConfiguration;
    if (argc > 2) g_pairs = std::atoi(argv[2]);
    sgemm_handle_t h = nullptr;
    const int made = sgemm_create_for_device(0, &h);
    alignas(128) static char m[1024];
    float *f = reinterpret_cast<float *>(m);
    const long long *y = reinterpret_cast<const long long *>(m);
    if (argc == 2) {
        const int gemm = h != nullptr ? sgemm_run(h, 4, 4, 0, 1.0f, f, 4, f, 4, 0.5f, f, 4, nullptr) : -1;
        const int before = g_launches;
        const int loss = sgemm_xent(h, 4, 8, 8, 0, m, 8, m, 8, y, 1.0f, f, f, nullptr);
        const int grad = sgemm_xent_grad(h, 4, 8, 8, 0, m, 8, m, 8, y, 1.0f, f, f, 0.0f, m, 8, m, 8, nullptr);
        std::printf("%d %d %d %d %d\n", made, gemm, loss, grad, g_launches - before);
        return 0;
    }
    const int T = std::atoi(argv[3]), V = std::atoi(argv[4]), D = std::atoi(argv[5]), dtype = std::atoi(argv[6]);
    const int grads = std::atoi(argv[7]);  // bits: dH, dW
    sgemm_vocab_plan_t p{};
    const int planned = sgemm_vocab_plan(T, V, D, dtype, 0, grads != 0, 15, g_sms, SGEMM_MATH_FP32, &p);
    g_limit = static_cast<size_t>(p.workspace_bytes);  // no headroom
    const int reserved = sgemm_reserve(h, static_cast<size_t>(p.workspace_bytes));
    g_limit = g_largest = 0;
    g_launches = 0;
    const int ld = (D + 63) / 64 * 64;  // rows on 128-byte lines, as the plan is told
    const int rc = grads == 0 ? sgemm_xent(h, T, V, D, dtype, m, ld, m, ld, y, 1.0f, f, f, nullptr)
                              : sgemm_xent_grad(h, T, V, D, dtype, m, ld, m, ld, y, 1.0f, f, f, 0.0f,
                                                grads & 1 ? m : nullptr, ld, grads & 2 ? m : nullptr, ld, nullptr);
    std::printf("%d %d %d %d %zu %d %d\n", made, planned, reserved, rc, g_largest, p.launches, g_launches);
    sgemm_destroy(h);
    return 0;
}
