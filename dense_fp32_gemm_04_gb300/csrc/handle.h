// The library handle and what every entry point does with it: bind its device,
// grow its workspace. Shared by the files that implement the C ABI; not installed.
#pragma once

#include <cstddef>
#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/sgemm.h"
#include "planner.h"

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

struct sgemm_handle_s {
    int device = 0;
    int num_sms = 0;
    int tf32_pairs = -1;  // CTA pairs of the TF32 pair kernel resident at once (-1: none fit)
    int vocab_pairs = -1; // the same for the vocabulary losses' kernel
    bool vocab_ok = false; // that kernel can run (without it the other calls still do)
    int vocab_piece = 0;  // SGEMM_OPT_FORCE_VOCAB_PIECE
    int math_mode = SGEMM_MATH_FP32;
    int *d_status = nullptr;
    void *workspace = nullptr;
    size_t ws_bytes = 0;
    float *stage = nullptr;  // sgemm_run_host device copies of A | B | C
    size_t stage_bytes = 0;
    sgemm_impl::Overrides ov;
    int inject_skip = -1;
    int skew_ns = 0;
    int log = 0;
    long long timeout_ns = 4000000000LL;
    sgemm_plan_t last{};
    EncodeTiledFn encode = nullptr;
    // sgemm_run_host pipeline: copy-in and copy-out streams and their events.
    cudaStream_t h2d = nullptr, d2h = nullptr;
    cudaEvent_t ev_start = nullptr, ev_end = nullptr;
    cudaEvent_t ev_in[12] = {}, ev_done[12] = {};  // one pair per pipeline step
    void *min2_cand = nullptr;  // sgemm_run_min2 per-block candidates
};

namespace sgemm_impl {

// Bind the handle's device for the duration of a call.
struct DeviceGuard {
    int prev = -1;
    bool ok = true;
    explicit DeviceGuard(int dev)
    {
        if (cudaGetDevice(&prev) != cudaSuccess) {
            ok = false;
            return;
        }
        if (prev != dev && cudaSetDevice(dev) != cudaSuccess) ok = false;
    }
    ~DeviceGuard()
    {
        int cur = -1;
        if (prev >= 0 && cudaGetDevice(&cur) == cudaSuccess && cur != prev) cudaSetDevice(prev);
    }
};

// Grow the handle's workspace to at least `bytes`. Growing synchronizes the
// device and reallocates, which a stream capture forbids: while `stream` is being
// captured, a workspace that is too small is SGEMM_ERR_NOT_SUPPORTED and nothing
// is called (size it first, with sgemm_reserve or an uncaptured call).
int ensure_workspace(sgemm_handle_t h, size_t bytes, cudaStream_t stream);

}  // namespace sgemm_impl
