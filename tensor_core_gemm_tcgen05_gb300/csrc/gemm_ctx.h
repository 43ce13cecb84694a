// Host-side state and helpers shared by the translation units of the C ABI (gemm_api.cu,
// serving_api.cu).
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "gemm.h"

namespace gb300_host {

constexpr uint64_t kDefaultTimeoutNs = 2000000000ull;
constexpr int kSoftmaxClusterMax = 8;   // softmax: clusters of 1, 2, 4 or 8 CTAs per row block
// gemm_run_host splits C into at most this many bands (column bands: also two row halves of
// A when A is at least kHostChunkMinBytes) whose uploads, GEMMs and downloads overlap;
// outputs smaller than kHostChunkMinBytes are not split.
constexpr int kHostChunksMax = 8;

}  // namespace gb300_host

struct gemm_ctx {
    int device = -1;
    int num_sms = 0;
    PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
    bool pair1w_ok = false;   // the one-wave pair instance runs as many clusters at once
    uint32_t *d_err = nullptr;
    uint64_t timeout_ns = gb300_host::kDefaultTimeoutNs;
    int debug = 0;
    int last_cuda_error = 0;
    int max_clusters = 0;   // co-resident CTA pairs of the pair kernel (0: pair kernel unusable)
    // stream-K workspace: one FP32 128 x 256 partial accumulator per SM, and per SM one
    // ready flag per epilogue warp (zero between launches)
    float *sk_ws = nullptr;
    uint32_t *sk_flags = nullptr;
    // softmax kernel: co-resident clusters of cs = 1, 2, 4, 8 CTAs (0: that size cannot be
    // scheduled; cs = 1 must be possible for the softmax epilogue to be offered at all)
    int softmax_clusters[gb300_host::kSoftmaxClusterMax + 1] = {};
    // split-K: co-resident clusters of 2, 4 and 8 CTAs of the split-K instance, per size
    int split_clusters[9] = {};
    // gemm_run_host: device staging buffers, two copy streams and the events that order
    // the chunked pipeline (created on first use)
    void *stage = nullptr;
    size_t stage_bytes = 0;
    cudaStream_t copy_in = nullptr, copy_out = nullptr;
    cudaEvent_t ev_start = nullptr, ev_done = nullptr;
    cudaEvent_t ev_in[2 * gb300_host::kHostChunksMax] = {}, ev_mm[2 * gb300_host::kHostChunksMax] = {};
};

namespace gb300_host {

// Make `device` current for the lifetime of the guard, then restore the caller's device.
class DeviceGuard {
  public:
    explicit DeviceGuard(int device)
    {
        if (cudaGetDevice(&prev_) != cudaSuccess) {
            cudaGetLastError();
            prev_ = -1;
        }
        if (prev_ != device)
            cudaSetDevice(device);
    }
    ~DeviceGuard()
    {
        int cur = -1;
        if (prev_ >= 0 && cudaGetDevice(&cur) == cudaSuccess && cur != prev_)
            cudaSetDevice(prev_);
    }

  private:
    int prev_ = -1;
};

inline int cuda_fail(gemm_ctx *ctx, cudaError_t e, int code)
{
    if (ctx)
        ctx->last_cuda_error = static_cast<int>(e);
    cudaGetLastError();   // clear the sticky-free error state
    return code;
}

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// True when p is device (or managed) memory that `device` can address directly.
inline bool on_device(const void *p, int device)
{
    cudaPointerAttributes a;
    if (cudaPointerGetAttributes(&a, p) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    if (a.type == cudaMemoryTypeManaged)
        return true;
    return a.type == cudaMemoryTypeDevice && a.device == device;
}

inline bool overlaps(const void *a, size_t na, const void *b, size_t nb)
{
    if (!a || !b || na == 0 || nb == 0)
        return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
    return a0 < b0 + nb && b0 < a0 + na;
}

// Sets the attributes of the serving kernels (serving_api.cu); called by gemm_create.
cudaError_t serving_init(gemm_ctx *ctx);

}  // namespace gb300_host
