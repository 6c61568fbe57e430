// Host-side launch helpers shared by the library's sources.
#pragma once

#include <cuda_runtime.h>

#include <atomic>

#include "pa_decode_kernels.cuh"
#include "pagedattn.h"

namespace pa {

// Notes what is wrong with a call for pa_last_error_detail and returns st.
pa_status fail(pa_status st, const char* fmt, const char* what);
void clear_detail();

inline bool aligned(const void* ptr, size_t a) {
    return (reinterpret_cast<uintptr_t>(ptr) % a) == 0;
}

inline int elem_bytes(pa_kv_dtype t) { return t == PA_KV_BF16 ? 2 : 1; }

// Codes with a scale per (block, kv head).
inline bool block_scales(pa_kv_dtype t) {
    return t == PA_KV_FP8_E4M3_BLOCK || t == PA_KV_INT8_BLOCK;
}

constexpr size_t kMaxSmemPerCta = 227 * 1024;  // opt-in limit of sm_100
constexpr size_t kStaticSmemReserve = 256;     // a kernel's own __shared__ variables
constexpr int kMaxDevices = 64;

// SM count of the current device (cached per device); 0 on success.
inline int device_sms(int* out) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return -1;
    static std::atomic<int> cache[kMaxDevices];
    if (dev >= 0 && dev < kMaxDevices) {
        int v = cache[dev].load(std::memory_order_relaxed);
        if (v > 0) {
            *out = v;
            return 0;
        }
    }
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
        return -1;
    if (dev >= 0 && dev < kMaxDevices) cache[dev].store(n, std::memory_order_relaxed);
    *out = n;
    return 0;
}

// Raise the kernel's dynamic shared-memory limit once per device.  `done` is
// owned by the caller's template instantiation, so every kernel variant keeps
// its own flags.
template <typename K>
cudaError_t ensure_smem(K kernel, std::atomic<int>* done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool cached = dev >= 0 && dev < kMaxDevices;
    if (cached && done[dev].load(std::memory_order_acquire)) return cudaSuccess;
    // The opt-in limit covers static and dynamic shared memory together.
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, kernel);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(kMaxSmemPerCta - fa.sharedSizeBytes));
    if (e != cudaSuccess) {
        (void)cudaGetLastError();  // do not leave the error for an unrelated later call
        return e;
    }
    if (cached) done[dev].store(1, std::memory_order_release);
    return e;
}

// Launch with programmatic stream serialization: the kernel may be scheduled
// while the kernel ahead of it in the stream drains, which hides the launch
// gap between back-to-back calls and between decode and combine.  Every
// kernel launched this way waits (griddepcontrol.wait) before touching memory,
// so stream order is kept for everything it reads and writes.
template <typename... Params>
cudaError_t launch_pdl(void (*kern)(Params...), dim3 grid, unsigned block, size_t smem,
                       cudaStream_t st, const Params&... p) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kern, p...);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <int D, int B, bool FP8, int NH, bool F8MMA, bool SC = false,
          int CODES = kE4m3Tensor>
cudaError_t launch_decode(const DecodeParams& p, long long grid, size_t smem,
                          cudaStream_t st) {
    static std::atomic<int> done[kMaxDevices];
    constexpr int W = decode_warps<D, B, FP8>();
    auto kern = pa_decode_kernel<D, B, FP8, NH, W, F8MMA, SC, CODES>;
    if (smem > kMaxSmemPerCta - kStaticSmemReserve) return cudaErrorInvalidValue;
    cudaError_t e = ensure_smem(kern, done);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, static_cast<unsigned>(grid), W * 32, smem, st, p);
}

// Decode over 8-bit pages with block scales (pa_decode_block.cu).
cudaError_t launch_decode_block(const DecodeParams& p, int D, int B, bool int8, long long grid,
                                size_t smem, cudaStream_t st);

}  // namespace pa
