// What a caller needs to know of stream capture to keep memory for a captured
// graph as long as the graph lives (pa_capture_*; host only).
#include <cuda_runtime.h>

#include <atomic>
#include <new>

#include "pa_launch.cuh"
#include "pagedattn.h"

// Shared by the caller and the graph: the last of the two to let go frees it.
struct pa_capture {
    std::atomic<int> holders{2};
    std::atomic<int> alive{1};
    void let_go() {
        if (holders.fetch_sub(1, std::memory_order_acq_rel) == 1) delete this;
    }
};

namespace {

// Called by the driver once the graph and all that was made from it are gone
// and their launches complete (on a thread that may not call CUDA).
void CUDART_CB graph_gone(void* c) {
    static_cast<pa_capture*>(c)->alive.store(0, std::memory_order_release);
    static_cast<pa_capture*>(c)->let_go();
}

pa_status cuda_fail(const char* fmt, cudaError_t e) {
    (void)cudaGetLastError();  // do not leave the error for an unrelated later call
    return pa::fail(PA_ERR_CUDA, fmt, cudaGetErrorString(e));
}

}  // namespace

extern "C" pa_status pa_capture_id(void* stream, uint64_t* id) {
    pa::clear_detail();
    if (!id) return pa::fail(PA_ERR_INVALID_ARG, "%s", "id is NULL");
    *id = 0;
    cudaStreamCaptureStatus st = cudaStreamCaptureStatusNone;
    unsigned long long n = 0;
    const cudaError_t e = cudaStreamGetCaptureInfo(static_cast<cudaStream_t>(stream), &st, &n);
    if (e != cudaSuccess) return cuda_fail("capture info: %s", e);
    if (st != cudaStreamCaptureStatusNone) *id = n;
    return PA_OK;
}

extern "C" pa_status pa_capture_watch(void* stream, pa_capture** out) {
    pa::clear_detail();
    if (!out) return pa::fail(PA_ERR_INVALID_ARG, "%s", "out is NULL");
    *out = nullptr;
    cudaStreamCaptureStatus st = cudaStreamCaptureStatusNone;
    cudaGraph_t graph = nullptr;
    cudaError_t e =
        cudaStreamGetCaptureInfo(static_cast<cudaStream_t>(stream), &st, nullptr, &graph);
    if (e != cudaSuccess) return cuda_fail("capture info: %s", e);
    if (st != cudaStreamCaptureStatusActive)
        return pa::fail(PA_ERR_INVALID_ARG, "%s", "the stream is not being captured");
    pa_capture* c = new (std::nothrow) pa_capture;
    if (!c) return pa::fail(PA_ERR_CUDA, "%s", "out of host memory");
    cudaUserObject_t obj = nullptr;
    e = cudaUserObjectCreate(&obj, c, graph_gone, 1, cudaUserObjectNoDestructorSync);
    if (e != cudaSuccess) {
        delete c;
        return cuda_fail("user object: %s", e);
    }
    e = cudaGraphRetainUserObject(graph, obj, 1, cudaGraphUserObjectMove);
    if (e != cudaSuccess) {
        c->let_go();                          // the caller's share ...
        (void)cudaUserObjectRelease(obj, 1);  // ... and the graph's, by graph_gone
        return cuda_fail("user object: %s", e);
    }
    *out = c;
    return PA_OK;
}

extern "C" int pa_capture_alive(const pa_capture* c) {
    return c ? c->alive.load(std::memory_order_acquire) : 0;
}

extern "C" void pa_capture_free(pa_capture* c) {
    if (c) c->let_go();
}

extern "C" pa_status pa_capture_mode(int* mode) {
    pa::clear_detail();
    if (!mode) return pa::fail(PA_ERR_INVALID_ARG, "%s", "mode is NULL");
    if (*mode < 0 || *mode > 2) return pa::fail(PA_ERR_INVALID_ARG, "%s", "mode must be 0, 1 or 2");
    cudaStreamCaptureMode m = static_cast<cudaStreamCaptureMode>(*mode);
    const cudaError_t e = cudaThreadExchangeStreamCaptureMode(&m);
    if (e != cudaSuccess) return cuda_fail("capture mode: %s", e);
    *mode = static_cast<int>(m);
    return PA_OK;
}
