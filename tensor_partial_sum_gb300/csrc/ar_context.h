// What the library's translation units share on the host: the process-wide
// context behind ar_init (owned by ar.cu) and the launch helper.
#pragma once

#include <cstddef>
#include <cstdint>
#include <mutex>

#include <cuda_runtime.h>

#include "ar.h"

namespace tps {

// The part of the context that a launch outside ar.cu needs.
struct CallContext {
    int R;
    size_t max_elems;
    int device;
    int sm_count;
    bool pdl;
    bool fault_inject;
    unsigned *dev_status;
};

// Guards the context; a call holds it from its checks to its last launch.
std::mutex &context_mutex();

// The current context (the caller holds context_mutex()); false before ar_init.
bool current_context(CallContext *out);

// AR_OK when the context's device is current and no launch failure is injected.
int check_launch_device(const CallContext &c);

// Bytes of an element, 0 for an unknown ar_dtype.
inline size_t dtype_bytes(int dtype) { return dtype == 0 ? 4 : (dtype == 1 || dtype == 2) ? 2 : 0; }

// Whether [a, a + na) and [b, b + nb) share a byte.
inline bool spans_overlap(const void *a, size_t na, const void *b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return na && nb && x < y + nb && y < x + na;
}

// The status of a launch, whose error is cleared.
inline int launched(cudaError_t e) {
    if (e == cudaSuccess) return AR_OK;
    cudaGetLastError();
    return AR_ERR_CUDA;
}

// Launch a kernel that runs griddepcontrol.launch_dependents and
// griddepcontrol.wait before it loads or stores anything: as a programmatic
// dependent of the kernel before it on the stream when `pdl`, else plainly.
template <typename... Params, typename... Args>
cudaError_t launch_dependent(void (*fn)(Params...), dim3 grid, unsigned threads, size_t smem, cudaStream_t stream,
                             bool pdl, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    // Not on the default streams: their implicit ordering against other
    // streams is left exactly as a plain launch has it.
    const bool default_stream = stream == nullptr || stream == cudaStreamLegacy || stream == cudaStreamPerThread;
    cfg.numAttrs = (pdl && !default_stream) ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, fn, args...);
}

}  // namespace tps
