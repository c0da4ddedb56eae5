// cpa_launch.cuh -- the status word and the launches of calls whose workspace holds
// nothing else: page operations, and rows written to pages and read back.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "cpa.h"
#include "cpa_checks.h"

namespace cpa {
namespace {

__device__ __forceinline__ void flag(uint32_t* status, uint32_t bit) { atomicOr(status, bit); }

// Clears the status word for the kernel after it, which is launched while this one
// runs and waits for it on the device (a memset in its place cost 3.5 us of a
// captured call).
__global__ void clear_kernel(uint32_t* status) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    *status = 0u;
}
__device__ __forceinline__ void wait_for_clear() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

// All that a call with nothing to do does.
inline cpa_status clear_status(void* workspace, cudaStream_t s) {
    return cudaMemsetAsync(workspace, 0, 4, s) == cudaSuccess ? CPA_OK : CPA_ERR_CUDA;
}

inline cpa_status status_ws(const void* workspace, size_t bytes) {
    if (!workspace || bytes < kStatusBytes) return CPA_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(workspace) & 3u) return CPA_ERR_INVALID_ARG;
    return CPA_OK;
}

inline cpa_status launched() { return cudaGetLastError() == cudaSuccess ? CPA_OK : CPA_ERR_LAUNCH; }

// Launches a kernel that may start while the one before it on the stream runs.
template <class... P, class... A>
cpa_status launch_dependent(void (*kernel)(P...), dim3 grid, int threads, cudaStream_t s, A... args) {
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, (P)args...) == cudaSuccess ? CPA_OK : CPA_ERR_LAUNCH;
}

// A kernel that begins with a cleared status word.
template <class... P, class... A>
cpa_status launch_cleared(void (*kernel)(P...), dim3 grid, int threads, cudaStream_t s,
                          uint32_t* status, A... args) {
    clear_kernel<<<1, 1, 0, s>>>(status);
    const cpa_status st = launched();
    return st != CPA_OK ? st : launch_dependent(kernel, grid, threads, s, args...);
}

}  // namespace
}  // namespace cpa
