// mla_launch.h -- launching kernels as programmatic dependents, and the checks of a
// workspace whose header alone is used: what the cache's calls and those between two
// decode steps have in common.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/mla_decode.h"

namespace mla {
namespace {

// Launches kernel as a programmatic dependent of the preceding kernel on the
// stream: it may be scheduled while that one drains and waits for its
// completion (griddepcontrol.wait) before it reads anything.
// With `overlap` false it starts only when all earlier work on the stream is
// done (after a memset, which is no kernel to depend on).
template <typename... KArgs, typename... Args>
inline cudaError_t launch_dependent_shared(void (*kernel)(KArgs...), dim3 grid, int threads,
                                           int shared, cudaStream_t stream, bool overlap,
                                           Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = (size_t)shared;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = overlap ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

// The same without dynamic shared memory.
template <typename... KArgs, typename... Args>
inline cudaError_t launch_dependent(void (*kernel)(KArgs...), dim3 grid, int threads,
                                    cudaStream_t stream, bool overlap, Args... args)
{
    return launch_dependent_shared(kernel, grid, threads, 0, stream, overlap, args...);
}

__device__ __forceinline__ void wait_for_predecessor()
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

__device__ __forceinline__ void allow_dependents()
{
    asm volatile("griddepcontrol.launch_dependents;");
}

inline int64_t align256(int64_t n) { return (n + 255) / 256 * 256; }

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline int check_header(const void* ws, int64_t bytes)
{
    if (!ws) return MLA_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return MLA_ERR_MISALIGNED;
    return bytes < MLA_WORKSPACE_HEADER_BYTES ? MLA_ERR_WORKSPACE_TOO_SMALL : MLA_OK;
}

inline int status_of(cudaError_t e) { return e == cudaSuccess ? MLA_OK : MLA_ERR_LAUNCH_FAILED; }

}  // namespace
}  // namespace mla
