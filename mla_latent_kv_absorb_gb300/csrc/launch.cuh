// launch.cuh -- host helpers of the translation units beside api.cu: pointer checks, programmatic
// dependent launches and the record of a failed launch.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstdio>
#include <utility>

#include "../../include/mla.h"

namespace mla {

void set_last_error_text(const char* text);

// A tiled map of bf16 with 128-byte swizzle; dims and strides innermost first, strides in bytes for dims
// 1.. (defined in api.cu).
bool make_bf16_map(CUtensorMap* m, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
                   const cuuint32_t* box);

inline bool is_aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline mla_status cuda_status(cudaError_t e, const char* where)
{
    if (e == cudaSuccess) return MLA_OK;
    char msg[200];
    snprintf(msg, sizeof msg, "%s: %s (%s)", where, cudaGetErrorString(e), cudaGetErrorName(e));
    set_last_error_text(msg);
    return MLA_ERR_CUDA;
}

// The kernel may be scheduled while the kernel ahead of it in the stream still runs; it waits for
// that kernel's end itself (griddepcontrol.wait) before it touches any caller memory.
template <typename... KArgs, typename... Args>
mla_status launch_dependent(const char* where, void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                            void* stream, Args&&... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cuda_status(cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...), where);
}

// True when the elements [a][b][0..width) at a * sa + b * sb are all distinct (strides in elements):
// one of the two outer dimensions steps over the other's whole extent (up to 2^31 x 2^40 elements: more
// than 64 bits hold).
inline bool distinct_elements(int64_t na, int64_t sa, int64_t nb, int64_t sb, int64_t width)
{
    if (sa < 0 || sb < 0) return false;
    const bool inner_b = nb <= 1 || sb >= width, inner_a = na <= 1 || sa >= width;
    if (!inner_a || !inner_b) return false;
    if (na <= 1 || nb <= 1) return true;
    return sa >= (__int128)(nb - 1) * sb + width || sb >= (__int128)(na - 1) * sa + width;
}

}  // namespace mla
