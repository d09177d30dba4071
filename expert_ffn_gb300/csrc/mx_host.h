// mx_host.h -- host helpers that the operators' entry points share.
#pragma once

#include "mx_error.h"

#include <cstdint>
#include <cuda_runtime.h>

namespace mx {

constexpr size_t kErrBytes = 256;  // a workspace's error word

inline bool aligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
inline size_t up256(size_t n) { return (n + 255) & ~size_t(255); }

inline mx_status cuda_fail(cudaError_t e, const char *what)
{
    return fail(MX_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

// SMs of the current device.
int num_sms();

inline mx_status check_dtype(int dtype, const char *name)
{
    if (dtype != MX_F32 && dtype != MX_BF16)
        return fail(MX_ERR_INVALID_ARG, "%s %d is not MX_F32 or MX_BF16", name, dtype);
    return MX_OK;
}

inline mx_status check_ws(const void *ws, size_t have, size_t need)
{
    if (!ws || have < need)
        return fail(MX_ERR_WORKSPACE, "workspace of %zu bytes, %zu are needed", ws ? have : (size_t)0, need);
    if (!aligned(ws, 256))
        return fail(MX_ERR_ALIGNMENT, "workspace must be 256-byte aligned");
    return MX_OK;
}

inline size_t dtype_bytes(int dtype) { return dtype == MX_BF16 ? 2 : 4; }

// Whether rows of `out` start at multiples of 16 bytes.
inline bool vec16(const void *out, int64_t ldo, int bf16) { return aligned(out, 16) && ldo * (bf16 ? 2 : 4) % 16 == 0; }

// A launch that may begin while the kernel before it in the stream still runs (programmatic
// dependent launch): the kernel waits for that one's memory by pdl_wait.
template <typename Args>
cudaError_t launch_dependent(void (*k)(Args), int grid, int block, size_t smem, cudaStream_t s, const Args &a)
{
    cudaLaunchConfig_t c{};
    c.gridDim = dim3(grid);
    c.blockDim = dim3(block);
    c.dynamicSmemBytes = smem;
    c.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    c.attrs = at;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, k, a);
}

}  // namespace mx
