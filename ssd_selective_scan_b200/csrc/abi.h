// abi.h -- what the C entry points' argument checks share.
#pragma once

#include "ssd.h"

namespace ssd {

struct Range {
    uintptr_t lo, hi;   // [lo, hi)
};

inline Range span(const void* p, int64_t bytes)
{
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return Range{a, a + (uintptr_t)(bytes > 0 ? bytes : 0)};
}

inline bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi && a.hi > a.lo && b.hi > b.lo; }

inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

inline bool valid_dtype(ssd_dtype_t d) { return d == SSD_F32 || d == SSD_BF16; }

inline int elem_bytes(ssd_dtype_t d) { return d == SSD_F32 ? 4 : 2; }

inline ssd_status_t from_cuda(cudaError_t e)
{
    if (e == cudaSuccess) return SSD_OK;
    (void)cudaGetLastError();
    return SSD_ERR_CUDA;
}

inline int max_optin_smem()
{
    int dev = 0, v = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    if (cudaDeviceGetAttribute(&v, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) != cudaSuccess) return 0;
    return v;
}

inline size_t round_up_256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace ssd
