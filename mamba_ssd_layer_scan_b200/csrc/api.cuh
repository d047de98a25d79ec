// What the files with C ABI entry points share: the error string, shape checks, alignment.
// Defined in ssd_api.cu.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/ssd.h"

namespace ssd {

// Sets the calling thread's message (printf style) and returns `s`.
ssd_status api_fail(ssd_status s, const char *fmt, ...);
ssd_status api_cuda_fail(cudaError_t e, const char *what);
ssd_status api_check_shape(const ssd_shape *s, bool need_seq);

inline bool api_aligned(const void *p, uintptr_t bytes)
{
    return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}
inline size_t api_round256(size_t v) { return (v + 255) & ~size_t(255); }

}  // namespace ssd
