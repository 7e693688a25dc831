// Host side shared by the delta entry points: device and pointer checks, extents.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/sdm_gx_gemm.h"

namespace sdm_delta {

int record_hip_error(hipError_t e);             // keeps e for sdm_delta_last_hip_error, returns SDM_GX_ERR_HIP
int current_gfx950(int* dev);                   // the current device, SDM_GX_ERR_DEVICE if it is not gfx950
int pointer_on(const void* p, int dev);         // SDM_GX_OK: device memory of dev

struct Extent {
    uintptr_t lo, hi;
};
inline bool overlap(Extent a, Extent b) { return a.lo < b.hi && b.lo < a.hi; }
inline Extent extent(const void* p, int64_t bytes) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return Extent{a, a + static_cast<uintptr_t>(bytes)};
}
inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t elem_size(int dtype) { return dtype == 0 ? 4 : 2; }
inline bool aligned(const void* p, int64_t to) { return reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(to) == 0; }

}  // namespace sdm_delta
