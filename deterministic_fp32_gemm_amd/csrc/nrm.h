// Internal interface between the norm kernels and their host entry points (not the C ABI).
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/sdm_nrm.h"

namespace sdm_delta {

struct NrmPlan {
    int most;       // threads of the kernel's instance at the most: 64, 128, 256 or 512
    int threads;    // of a workgroup, which takes one row at a time: the wavefronts that have columns
    int vecs;       // groups of 8 columns a thread: threads * vecs * 8 >= D
    int groups;     // workgroups; workgroup i takes rows i, i + groups, ...
};

hipError_t launch_nrm_forward(const sdm_nrm_args_t& a, const NrmPlan& p, hipStream_t stream);
// part: float [groups][2][D], the workgroups' sums
hipError_t launch_nrm_backward(const sdm_nrm_args_t& a, const NrmPlan& p, float* part, hipStream_t stream);

}  // namespace sdm_delta
