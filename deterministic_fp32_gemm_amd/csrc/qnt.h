// Internal interface between the 8-bit rows' kernel and its host entry point (not the C ABI).
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/sdm_qnt.h"

namespace sdm_delta {

struct QntPlan {
    int most;       // threads of the kernel's instance at the most: 64, 256 or 1024
    int vecs;       // groups of 8 columns a thread: threads * vecs * 8 >= D
    int threads;    // of a workgroup, which takes one row at a time: the wavefronts that have columns
    int groups;     // workgroups; workgroup i takes rows i, i + groups, ...
};

hipError_t launch_qnt(const sdm_qnt_args_t& a, const QntPlan& p, hipStream_t stream);

}  // namespace sdm_delta
