// Internal interface between the gated linear recurrence's kernels and its host entry points (not the C ABI).
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/sdm_glr.h"

namespace sdm_delta {

constexpr int kGlrWaves = 8, kGlrTokens = SDM_GLR_TILE / kGlrWaves;     // of a tile: wavefronts, tokens of each
constexpr int kGlrThreads = kGlrWaves * 64, kGlrStepThreads = 256;

struct GlrPlan {
    int cblocks;        // blocks of 64 channels
    int segs;           // parts that a run is cut into
};

// part: float [nseq][segs][2][D], what each part makes of the state that enters it (segs > 1)
hipError_t launch_glr_forward(const sdm_glr_args_t& a, const GlrPlan& p, float* part, hipStream_t stream);
hipError_t launch_glr_backward(const sdm_glr_args_t& a, const GlrPlan& p, float* part, hipStream_t stream);
hipError_t launch_glr_step(const sdm_glr_step_args_t& a, hipStream_t stream);

}  // namespace sdm_delta
