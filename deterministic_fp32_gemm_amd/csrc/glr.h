// Internal interface between the gated linear recurrence's kernels and its host entry points (not the C ABI).
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/sdm_glr.h"

namespace sdm_delta {

constexpr int kGlrWaves = 8, kGlrTokens = SDM_GLR_TILE / kGlrWaves;     // of a tile: wavefronts, tokens of each
constexpr int kGlrThreads = kGlrWaves * 64, kGlrStepThreads = 256;

// of the queue's kernel: eight wavefronts and one that takes tickets; a workgroup a CU
constexpr int kGlrChainThreads = (kGlrWaves + 1) * 64, kGlrChainGroups = 256;

struct GlrPlan {
    int cblocks;        // blocks of 64 channels
    int64_t rows;       // forward: rows of marks, whose tiles are taken from a queue; 0: a workgroup walks a run
    int segs;           // backward: parts that a run is cut into
};
// Words of 8 bytes of the forward's workspace: the queue's counter in the first 64, then three for each tile and channel.
inline int64_t glr_chain_words(const sdm_glr_args_t&, const GlrPlan& p) { return p.rows ? 64 + p.rows * p.cblocks * 192 : 0; }

// ws: forward: glr_chain_words; backward: float [nseq][segs][2][D], what each part makes of what enters it (segs > 1)
hipError_t launch_glr_forward(const sdm_glr_args_t& a, const GlrPlan& p, void* ws, hipStream_t stream);
hipError_t launch_glr_backward(const sdm_glr_args_t& a, const GlrPlan& p, void* ws, hipStream_t stream);
hipError_t launch_glr_step(const sdm_glr_step_args_t& a, hipStream_t stream);

}  // namespace sdm_delta
