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
    int64_t rows;       // forward: rows of marks, whose tiles are taken from a queue (packed runs: perhaps); 0: a workgroup walks a run
    int segs;           // backward: parts that a run is cut into
};
// Whether runs are walked: a workgroup takes 2.7 us a tile of the longest run, the queue 10 us and 4.6 us for 256 tiles (bfloat16,
// whole calls; 2 rows of 4096 tokens and 4096 channels: 106 us walked, 83 from the queue; 7 of 2048 and 2048: 65 and 73; 16 packed runs
// of 512 tokens, 2048 channels: 46 and 62, 52 where the GPU chooses; one of 6784 and 22 of 64: 168 and 71).
__host__ __device__ inline bool glr_walks(int64_t longest, int64_t tickets) { return 27 * longest <= 100 + 46 * tickets / 256; }
// Words of 8 bytes of the forward's workspace: the queue's counter and the choice in the first 64, then two for each tile
// and channel.
inline int64_t glr_chain_words(const GlrPlan& p) { return p.rows ? 64 + p.rows * p.cblocks * 128 : 0; }

// ws: forward: glr_chain_words; backward: float [nseq][segs][3][D], what each part makes of what enters it (segs > 1)
hipError_t launch_glr_forward(const sdm_glr_args_t& a, const GlrPlan& p, void* ws, hipStream_t stream);
hipError_t launch_glr_backward(const sdm_glr_args_t& a, const GlrPlan& p, void* ws, hipStream_t stream);
hipError_t launch_glr_step(const sdm_glr_step_args_t& a, hipStream_t stream);

}  // namespace sdm_delta
