// Internal interface between the gated-delta-rule kernels and their host entry points (not the C ABI).
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/sdm_gdr.h"

namespace sdm_delta {

constexpr int kChunk = 64;      // tokens a chunk

// Where a call's intermediate results live. A chunk slot is one chunk of one sequence; "fragments" are matrix-core
// operand tiles, [16-row tile][32-wide k block][bfloat16 part][64 lanes][8 values].
struct GdrWork {
    float* tok;         // [slots][Hv][kTokFields][64]: per-token factors
    uint16_t* inv;      // [slots][Hv] fragments of (I + A)^-1, 64 x 64
    uint16_t* invt;     // of its transpose (backward)
    uint16_t* pm;       // of P (forward) or P^T (backward), 64 x 64
    uint16_t* kf;       // [slots][Hk] fragments of K, 64 x dkp
    uint16_t* qf;       // of Q (forward)
    uint16_t* kt;       // of K^T, dkp x 64
    uint16_t* qt;       // of Q^T (backward)
    float* st;          // [slots][Hv][dk][dvp]: each chunk's entering state (backward)
    float* dst;         // [slots][Hv][dk][dvp]: gradient of each chunk's last state (backward)
    float* u;           // [slots][Hv][64][dvp] (backward)
    float* dr;          // [slots][Hv][64][dvp] (backward)
    float* dqp;         // [slots][Hv][64][dk] per-value-head parts of dq and dk, when value heads share a q/k head
    float* dkp;
};

enum { kTokG = 0, kTokGlo, kTokEg, kTokLast, kTokBeta, kTokFields };

struct GdrLaunch {
    sdm_gdr_args_t a;
    GdrWork w;
    int32_t slots;      // chunk slots
    int32_t dkp;        // dk padded to 64, 128 or 256
    int32_t dvp;        // dv rounded up to a multiple of 8: rows of st, dst, u, dr, zero past dv
    int32_t vec_qk, vec_v;      // dk and dv are multiples of 8
};

// bfloat16 parts that hold an element of a type exactly: 3, 1, 2
inline int parts_of(int dtype) { return dtype == SDM_F32 ? 3 : dtype == SDM_BF16 ? 1 : 2; }

// Workgroups and their sizes. A launch holds fewer than 2^32 threads along x.
constexpr int64_t kMaxThreads = int64_t(1) << 32;
constexpr int kChunkThreads = 256, kScanThreads = 512, kGradThreads = 512, kStepThreads = 256;
// Tiles of 16 state columns that a scan's workgroup owns: two where one each would be more than a workgroup a CU, half
// the operands for 1.6 times the step (forward, dk = 128, bfloat16: a lone head of 16384 tokens 325 us with one tile, 508
// with two; 32 heads of 4 x 2048 tokens 341 and 250, of 2 x 2048 145 and 119).
inline int scan_tiles(const sdm_gdr_args_t& a, int dkp) {
    return dkp <= 128 && (a.dv + 15) / 16 * a.Hv * a.nseq > 256 ? 2 : 1;
}
inline int64_t scan_groups(const sdm_gdr_args_t& a, int dkp) {
    const int64_t cols = 16 * scan_tiles(a, dkp);
    return (a.dv + cols - 1) / cols * a.Hv * a.nseq;
}
// State columns of a step's workgroup: 32 where those of 128 would be at most one a CU (bfloat16, dk = dv = 128, us a
// call with 32 and with 128 columns: 256 heads 11.4 and 14.5, 384 17.1 and 15.6, 512 19.3 and 16.8, 2048 70 and 50; of
// fewer heads the call on the host shows, not the kernel's 6.2 and 9.0 for 16); for dk = 256, whose rows fill the
// registers, 64 always (a form of 32 took 54 us for 128 heads that take 18).
inline int step_columns(const sdm_gdr_step_args_t& a) {
    if (a.dk > 128) return 64;
    return a.B * a.Hv * ((a.dv + 127) / 128) <= 256 ? 32 : 128;
}
inline int64_t step_groups(const sdm_gdr_step_args_t& a) {
    const int64_t cols = step_columns(a);
    return (a.dv + cols - 1) / cols * a.Hv * a.B;
}

hipError_t launch_gdr_forward(const GdrLaunch& g, hipStream_t stream);
hipError_t launch_gdr_backward(const GdrLaunch& g, hipStream_t stream);
hipError_t launch_gdr_step(const sdm_gdr_step_args_t& a, bool vec, hipStream_t stream);

}  // namespace sdm_delta
