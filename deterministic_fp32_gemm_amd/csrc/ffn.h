// Internal interface between the gated feed-forward product's kernels and its host entry points (not the C ABI).
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/sdm_ffn.h"

namespace sdm_delta {

// What the matrix cores are given: element types of a product's operands.
enum FfnType { kBf16 = 0, kF16 = 1, kE4m3 = 2, kTypes = 3 };

// Rows of `bytes` each, 16-byte aligned, `bytes` a multiple of 16; `plane` bytes from one part of the values to the next.
struct FfnOperand {
    const char* p;
    int64_t ld, plane;      // bytes
};

// C[m][n] = sum over segments s and k of A[part a(s)][m][k] B[part b(s)][n][k]. A pair of B's is gate and up: C is h.
struct FfnProduct {
    FfnOperand A, B, B2;
    int64_t M, N;
    int64_t bytes;              // of a row of each segment
    int segments, type, act, otype;
    uint32_t aparts, bparts;    // two bits a segment
    const float *sm, *sn, *sn2; // kE4m3: scales of A's, B's and B2's rows
    char* c;                    // rows below `split`
    char* c2;                   // rows from `split` on, numbered from 0
    int64_t ldc, ldc2, split;   // elements
    float *gate, *up;           // the pair's products, or NULL
    int64_t ld_gate, ld_up;
};
// tile: rows and columns of a workgroup's tile, 64, 128 or 256. Two products of one type go in one launch.
hipError_t launch_ffn_pair(const FfnProduct& p, int tile, hipStream_t stream);
hipError_t launch_ffn_products(const FfnProduct (&p)[2], int tile, hipStream_t stream);

// Few rows: weights straight from memory, at any alignment.
constexpr int kFfnFewRows = 32;
hipError_t launch_ffn_few(const sdm_ffn_args_t& a, hipStream_t stream);

// dst[part][r][c] = src[r][c] for c < C, zero up to `pad` columns; turned: dst[part][c][r], pad rows of src. float32 sources
// become three bfloat16 parts, others are copied.
struct FfnLay {
    const void* src;
    int64_t ld, R, C;           // elements
    int dtype;                  // sdm_dtype or SDM_E4M3
    char* dst;
    int64_t ldd, plane;         // bytes
    int64_t pad;                // elements
};
hipError_t launch_ffn_lay(const FfnLay (&l)[3], bool turned, hipStream_t stream);     // one launch; without rows: none

// dg and du from dh, g and u: rows[part][m] = dg, zeros to Fp, du, zeros to 2 Fp; cols[part][f] = dg's column f, zeros to Mp,
// and du's at row F + f.
struct FfnGrad {
    const void* dh;
    const float *gate, *up;
    int64_t ld_dh, ld_gate, ld_up, M, F, Mp, Fp;
    int dtype, act;
    char *rows, *cols;
    int64_t rows_plane, cols_plane;     // bytes
};
hipError_t launch_ffn_grad(const FfnGrad& g, hipStream_t stream);

}  // namespace sdm_delta
