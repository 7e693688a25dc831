// Internal interface between the gated feed-forward product's kernels and its host entry points (not the C ABI).
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/sdm_ffn.h"

namespace sdm_delta {

// What the matrix cores are given: element types of a product's operands.
enum FfnType { kBf16, kF16, kE4m3, kF32 };

// Rows of `bytes` each, 16-byte aligned, `bytes` a multiple of 16.
struct FfnOperand {
    const char* p;
    int64_t ld;     // bytes
};

// C[m][n] = sum over k of A[m][k] B[n][k]. A pair of B's is gate and up: C is h.
struct FfnProduct {
    FfnOperand A, B, B2;
    int64_t M, N;
    int64_t bytes;              // of a row of A and of B
    int type, act, otype;       // FfnType, sdm_act or SDM_ACT_GELU, sdm_dtype
    const float *sm, *sn, *sn2; // kE4m3: scales of A's, B's and B2's rows
    char* c;                    // rows below `split`
    char* c2;                   // rows from `split` on, numbered from 0
    int64_t ldc, ldc2, split;   // elements
    float *gate, *up;           // the pair's products, or NULL
    int64_t ld_gate, ld_up;
    // No pair: the sum in `parts` parts of `part` bytes of each row (a multiple of 128), float32 sums of part i in rows i M and on
    int64_t part;
    int parts;
};
// tile: rows and columns of a workgroup's tile, 64, 128 or 256. Two products of one type go in one launch.
hipError_t launch_ffn_pair(const FfnProduct& p, int tile, hipStream_t stream);
hipError_t launch_ffn_products(const FfnProduct (&p)[2], int tile, hipStream_t stream);

// Sums of parts, in order, into a product's rows: c, and c2 from `split` on.
struct FfnJoin {
    const float* from;          // [parts][M][ld], 16-byte aligned, ld a multiple of 4
    int64_t M, N, ld;
    int parts, otype;
    char *c, *c2;
    int64_t ldc, ldc2, split;
};
hipError_t launch_ffn_join(const FfnJoin (&j)[2], hipStream_t stream);      // one launch; without parts: none

// Few rows: weights straight from memory, at any alignment. 16-bit and 8-bit rows from 17 on are faster in tiles (4096 to 8192,
// 32 rows: bfloat16 40 us here and 36 in tiles, 8 bits 21 and 15); float32 ones from 33 on.
constexpr int kFfnFewRows = 16, kFfnFewFloatRows = 32;
hipError_t launch_ffn_few(const sdm_ffn_args_t& a, hipStream_t stream);

// dst[r][c] = src[r][c] for c < C, zero up to `pad` columns; turned: dst[c][r], pad rows of src.
struct FfnLay {
    const void* src;
    int64_t ld, R, C;           // elements
    int dtype;                  // sdm_dtype or SDM_E4M3
    char* dst;
    int64_t ldd;                // bytes
    int64_t pad;                // elements
    int64_t again;              // turned: bytes from dst to a second copy; 0: none
};
hipError_t launch_ffn_lay(const FfnLay (&l)[3], hipStream_t stream);     // one launch; without rows: none

// dg and du from dh, g and u: rows[m] = dg, zeros to Fp, du, zeros to 2 Fp; cols[f] = dg's column f, zeros to Mp, and du's at
// row F + f. Two parts: behind them, in rows of twice the length, what dg and du lost by their rounding.
struct FfnGrad {
    const void* dh;
    const float *gate, *up;
    int64_t ld_dh, ld_gate, ld_up, M, F, Mp, Fp;
    int dtype, act, parts;
    char *rows, *cols;
};
// One launch, with the three operands turned.
hipError_t launch_ffn_grad(const FfnGrad& g, const FfnLay (&l)[3], hipStream_t stream);

}  // namespace sdm_delta
