/*
 * sdm_qnt -- rows brought to 8 bits on MI355X (gfx950), C ABI: the norm before a feed-forward, with the residual's
 * addition, and the rounding alone. In libsdm_block; status codes are sdm_gx_status (sdm_gx_gemm.h).
 *
 * For each of `rows` rows of D values, with sums in float32:
 *     x' = x + r                       stored in dtype (r NULL: x' is x and is not written)
 *     y  = x' w / sqrt(mean(x'^2) + eps)        from the stored x' (w NULL: y is x')
 *     s  = max(max |y| / 448, 2^-126);   q = e4m3(y / s)
 * q is OCP e4m3 (one byte: sign, 4 bits of exponent, 3 of fraction, no infinities), to the nearest, ties to even; q s stands
 * for y within 2^-4 of it where |y| >= 2^-6 s and within 2^-10 s below. y / s is taken as y times the float32 nearest 1 / s:
 * 2^-23 before a rounding of 2^-4. A row with a value that is not finite, or whose sum of squares or largest |x' w|
 * leaves float32, gets s = NaN and q = NaN throughout.
 *
 * Types: x, r, x' float32, bfloat16 or float16 (dtype, sdm_gdr.h); w in wtype, that or float32; s float32. Rows are
 * contiguous with a row stride `ld_*` >= D in elements (of q: bytes), below 2^31. 1 <= D <= SDM_QNT_MAX_D; rows below 2^40. Outputs must not overlap
 * inputs, except that x_new may be x or r exactly (same address and stride). Asynchronous on `stream`; nothing is
 * allocated; calls may be captured into a graph.
 */
#ifndef SDM_QNT_H
#define SDM_QNT_H

#include <stdint.h>

#include "sdm_gdr.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SDM_QNT_MAX_D 16384

typedef struct sdm_qnt_args {
    int32_t dtype, wtype;
    float eps;
    int32_t reserved;
    int64_t rows, D;
    const void *x, *r, *w;
    int64_t ld_x, ld_r;
    void *x_new, *q;
    int64_t ld_xn, ld_q;
    float* scale;                 /* [rows] */
} sdm_qnt_args_t;

SDM_GX_API int sdm_qnt_check(const sdm_qnt_args_t* args);
SDM_GX_API int sdm_qnt_rows(const sdm_qnt_args_t* args, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SDM_QNT_H */
