/*
 * sdm_nrm -- the norms after one residual block and before the next, fused with the block's gate and residual scale,
 * on MI355X (gfx950), C ABI. In libsdm_delta; status codes are sdm_gx_status (sdm_gx_gemm.h).
 *
 * For each of `rows` rows of D values (sums and norms in float32):
 *     r1 = 1 / sqrt(mean(o^2) + eps);   x' = x + scale * (o r1 w_post) act(z);   stored in dtype
 *     r2 = 1 / sqrt(mean(x'^2) + eps);  y = x' r2 w_pre                          of the stored x'
 * act: none (z NULL), sigmoid(z) or z sigmoid(z). x NULL: no residual. w_pre NULL: no second norm (y NULL). o NULL:
 * only the second norm, of x (x', z, w_post and scale NULL). rstd, two float32 a row, gets r1 and r2 (0 for one that
 * is not computed); the backward call reads it.
 *
 * Backward, from dx' (NULL: zero) and dy (NULL without a second norm), both gradients of the call's outputs:
 *     dx = dx' + r2 (dy w_pre - x' r2^2 mean(dy w_pre x'));   dn = dx scale act(z)
 *     do = r1 (dn w_post - o r1^2 mean(dn w_post o));          dz = dx scale o r1 w_post act'(z)
 *     dw_post = sum over rows of dn o r1;  dw_pre = sum of dy x' r2;  dscale = sum of dx o r1 w_post act(z)
 * The sums over rows run in a fixed order (no atomics): the same bits in every run.
 *
 * Types: x, o, z, x', y and their gradients float32, bfloat16 or float16 (dtype, sdm_gdr.h); weights, scale and their
 * gradients in wtype. Rows are contiguous with a row stride `ld_*` >= D in elements. 1 <= D <= SDM_NRM_MAX_D.
 * Outputs must not overlap inputs, except that x_new may be x and dx may be dx' exactly (same address and stride).
 */
#ifndef SDM_NRM_H
#define SDM_NRM_H

#include <stdint.h>

#include "sdm_gdr.h"

#ifdef __cplusplus
extern "C" {
#endif

enum sdm_act { SDM_ACT_NONE = 0, SDM_ACT_SIGMOID = 1, SDM_ACT_SILU = 2 };

#define SDM_NRM_MAX_D 8192

typedef struct sdm_nrm_args {
    int32_t dtype, wtype, act;
    float eps;
    int64_t rows, D;
    const void *x, *o, *z;
    int64_t ld_x, ld_o, ld_z;
    const void *w_post, *w_pre, *scale;
    void *x_new, *y;              /* forward: written; backward: x_new is read (the stored x', or x when o is NULL) */
    int64_t ld_xn, ld_y;
    float* rstd;                  /* [rows][2] */
    /* backward */
    const void *dxn, *dy;
    int64_t ld_dxn, ld_dy;
    void *dx, *d_o, *dz;
    int64_t ld_dx, ld_do, ld_dz;
    void *dw_post, *dw_pre, *dscale;
} sdm_nrm_args_t;

SDM_GX_API int sdm_nrm_check(const sdm_nrm_args_t* args, int32_t backward);

/* Workspace bytes of the backward call (partial sums of the weights' gradients): at least 1, or a negative status. */
SDM_GX_API int64_t sdm_nrm_workspace(const sdm_nrm_args_t* args);

SDM_GX_API int sdm_nrm_forward(const sdm_nrm_args_t* args, void* stream);
SDM_GX_API int sdm_nrm_backward(const sdm_nrm_args_t* args, void* workspace, int64_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SDM_NRM_H */
