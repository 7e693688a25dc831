/*
 * sdm_glr -- the gated linear recurrence on MI355X (gfx950), C ABI: forward over whole sequences, its gradient, and the
 * recurrent form for one or a few tokens. In libsdm_block; status codes are sdm_gx_status (sdm_gx_gemm.h).
 *
 * The operation. Every channel of a sequence has a float32 state h. For each token t in order
 *     h_t = exp(g_t) h_{t-1} + x_t;   y_t = h_t act(z_t)
 * from h = h0 (zero when NULL). g is a log decay: -inf forgets everything. act: none (z NULL: y is h), sigmoid(z) or
 * z sigmoid(z). Sequences are the B rows of T tokens, or, with cu_seqlens, nseq runs packed into one row of T tokens
 * (B = 1): run i is tokens cu_seqlens[i] .. cu_seqlens[i+1]-1, possibly none. cu_seqlens is device data that the library
 * does not read on the host: the kernels clamp every entry to 0 .. T, so a bad one gives unspecified values and never an
 * access outside the buffers. Tokens of no run keep what their output rows held.
 *
 * Backward, from dy and dh_final (NULL: zero), the gradients of y and of the last state:
 *     D_t = dy_t act(z_t) + exp(g_{t+1}) D_{t+1}  (+ dh_final at the last token)
 *     dx_t = D_t;  dg_t = D_t exp(g_t) h_{t-1};  dz_t = dy_t h_t act'(z_t);  dh0 = exp(g_1) D_1
 * It reads `marks`, what the forward call left: the state before every SDM_GLR_TILE-th token of a sequence, in the order of
 * the sequences. The states between them are computed again.
 *
 * Types. x, y, z and their gradients are float32, bfloat16 or float16 (dtype); g and dg that or float32 (gtype); states
 * float32, and so is every sum. No atomics in sums and an order of operations set by the sizes and the sequences' lengths: the
 * same bits in every run.
 * exp(g) below 2^-126 may be zero. Gates may grow (g > 0) and fall as far as the states stay in float32: products of decays over many
 * tokens need not.
 * Values that are not finite stay in their channel and sequence; what they make of later tokens is not finite or NaN.
 *
 * Where few runs are long, the forward call's workgroups wait on the GPU for one another's states. Each of those waits ends by
 * itself; one of 2^22 looks (some seconds, which nothing but a fault of the machine explains) is given up, and the outputs, marks and
 * states that come after it in its run are NaN. The status, that of the launch, does not tell.
 *
 * Memory. sdm_seq_t: element (b, t, c) is data[b*batch + t*token + c], strides in elements; token strides below 2^31, any
 * element alignment. 1 <= D <= SDM_GLR_MAX_D; B and nseq below 2^20, B T up to 2^30, pool below 2^31. The states are contiguous
 * [sequences][D], marks [sdm_glr_marks rows][D]. Outputs must not overlap
 * inputs or each other. Calls are asynchronous on `stream`, allocate nothing and may be captured into a graph.
 * Workspaces are the caller's (sdm_glr_workspace bytes, 16-byte aligned, contents free to lose after the call).
 */
#ifndef SDM_GLR_H
#define SDM_GLR_H

#include <stdint.h>

#include "sdm_nrm.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SDM_GLR_TILE 128 /* tokens between two marks */
#define SDM_GLR_MAX_D 65536

typedef struct sdm_seq {
    void* data;
    int64_t batch, token;
} sdm_seq_t;

typedef struct sdm_glr_args {
    int32_t dtype, gtype, act, reserved;
    int64_t B, T, D;
    int64_t nseq;              /* runs in cu_seqlens; B when cu_seqlens is NULL */
    const int32_t* cu_seqlens; /* nseq + 1, or NULL */
    sdm_seq_t x, g, z;
    const float* h0;           /* [nseq][D] or NULL */
    float* marks;              /* forward: written, NULL: not wanted; backward: read */
    /* forward */
    sdm_seq_t y;
    float* h_final;            /* or NULL */
    /* backward */
    sdm_seq_t dy;
    const float* dh_final;     /* or NULL: zero */
    sdm_seq_t dx, dg, dz;
    float* dh0;                /* or NULL */
} sdm_glr_args_t;

/* The recurrent form: T tokens (one, or the few of a draft) of B streams against a pool of states, updated in place.
 * Stream b uses state slots[b] (slots NULL: state b). A stream whose slot is outside 0 .. pool-1 is idle: its y rows are
 * set to zero and no state changes. No two streams may name one slot. */
typedef struct sdm_glr_step_args {
    int32_t dtype, gtype, act, reserved;
    int64_t B, T, D, pool;
    sdm_seq_t x, g, z, y;
    float* state;              /* [pool][D] */
    const int32_t* slots;      /* [B] or NULL */
} sdm_glr_step_args_t;

/* Argument checks without a device call: null pointers, sizes, strides, alignment, overlap. */
SDM_GX_API int sdm_glr_check(const sdm_glr_args_t* args, int32_t backward);
SDM_GX_API int sdm_glr_step_check(const sdm_glr_step_args_t* args);

/* Rows of `marks`, and workspace bytes of a forward (backward = 0) or backward call: at least 0, or a negative status.
 * They depend on the sizes and on whether cu_seqlens is NULL. Calls of 2^23 workgroups or more (runs times D / 64, rounded up)
 * are refused. */
SDM_GX_API int64_t sdm_glr_marks(const sdm_glr_args_t* args);
SDM_GX_API int64_t sdm_glr_workspace(const sdm_glr_args_t* args, int32_t backward);

SDM_GX_API int sdm_glr_forward(const sdm_glr_args_t* args, void* workspace, int64_t workspace_bytes, void* stream);
SDM_GX_API int sdm_glr_backward(const sdm_glr_args_t* args, void* workspace, int64_t workspace_bytes, void* stream);
SDM_GX_API int sdm_glr_step(const sdm_glr_step_args_t* args, void* stream);

/* The status text and last HIP error of this library's calls. */
SDM_GX_API const char* sdm_block_strerror(int status);
SDM_GX_API int sdm_block_last_hip_error(void);

#ifdef __cplusplus
}
#endif

#endif /* SDM_GLR_H */
