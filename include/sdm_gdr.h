/*
 * sdm_gdr -- the gated delta rule on MI355X (gfx950), C ABI: forward over whole sequences, its gradient, and the
 * recurrent form for one or a few tokens. In libsdm_delta; status codes are sdm_gx_status (sdm_gx_gemm.h).
 *
 * The operation. A sequence and value head h has a state S (dk x dv, float32); value heads h share the q/k head
 * h / (Hv / Hk). For each token t in order
 *     S' = exp(g_t) S;   u_t = beta_t (v_t - S'^T k_t);   S = S' + k_t u_t^T;   o_t = scale S^T q_t
 * from S = s0 (zero when NULL). g is a log decay: -inf forgets everything. Sequences are the B rows of T tokens, or,
 * with cu_seqlens, nseq runs packed into one row of T tokens (B = 1): run i is tokens cu_seqlens[i] ..
 * cu_seqlens[i+1]-1, possibly none. cu_seqlens is device data that the library does not read on the host: the kernels
 * clamp every entry to 0 .. T, so a bad one gives unspecified values and never an access outside the buffers. Tokens
 * of no run keep what their output rows held.
 *
 * Types. q, k, v, o and their gradients are float32, bfloat16 or float16 (dtype); g, beta, their gradients and every
 * state are float32. Products run on the matrix cores on operands split into bfloat16 parts that together hold a
 * float32's 24 bits, sums are float32: results carry float32 accuracy before the one rounding to dtype. There are no
 * atomics and the order of every sum is set by the sizes alone, so results are the same bits in every run.
 *
 * Values that are not finite (or within 2^-8 of the largest float32) make NaN of what depends on them, and of what shares
 * their head and their chunk of 64 tokens, tokens before them included: zeros above a triangular matrix's diagonal meet
 * them in a product. One in v stays in its column and one in q in its token's o; the recurrent form has no chunks.
 * Earlier chunks (in a gradient: none of the sequence), other sequences and other q/k heads keep their bits, and tokens of
 * no run and states of no stream are not read.
 *
 * Memory. sdm_rows_t: element (b, t, h, c) is data[b*batch + t*token + h*head + c], strides in elements; g and beta
 * have no c. Token and head strides below 2^31, any element alignment; dk and dv that are multiples of 8 are faster. The
 * states are contiguous [sequences][Hv][dk][dv]. Outputs must not overlap inputs or each other. Calls are asynchronous on
 * `stream`, allocate nothing and may be captured into a graph.
 *
 * Workspaces are the caller's (sdm_gdr_workspace bytes, 256-byte aligned, contents free to lose after the call). With P =
 * 1, 2 or 3 parts for bfloat16, float16 or float32, dkp = dk up to 64, 128 or 256 and dvp = dv up to a multiple of 8, each
 * chunk of 64 tokens (of every sequence) takes, in bytes,
 *     forward:   Hv * 50432 + Hk * 384 P dkp
 *     gradient:  Hv * (75008 + 8 dvp (dk + 64) + 512 dk where Hv > Hk) + Hk * 384 P dkp
 * since the gradient holds every chunk's state and its gradient at once: with 16 value heads on 8 of 128 x 128 in bfloat16
 * 0.74 GB for 8192 tokens, whose q, k and v are 67 MB, and 11.9 GB for 65536 tokens of twice the heads (1.1 GB).
 */
#ifndef SDM_GDR_H
#define SDM_GDR_H

#include <stdint.h>

#include "sdm_gx_gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

enum sdm_dtype { SDM_F32 = 0, SDM_BF16 = 1, SDM_F16 = 2 };

#define SDM_GDR_MAX_DIM 256 /* dk and dv */

typedef struct sdm_rows {
    void* data;
    int64_t batch, token, head;
} sdm_rows_t;

typedef struct sdm_gdr_args {
    int32_t dtype;
    float scale;
    int64_t B, T, Hk, Hv, dk, dv;
    int64_t nseq;              /* runs in cu_seqlens; B when cu_seqlens is NULL */
    const int32_t* cu_seqlens; /* nseq + 1, or NULL */
    sdm_rows_t q, k, v, g, beta;
    const float* s0;           /* [nseq][Hv][dk][dv] or NULL */
    /* forward */
    sdm_rows_t o;
    float* s_final;            /* or NULL */
    /* backward */
    sdm_rows_t d_o;
    const float* ds_final;     /* or NULL: zero */
    sdm_rows_t d_q, d_k, d_v, d_g, d_beta;
    float* ds0;                /* or NULL */
} sdm_gdr_args_t;

/* The recurrent form: T tokens (one, or the few of a draft) of B streams against a pool of states, updated in place.
 * Stream b uses state slots[b] (slots NULL: state b). A stream whose slot is outside 0 .. pool-1 is idle: its o rows
 * are set to zero and no state changes. No two streams may name one slot. */
typedef struct sdm_gdr_step_args {
    int32_t dtype;
    float scale;
    int64_t B, T, Hk, Hv, dk, dv, pool;
    sdm_rows_t q, k, v, g, beta, o;
    float* state;              /* [pool][Hv][dk][dv] */
    const int32_t* slots;      /* [B] or NULL */
} sdm_gdr_step_args_t;

/* Argument checks without a device call: null pointers, sizes, strides, alignment, overlap. */
SDM_GX_API int sdm_gdr_check(const sdm_gdr_args_t* args, int32_t backward);
SDM_GX_API int sdm_gdr_step_check(const sdm_gdr_step_args_t* args);

/* Workspace bytes of a forward (backward = 0) or backward call: at least 1, or a negative status. */
SDM_GX_API int64_t sdm_gdr_workspace(const sdm_gdr_args_t* args, int32_t backward);

SDM_GX_API int sdm_gdr_forward(const sdm_gdr_args_t* args, void* workspace, int64_t workspace_bytes, void* stream);
SDM_GX_API int sdm_gdr_backward(const sdm_gdr_args_t* args, void* workspace, int64_t workspace_bytes, void* stream);
SDM_GX_API int sdm_gdr_step(const sdm_gdr_step_args_t* args, void* stream);

/* The status text and last HIP error of this library's calls. */
SDM_GX_API const char* sdm_delta_strerror(int status);
SDM_GX_API int sdm_delta_last_hip_error(void);

#ifdef __cplusplus
}
#endif

#endif /* SDM_GDR_H */
