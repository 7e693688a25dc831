// Host entry points of the gated linear recurrence (sdm_glr.h): argument checks, parts of runs, workspaces. The arithmetic
// is in glr_kernel.hip.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/sdm_glr.h"
#include "delta_host.h"
#include "glr.h"

using namespace sdm_delta;

namespace {

constexpr int64_t kMaxTokens = int64_t(1) << 30;
constexpr int64_t kMaxThreads = int64_t(1) << 32;       // of a launch: 2^32 or more are refused by size

int check_sizes(int32_t dtype, int32_t gtype, int32_t act, int64_t B, int64_t T, int64_t D) {
    if (dtype < SDM_F32 || dtype > SDM_F16 || (gtype != SDM_F32 && gtype != dtype)) return SDM_GX_ERR_ARG;
    if (act < SDM_ACT_NONE || act > SDM_ACT_SILU) return SDM_GX_ERR_ARG;
    if (B < 1 || B >= (int64_t(1) << 20) || T < 0 || T > kMaxTokens || (T && B > kMaxTokens / T)) return SDM_GX_ERR_SHAPE;
    if (D < 1 || D > SDM_GLR_MAX_D) return SDM_GX_ERR_SHAPE;
    return SDM_GX_OK;
}

struct Operand {
    const sdm_seq_t* r;
    int64_t size;
    bool written;
};

// A strided operand's extent, or a refusal. No two elements of a written one may share a place.
int check_seq(const Operand& o, int64_t B, int64_t T, int64_t D, Extent* e) {
    const sdm_seq_t& r = *o.r;
    if (!r.data) return SDM_GX_ERR_NULL;
    if (r.batch < 0 || r.token < 0 || r.batch >= (int64_t(1) << 40) || r.token >= SDM_GX_LD_LIMIT) return SDM_GX_ERR_STRIDE;
    if (!aligned(r.data, o.size)) return SDM_GX_ERR_ALIGN;
    // the products may leave 64 bits together: bound them before the sum
    if (double(B - 1) * double(r.batch) + double(T > 0 ? T - 1 : 0) * double(r.token) + double(D) >= 4e17) return SDM_GX_ERR_STRIDE;
    if (o.written && T > 0) {
        const bool by_row = r.token <= r.batch;     // the shorter stride first; each has to step over what is below
        const int64_t s0 = by_row ? r.token : r.batch, n0 = by_row ? T : B, s1 = by_row ? r.batch : r.token, n1 = by_row ? B : T;
        int64_t below = D;
        if (n0 > 1) {
            if (s0 < below) return SDM_GX_ERR_STRIDE;
            below = (n0 - 1) * s0 + below;
        }
        if (n1 > 1 && s1 < below) return SDM_GX_ERR_STRIDE;
    }
    *e = extent(r.data, T > 0 ? ((B - 1) * r.batch + (T - 1) * r.token + D) * o.size : 0);
    return SDM_GX_OK;
}

int64_t mark_rows(const sdm_glr_args_t* a, bool packed) {
    return packed ? a->T / SDM_GLR_TILE + a->nseq : a->nseq * cdiv(a->T, SDM_GLR_TILE);
}

int check(const sdm_glr_args_t* a, bool backward) {
    if (!a) return SDM_GX_ERR_ARG;
    if (int st = check_sizes(a->dtype, a->gtype, a->act, a->B, a->T, a->D)) return st;
    if (a->nseq < 1 || a->nseq >= (int64_t(1) << 20)) return SDM_GX_ERR_SHAPE;
    if (a->cu_seqlens ? a->B != 1 : a->nseq != a->B) return SDM_GX_ERR_SHAPE;
    if (!aligned(a->cu_seqlens, 4) || !aligned(a->h0, 4) || !aligned(a->marks, 4)) return SDM_GX_ERR_ALIGN;
    const bool z = a->act != SDM_ACT_NONE;
    const int64_t es = elem_size(a->dtype), gs = elem_size(a->gtype);
    Operand ops[8];
    int n = 0;
    ops[n++] = {&a->x, es, false};
    ops[n++] = {&a->g, gs, false};
    if (z) ops[n++] = {&a->z, es, false};
    if (backward) {
        if (!a->marks && a->T) return SDM_GX_ERR_NULL;
        if (!aligned(a->dh_final, 4) || !aligned(a->dh0, 4)) return SDM_GX_ERR_ALIGN;
        ops[n++] = {&a->dy, es, false};
        ops[n++] = {&a->dx, es, true};
        ops[n++] = {&a->dg, gs, true};
        if (z) ops[n++] = {&a->dz, es, true};
    } else {
        if (!aligned(a->h_final, 4)) return SDM_GX_ERR_ALIGN;
        ops[n++] = {&a->y, es, true};
    }
    Extent in[8], out[8];
    int ni = 0, no = 0;
    for (int i = 0; i < n; ++i) {
        Extent& e = ops[i].written ? out[no++] : in[ni++];
        if (int st = check_seq(ops[i], a->B, a->T, a->D, &e)) return st;
    }
    const int64_t state = a->nseq * a->D * 4;
    auto plain = [](const void* p, int64_t bytes) { return extent(p, p ? bytes : 0); };
    in[ni++] = plain(a->cu_seqlens, (a->nseq + 1) * 4);
    in[ni++] = plain(a->h0, state);
    const Extent marks = plain(a->marks, mark_rows(a, a->cu_seqlens != nullptr) * a->D * 4);
    if (backward) {
        in[ni++] = marks;
        in[ni++] = plain(a->dh_final, state);
        out[no++] = plain(a->dh0, state);
    } else {
        out[no++] = marks;
        out[no++] = plain(a->h_final, state);
    }
    for (int i = 0; i < no; ++i) {
        for (int j = i + 1; j < no; ++j)
            if (overlap(out[i], out[j])) return SDM_GX_ERR_OVERLAP;
        for (int j = 0; j < ni; ++j)
            if (overlap(out[i], in[j])) return SDM_GX_ERR_OVERLAP;
    }
    return SDM_GX_OK;
}

// Backward: runs are cut until there is a workgroup a CU, into parts of 512 tokens at the least: a part's map costs another
// reading of its inputs. Forward: the queue where it is faster than one workgroup a run and 64 channels; of packed runs the GPU
// finds out, but where a run of all tokens would be walked. So the queue's words, 1 KB a tile and 64 channels, stay below 1.3 KB a
// token however many runs there are (4096 runs in 16384 tokens of 4096 channels would have 277 MB of them). More than a launch
// clears: walked.
GlrPlan plan(const sdm_glr_args_t* a, bool packed, bool backward) {
    GlrPlan p{};
    p.cblocks = static_cast<int>(cdiv(a->D, 64));
    const int64_t have = a->nseq * p.cblocks, each = cdiv(a->T * a->B, a->nseq), tiles = cdiv(a->T, SDM_GLR_TILE);
    p.segs = backward ? static_cast<int>(std::max<int64_t>(1, std::min(256 / have, each / 512))) : 1;
    const int64_t rows = mark_rows(a, packed);
    if (!backward && !(packed && tiles <= 4) && !glr_walks(tiles, rows * p.cblocks)) p.rows = rows;
    if (glr_chain_words(p) / 2 >= kMaxThreads) p.rows = 0;
    return p;
}
int64_t workspace(const sdm_glr_args_t* a, bool packed, bool backward) {
    const GlrPlan p = plan(a, packed, backward);
    return backward ? (p.segs > 1 ? a->nseq * p.segs * 3 * a->D * 4 : 0) : glr_chain_words(p) * 8;
}

int run(const sdm_glr_args_t* a, bool backward, void* ws, int64_t ws_bytes, void* stream) {
    int st = check(a, backward), dev = 0;
    if (st) return st;
    const bool packed = a->cu_seqlens != nullptr;
    const int64_t need = workspace(a, packed, backward);
    if (need && !ws) return SDM_GX_ERR_NULL;
    if (!aligned(ws, 16)) return SDM_GX_ERR_ALIGN;
    if (ws_bytes < need) return SDM_GX_ERR_LIMIT;
    const GlrPlan p = plan(a, packed, backward);
    if (a->nseq * p.segs * p.cblocks * kGlrThreads >= kMaxThreads) return SDM_GX_ERR_LIMIT;
    if ((st = current_gfx950(&dev))) return st;
    // without tokens the kernels still read and write the states
    const void* always[] = {a->cu_seqlens, need ? ws : nullptr, backward ? a->dh_final : a->h0, backward ? a->dh0 : a->h_final};
    for (const void* q : always)
        if (q && (st = pointer_on(q, dev))) return st;
    const void* tokens[] = {a->x.data, a->g.data, a->act ? a->z.data : nullptr, a->marks, backward ? a->dy.data : a->y.data, backward ? a->h0 : nullptr,
                            backward ? a->dx.data : nullptr, backward ? a->dg.data : nullptr, backward && a->act ? a->dz.data : nullptr};
    for (const void* q : tokens)
        if (q && a->T && (st = pointer_on(q, dev))) return st;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const hipError_t e = backward ? launch_glr_backward(*a, p, ws, s) : launch_glr_forward(*a, p, ws, s);
    return e == hipSuccess ? SDM_GX_OK : record_hip_error(e);
}

int check_step(const sdm_glr_step_args_t* a) {
    if (!a) return SDM_GX_ERR_ARG;
    if (int st = check_sizes(a->dtype, a->gtype, a->act, a->B, a->T, a->D)) return st;
    if (a->pool < 1 || a->pool >= (int64_t(1) << 31) || (!a->slots && a->pool < a->B)) return SDM_GX_ERR_SHAPE;
    if (!a->state) return SDM_GX_ERR_NULL;
    if (!aligned(a->state, 4) || !aligned(a->slots, 4)) return SDM_GX_ERR_ALIGN;
    const bool z = a->act != SDM_ACT_NONE;
    const int64_t es = elem_size(a->dtype), gs = elem_size(a->gtype);
    const Operand ops[] = {{&a->x, es, false}, {&a->g, gs, false}, {&a->y, es, true}, {&a->z, es, false}};
    Extent e[4];
    for (int i = 0; i < (z ? 4 : 3); ++i)
        if (int st = check_seq(ops[i], a->B, a->T, a->D, &e[i])) return st;
    const Extent state = extent(a->state, a->pool * a->D * 4), slots = extent(a->slots, a->slots ? a->B * 4 : 0), y = e[2];
    for (int i = 0; i < (z ? 4 : 3); ++i)
        if (overlap(state, e[i]) || (i != 2 && overlap(y, e[i]))) return SDM_GX_ERR_OVERLAP;
    return overlap(state, slots) || overlap(y, slots) ? SDM_GX_ERR_OVERLAP : SDM_GX_OK;
}

}  // namespace

extern "C" {

int sdm_glr_check(const sdm_glr_args_t* args, int32_t backward) { return check(args, backward != 0); }
int sdm_glr_step_check(const sdm_glr_step_args_t* args) { return check_step(args); }

int64_t sdm_glr_marks(const sdm_glr_args_t* args) {
    if (!args) return SDM_GX_ERR_ARG;
    const int st = check_sizes(args->dtype, args->gtype, args->act, args->B, args->T, args->D);
    if (st || args->nseq < 1 || args->nseq >= (int64_t(1) << 20)) return st ? st : SDM_GX_ERR_SHAPE;
    return mark_rows(args, args->cu_seqlens != nullptr);
}

int64_t sdm_glr_workspace(const sdm_glr_args_t* args, int32_t backward) {
    if (!args) return SDM_GX_ERR_ARG;
    const int st = check_sizes(args->dtype, args->gtype, args->act, args->B, args->T, args->D);
    if (st || args->nseq < 1 || args->nseq >= (int64_t(1) << 20)) return st ? st : SDM_GX_ERR_SHAPE;
    return workspace(args, args->cu_seqlens != nullptr, backward != 0);
}

int sdm_glr_forward(const sdm_glr_args_t* args, void* ws, int64_t ws_bytes, void* stream) { return run(args, false, ws, ws_bytes, stream); }
int sdm_glr_backward(const sdm_glr_args_t* args, void* ws, int64_t ws_bytes, void* stream) { return run(args, true, ws, ws_bytes, stream); }

int sdm_glr_step(const sdm_glr_step_args_t* a, void* stream) {
    int st = check_step(a), dev = 0;
    if (st || a->T == 0) return st;
    if (a->B * cdiv(a->D, kGlrStepThreads) * kGlrStepThreads >= kMaxThreads) return SDM_GX_ERR_LIMIT;
    if ((st = current_gfx950(&dev))) return st;
    const void* ps[] = {a->x.data, a->g.data, a->act ? a->z.data : nullptr, a->y.data, a->state, a->slots};
    for (const void* p : ps)
        if (p && (st = pointer_on(p, dev))) return st;
    const hipError_t e = launch_glr_step(*a, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? SDM_GX_OK : record_hip_error(e);
}

const char* sdm_block_strerror(int code) { return status_text(code); }
int sdm_block_last_hip_error(void) { return last_hip_error(); }

}  // extern "C"
