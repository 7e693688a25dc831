// Host entry points of the block norm (sdm_nrm.h): argument checks, launch shapes. The arithmetic is in
// nrm_kernel.hip.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/sdm_nrm.h"
#include "delta_host.h"
#include "nrm.h"

using namespace sdm_delta;

namespace {

struct Row {
    const void* p;
    int64_t ld;
};

int check(const sdm_nrm_args_t* a, bool backward) {
    if (!a) return SDM_GX_ERR_ARG;
    if (a->dtype < SDM_F32 || a->dtype > SDM_F16 || (a->wtype != SDM_F32 && a->wtype != a->dtype)) return SDM_GX_ERR_ARG;
    if (a->act < SDM_ACT_NONE || a->act > SDM_ACT_SILU || !(a->eps >= 0.f)) return SDM_GX_ERR_ARG;
    if (a->rows < 0 || a->rows >= (int64_t(1) << 40) || a->D < 1 || a->D > SDM_NRM_MAX_D) return SDM_GX_ERR_SHAPE;
    const bool o = a->o != nullptr, y = a->w_pre != nullptr;
    if (!o && (!y || a->act != SDM_ACT_NONE)) return SDM_GX_ERR_NULL;
    if ((a->act != SDM_ACT_NONE) != (a->z != nullptr)) return SDM_GX_ERR_NULL;
    if (o && (!a->w_post || !a->scale)) return SDM_GX_ERR_NULL;
    if (!a->rstd) return SDM_GX_ERR_NULL;
    const int64_t es = elem_size(a->dtype), ws = elem_size(a->wtype);
    Row in[6], out[4];
    int ni = 0, no = 0;
    auto add = [](Row* r, int* n, const void* p, int64_t ld) {
        if (p) r[(*n)++] = Row{p, ld};
    };
    if (o) add(in, &ni, a->o, a->ld_o);
    add(in, &ni, a->z, a->ld_z);
    if (!backward) {
        if (!o && !a->x) return SDM_GX_ERR_NULL;
        if (o && !a->x_new) return SDM_GX_ERR_NULL;
        if (y && !a->y) return SDM_GX_ERR_NULL;
        add(in, &ni, a->x, a->ld_x);
        if (o) add(out, &no, a->x_new, a->ld_xn);
        if (y) add(out, &no, a->y, a->ld_y);
    } else {
        if (y && (!a->dy || !a->x_new || !a->dw_pre)) return SDM_GX_ERR_NULL;
        if (!y && !a->dxn) return SDM_GX_ERR_NULL;
        if (!o && !a->dx) return SDM_GX_ERR_NULL;
        if (o && (!a->d_o || !a->dw_post || !a->dscale)) return SDM_GX_ERR_NULL;
        if (a->z && !a->dz) return SDM_GX_ERR_NULL;
        if (y) {
            add(in, &ni, a->dy, a->ld_dy);
            add(in, &ni, a->x_new, a->ld_xn);
        }
        add(in, &ni, a->dxn, a->ld_dxn);
        add(out, &no, a->dx, a->ld_dx);
        if (o) add(out, &no, a->d_o, a->ld_do);
        if (a->z) add(out, &no, a->dz, a->ld_dz);
    }
    auto span = [&](const Row& r) { return extent(r.p, a->rows ? ((a->rows - 1) * r.ld + a->D) * es : 0); };
    for (int i = 0; i < ni + no; ++i) {
        const Row& r = i < ni ? in[i] : out[i - ni];
        if (r.ld < a->D || r.ld >= SDM_GX_LD_LIMIT) return SDM_GX_ERR_STRIDE;
        // before any extent is formed: the product may leave 64 bits
        if (double(a->rows) * double(r.ld) >= 4e17) return SDM_GX_ERR_STRIDE;
        if (!aligned(r.p, es)) return SDM_GX_ERR_ALIGN;
    }
    const void* w[] = {o ? a->w_post : nullptr, o ? a->scale : nullptr, a->w_pre,
                       backward && o ? a->dw_post : nullptr, backward && o ? a->dscale : nullptr,
                       backward && y ? a->dw_pre : nullptr};
    for (const void* p : w)
        if (!aligned(p, ws)) return SDM_GX_ERR_ALIGN;
    if (!aligned(a->rstd, 4)) return SDM_GX_ERR_ALIGN;
    // written against read; x_new over x and dx over dxn are row for row the same thread's and allowed
    Extent wr[8], rd[12];
    int nw = 0, nr = 0;
    for (int i = 0; i < no; ++i) wr[nw++] = span(out[i]);
    for (int i = 3; i < 6; ++i)
        if (w[i]) wr[nw++] = extent(w[i], a->D * ws);
    const Extent rs = extent(a->rstd, a->rows * 8);
    if (backward) rd[nr++] = rs; else wr[nw++] = rs;
    for (int i = 0; i < 3; ++i)
        if (w[i]) rd[nr++] = extent(w[i], a->D * ws);
    for (int i = 0; i < nw; ++i) {
        for (int j = i + 1; j < nw; ++j)
            if (overlap(wr[i], wr[j])) return SDM_GX_ERR_OVERLAP;
        for (int j = 0; j < nr; ++j)
            if (overlap(wr[i], rd[j])) return SDM_GX_ERR_OVERLAP;
    }
    const Row same_in = backward ? Row{a->dxn, a->ld_dxn} : Row{a->x, a->ld_x};
    const Row same_out = backward ? Row{a->dx, a->ld_dx} : Row{o ? a->x_new : nullptr, a->ld_xn};
    for (int i = 0; i < no; ++i)
        for (int j = 0; j < ni; ++j) {
            if (!overlap(span(out[i]), span(in[j]))) continue;
            if (out[i].p == same_out.p && in[j].p == same_in.p && in[j].p == out[i].p && out[i].ld == in[j].ld) continue;
            return SDM_GX_ERR_OVERLAP;
        }
    for (int j = 0; j < ni; ++j)
        for (int i = no; i < nw; ++i)
            if (overlap(wr[i], span(in[j]))) return SDM_GX_ERR_OVERLAP;
    return SDM_GX_OK;
}

NrmPlan plan(const sdm_nrm_args_t* a, bool backward) {
    NrmPlan p{};
    // 16384 rows of 4096: forward 111 us in bfloat16 and 260 in float32 with 256 threads of two groups of columns, 113
    // and 258 with 512 of one; backward in bfloat16, which holds two sums a column beside, 214 with 256 of two, 198 with
    // 512 of one
    const bool middle = a->D > 2048 && a->D <= 4096;
    p.most = a->D <= 512 ? 64 : a->D <= 1024 ? 128 : a->D <= 2048 || (middle && !backward) ? 256 : 512;
    p.vecs = static_cast<int>(cdiv(a->D, p.most * 8));
    // No wavefronts past the row (20000 rows of 2050 in bfloat16: backward 239 us, 260 with all 8); the backward of long
    // rows keeps its sums by full width.
    p.threads = backward && p.vecs > 1 ? p.most : static_cast<int>(cdiv(a->D, p.vecs * 512)) * 64;
    // forward: workgroups for up to 8 wavefronts a SIMD, whole ones a CU; backward: each leaves a partial sum, so a quarter
    const int64_t most = (backward ? 8 : 32) / (p.threads / 64) * 256;
    p.groups = static_cast<int>(a->rows < 1 ? 1 : a->rows < most ? a->rows : most);
    return p;
}

int pointers_on(const sdm_nrm_args_t* a, bool backward, int dev) {
    const void* fwd[] = {a->o, a->z, a->w_post, a->w_pre, a->scale, a->x_new, a->rstd, a->x, a->y};
    const void* bwd[] = {a->o, a->z, a->w_post, a->w_pre, a->scale, a->x_new, a->rstd, a->dxn, a->dy, a->dx, a->d_o,
                         a->dz, a->dw_post, a->dw_pre, a->dscale};
    const void* const* ps = backward ? bwd : fwd;
    const int n = backward ? 15 : 9;
    for (int i = 0; i < n; ++i)
        if (ps[i])
            if (int st = pointer_on(ps[i], dev)) return st;
    return SDM_GX_OK;
}

}  // namespace

extern "C" {

int sdm_nrm_check(const sdm_nrm_args_t* args, int32_t backward) { return check(args, backward != 0); }

int64_t sdm_nrm_workspace(const sdm_nrm_args_t* args) {
    if (!args) return SDM_GX_ERR_ARG;
    if (args->rows < 0 || args->rows >= (int64_t(1) << 40) || args->D < 1 || args->D > SDM_NRM_MAX_D)
        return SDM_GX_ERR_SHAPE;
    return static_cast<int64_t>(plan(args, true).groups) * 2 * args->D * 4;
}

int sdm_nrm_forward(const sdm_nrm_args_t* args, void* stream) {
    int st = check(args, false), dev = 0;
    if (st || args->rows == 0) return st;
    if ((st = current_gfx950(&dev)) || (st = pointers_on(args, false, dev))) return st;
    const hipError_t e = launch_nrm_forward(*args, plan(args, false), static_cast<hipStream_t>(stream));
    return e == hipSuccess ? SDM_GX_OK : record_hip_error(e);
}

// rows == 0 still runs: the weights' gradients are sums over no rows, zero
int sdm_nrm_backward(const sdm_nrm_args_t* args, void* workspace, int64_t workspace_bytes, void* stream) {
    int st = check(args, true), dev = 0;
    if (st) return st;
    if (!workspace) return SDM_GX_ERR_NULL;
    if (!aligned(workspace, 16)) return SDM_GX_ERR_ALIGN;
    const NrmPlan p = plan(args, true);
    if (workspace_bytes < static_cast<int64_t>(p.groups) * 2 * args->D * 4) return SDM_GX_ERR_LIMIT;
    if ((st = current_gfx950(&dev)) || (st = pointers_on(args, true, dev)) || (st = pointer_on(workspace, dev))) return st;
    const hipError_t e = launch_nrm_backward(*args, p, static_cast<float*>(workspace), static_cast<hipStream_t>(stream));
    return e == hipSuccess ? SDM_GX_OK : record_hip_error(e);
}

}  // extern "C"
