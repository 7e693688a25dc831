// Host entry point of the 8-bit rows (sdm_qnt.h): argument checks, launch shapes. The arithmetic is in qnt_kernel.hip.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/sdm_qnt.h"
#include "delta_host.h"
#include "qnt.h"

using namespace sdm_delta;

namespace {

struct Row {
    const void* p;
    int64_t ld, size;
};

int check(const sdm_qnt_args_t* a) {
    if (!a) return SDM_GX_ERR_ARG;
    if (a->dtype < SDM_F32 || a->dtype > SDM_F16 || !(a->eps >= 0.f)) return SDM_GX_ERR_ARG;
    if (a->wtype != SDM_F32 && a->wtype != a->dtype) return SDM_GX_ERR_ARG;
    if (a->rows < 0 || a->rows >= (int64_t(1) << 40) || a->D < 1 || a->D > SDM_QNT_MAX_D) return SDM_GX_ERR_SHAPE;
    if (!a->x || !a->q || !a->scale || (a->r && !a->x_new)) return SDM_GX_ERR_NULL;
    const int64_t es = elem_size(a->dtype);
    const Row in[] = {{a->x, a->ld_x, es}, {a->r, a->ld_r, es}};
    const Row out[] = {{a->q, a->ld_q, 1}, {a->r ? a->x_new : nullptr, a->ld_xn, es}};
    for (const Row* rows : {in, out})
        for (int i = 0; i < 2; ++i) {
            const Row& r = rows[i];
            if (!r.p) continue;
            if (r.ld < a->D || r.ld >= SDM_GX_LD_LIMIT || double(a->rows) * double(r.ld) >= 4e17) return SDM_GX_ERR_STRIDE;
            if (!aligned(r.p, r.size)) return SDM_GX_ERR_ALIGN;
        }
    if (!aligned(a->w, elem_size(a->wtype)) || !aligned(a->scale, 4)) return SDM_GX_ERR_ALIGN;
    auto span = [&](const Row& r) { return extent(r.p, r.p && a->rows ? ((a->rows - 1) * r.ld + a->D) * r.size : 0); };
    const Extent q = span(out[0]), xn = span(out[1]), s = extent(a->scale, a->rows * 4);
    const Extent x = span(in[0]), r = span(in[1]), w = extent(a->w, a->w ? a->D * elem_size(a->wtype) : 0);
    if (overlap(q, xn) || overlap(q, s) || overlap(xn, s)) return SDM_GX_ERR_OVERLAP;
    for (const Extent& i : {x, r, w})
        if (overlap(q, i) || overlap(s, i)) return SDM_GX_ERR_OVERLAP;
    if (overlap(xn, w)) return SDM_GX_ERR_OVERLAP;
    // x' over x or r is row for row the same thread's
    for (int i = 0; i < 2; ++i)
        if (overlap(xn, i ? r : x) && !(in[i].p == a->x_new && in[i].ld == a->ld_xn)) return SDM_GX_ERR_OVERLAP;
    return SDM_GX_OK;
}

QntPlan plan(const sdm_qnt_args_t* a) {
    QntPlan p{};
    p.most = a->D <= 512 ? 64 : a->D <= 4096 ? 256 : 1024;
    p.vecs = static_cast<int>(cdiv(a->D, p.most * 8));
    p.threads = static_cast<int>(cdiv(a->D, p.vecs * 512)) * 64;      // no wavefronts past the row
    const int64_t most = 32 / (p.threads / 64) * 256;
    p.groups = static_cast<int>(a->rows < 1 ? 1 : a->rows < most ? a->rows : most);
    return p;
}

}  // namespace

extern "C" {

int sdm_qnt_check(const sdm_qnt_args_t* args) { return check(args); }

int sdm_qnt_rows(const sdm_qnt_args_t* a, void* stream) {
    int st = check(a), dev = 0;
    if (st || a->rows == 0) return st;
    if ((st = current_gfx950(&dev))) return st;
    const void* ps[] = {a->x, a->r, a->w, a->r ? a->x_new : nullptr, a->q, a->scale};
    for (const void* p : ps)
        if (p && (st = pointer_on(p, dev))) return st;
    const hipError_t e = launch_qnt(*a, plan(a), static_cast<hipStream_t>(stream));
    return e == hipSuccess ? SDM_GX_OK : record_hip_error(e);
}

}  // extern "C"
