// Host entry points of the gated delta rule (sdm_gdr.h): argument checks, workspaces, launch shapes. The arithmetic
// is in the gdr_*.hip files.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <atomic>
#include <cstring>

#include "../../include/sdm_gdr.h"
#include "delta_host.h"
#include "gdr.h"

namespace sdm_delta {

namespace {
thread_local int t_last_hip_error = 0;
constexpr int kDevices = 64;
std::atomic<int> g_known[kDevices];     // per device: 0 not asked yet, 1 gfx950, 2 another
}  // namespace

int record_hip_error(hipError_t e) {
    t_last_hip_error = static_cast<int>(e);
    return SDM_GX_ERR_HIP;
}

int current_gfx950(int* dev) {
    hipError_t e = hipGetDevice(dev);
    if (e != hipSuccess) return record_hip_error(e);
    if (*dev < 0 || *dev >= kDevices) return SDM_GX_ERR_DEVICE;
    int k = g_known[*dev].load(std::memory_order_relaxed);
    if (!k) {
        hipDeviceProp_t prop;
        e = hipGetDeviceProperties(&prop, *dev);
        if (e != hipSuccess) return record_hip_error(e);
        k = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0 ? 1 : 2;
        g_known[*dev].store(k, std::memory_order_relaxed);
    }
    return k == 1 ? SDM_GX_OK : SDM_GX_ERR_DEVICE;
}

int pointer_on(const void* p, int dev) {
    hipPointerAttribute_t at;
    if (hipPointerGetAttributes(&at, p) != hipSuccess) {
        (void)hipGetLastError();
        return SDM_GX_ERR_DEVICE;
    }
    return (at.type == hipMemoryTypeDevice || at.type == hipMemoryTypeManaged) && at.device == dev ? SDM_GX_OK
                                                                                                  : SDM_GX_ERR_DEVICE;
}

}  // namespace sdm_delta

using namespace sdm_delta;

namespace {

constexpr int64_t kMaxTokens = int64_t(1) << 31;

// Shapes shared by the sequence and step forms.
int check_sizes(int32_t dtype, int64_t B, int64_t T, int64_t Hk, int64_t Hv, int64_t dk, int64_t dv) {
    if (dtype < SDM_F32 || dtype > SDM_F16) return SDM_GX_ERR_ARG;
    if (B < 1 || B >= (int64_t(1) << 20) || T < 0 || T >= kMaxTokens || (T && B > kMaxTokens / T)) return SDM_GX_ERR_SHAPE;
    if (Hk < 1 || Hv < Hk || Hv > 65535 || Hv % Hk) return SDM_GX_ERR_SHAPE;
    if (dk < 1 || dk > SDM_GDR_MAX_DIM || dv < 1 || dv > SDM_GDR_MAX_DIM) return SDM_GX_ERR_SHAPE;
    return SDM_GX_OK;
}

// One strided operand: its bytes, or a refusal.
struct Operand {
    const sdm_rows_t* r;
    int64_t heads, cols, size;
};

int check_rows(const Operand& o, int64_t B, int64_t T, Extent* e) {
    if (!o.r->data) return SDM_GX_ERR_NULL;
    const sdm_rows_t& r = *o.r;
    if (r.batch < 0 || r.token < 0 || r.head < 0 || r.batch >= (int64_t(1) << 40) || r.token >= SDM_GX_LD_LIMIT ||
        r.head >= SDM_GX_LD_LIMIT)
        return SDM_GX_ERR_STRIDE;
    if (!aligned(r.data, o.size)) return SDM_GX_ERR_ALIGN;
    // the products may overflow together: bound them before the sum
    const double span = double(B - 1) * double(r.batch) + double(T > 0 ? T - 1 : 0) * double(r.token) +
                        double(o.heads - 1) * double(r.head) + double(o.cols);
    if (span >= 4e17) return SDM_GX_ERR_STRIDE;
    const int64_t n = (B - 1) * r.batch + (T - 1) * r.token + (o.heads - 1) * r.head + o.cols;
    *e = extent(r.data, T > 0 ? n * o.size : 0);
    return SDM_GX_OK;
}

// Written rows: no two elements of one operand may share a place (a stride of zero or rows that run into each
// other). The three strided axes, sorted by stride, each have to step over all that is below.
int check_written(const Operand& o, int64_t B, int64_t T) {
    struct Axis {
        int64_t n, s;
    } ax[3] = {{B, o.r->batch}, {T, o.r->token}, {o.heads, o.r->head}};
    for (int i = 0; i < 3; ++i)
        for (int j = i + 1; j < 3; ++j)
            if (ax[j].s < ax[i].s) {
                const Axis t = ax[i];
                ax[i] = ax[j];
                ax[j] = t;
            }
    int64_t below = o.cols;
    for (const Axis& x : ax) {
        if (x.n <= 1) continue;
        if (x.s < below) return SDM_GX_ERR_STRIDE;
        below = (x.n - 1) * x.s + below;
    }
    return SDM_GX_OK;
}

int check(const sdm_gdr_args_t* a, bool backward) {
    if (!a) return SDM_GX_ERR_ARG;
    if (int st = check_sizes(a->dtype, a->B, a->T, a->Hk, a->Hv, a->dk, a->dv)) return st;
    if (a->cu_seqlens) {
        if (a->B != 1 || a->nseq < 1 || a->nseq >= (int64_t(1) << 20)) return SDM_GX_ERR_SHAPE;
        if (!aligned(a->cu_seqlens, 4)) return SDM_GX_ERR_ALIGN;
    } else if (a->nseq != a->B) {
        return SDM_GX_ERR_SHAPE;
    }
    const int64_t es = elem_size(a->dtype), state = a->nseq * a->Hv * a->dk * a->dv * 4;
    const Operand in[] = {{&a->q, a->Hk, a->dk, es}, {&a->k, a->Hk, a->dk, es},   {&a->v, a->Hv, a->dv, es},
                          {&a->g, a->Hv, 1, 4},      {&a->beta, a->Hv, 1, 4},     {&a->d_o, a->Hv, a->dv, es}};
    const Operand fo[] = {{&a->o, a->Hv, a->dv, es}};
    const Operand bo[] = {{&a->d_q, a->Hk, a->dk, es},
                          {&a->d_k, a->Hk, a->dk, es},
                          {&a->d_v, a->Hv, a->dv, es},
                          {&a->d_g, a->Hv, 1, 4},
                          {&a->d_beta, a->Hv, 1, 4}};
    const Operand* out = backward ? bo : fo;
    const int ni = backward ? 6 : 5, no = backward ? 5 : 1;
    Extent rd[10], wr[8];
    int nr = 0, nw = 0;
    for (int i = 0; i < ni; ++i)
        if (int st = check_rows(in[i], a->B, a->T, &rd[nr++])) return st;
    for (int i = 0; i < no; ++i) {
        if (int st = check_rows(out[i], a->B, a->T, &wr[nw++])) return st;
        if (int st = check_written(out[i], a->B, a->T)) return st;
    }
    const void* sr[] = {a->s0, backward ? a->ds_final : nullptr};
    const void* sw[] = {backward ? static_cast<void*>(a->ds0) : static_cast<void*>(a->s_final)};
    for (const void* p : sr) {
        if (!aligned(p, 4)) return SDM_GX_ERR_ALIGN;
        if (p) rd[nr++] = extent(p, state);
    }
    for (const void* p : sw) {
        if (!aligned(p, 4)) return SDM_GX_ERR_ALIGN;
        if (p) wr[nw++] = extent(p, state);
    }
    if (a->cu_seqlens) rd[nr++] = extent(a->cu_seqlens, (a->nseq + 1) * 4);
    for (int i = 0; i < nw; ++i) {
        for (int j = i + 1; j < nw; ++j)
            if (overlap(wr[i], wr[j])) return SDM_GX_ERR_OVERLAP;
        for (int j = 0; j < nr; ++j)
            if (overlap(wr[i], rd[j])) return SDM_GX_ERR_OVERLAP;
    }
    return SDM_GX_OK;
}

// Chunk slots: sequence i's chunks start at slot i * ceil(T / 64), or for packed runs at cu_seqlens[i] / 64 + i,
// which leaves every run room for its last, partial chunk without the host knowing the lengths.
int64_t slots_of(const sdm_gdr_args_t* a) {
    return a->cu_seqlens ? a->T / kChunk + a->nseq + 1 : a->B * cdiv(a->T, kChunk);
}

int64_t padded_dk(int64_t dk) { return dk <= 64 ? 64 : dk <= 128 ? 128 : 256; }

// Lays the workspace out from `base`; its size.
int64_t lay_out(const sdm_gdr_args_t* a, bool backward, char* base, GdrWork* w) {
    const int64_t slots = slots_of(a), sv = slots * a->Hv, sk = slots * a->Hk;
    const int64_t in = parts_of(a->dtype), dkp = padded_dk(a->dk), dvp = (a->dv + 7) / 8 * 8;
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        char* p = base + at;
        at += (bytes + 255) / 256 * 256;
        return p;
    };
    GdrWork t{};
    t.tok = reinterpret_cast<float*>(take(sv * kTokFields * kChunk * 4));
    t.inv = reinterpret_cast<uint16_t*>(take(sv * kChunk * kChunk * 3 * 2));
    t.pm = reinterpret_cast<uint16_t*>(take(sv * kChunk * kChunk * 3 * 2));
    t.kf = reinterpret_cast<uint16_t*>(take(sk * dkp * kChunk * in * 2));
    if (!backward) t.qf = reinterpret_cast<uint16_t*>(take(sk * dkp * kChunk * in * 2));
    t.kt = reinterpret_cast<uint16_t*>(take(sk * dkp * kChunk * in * 2));
    if (backward) {
        t.invt = reinterpret_cast<uint16_t*>(take(sv * kChunk * kChunk * 3 * 2));
        t.qt = reinterpret_cast<uint16_t*>(take(sk * dkp * kChunk * in * 2));
        t.st = reinterpret_cast<float*>(take(sv * a->dk * dvp * 4));
        t.dst = reinterpret_cast<float*>(take(sv * a->dk * dvp * 4));
        t.u = reinterpret_cast<float*>(take(sv * kChunk * dvp * 4));
        t.dr = reinterpret_cast<float*>(take(sv * kChunk * dvp * 4));
        if (a->Hv != a->Hk) {
            t.dqp = reinterpret_cast<float*>(take(sv * kChunk * a->dk * 4));
            t.dkp = reinterpret_cast<float*>(take(sv * kChunk * a->dk * 4));
        }
    }
    if (w) *w = t;
    return at ? at : 1;
}

GdrLaunch plan(const sdm_gdr_args_t* a, bool backward, void* workspace) {
    GdrLaunch g{};
    g.a = *a;
    lay_out(a, backward, static_cast<char*>(workspace), &g.w);
    g.slots = static_cast<int32_t>(slots_of(a));
    g.dkp = static_cast<int32_t>(padded_dk(a->dk));
    g.dvp = static_cast<int32_t>((a->dv + 7) / 8 * 8);
    g.vec_qk = a->dk % 8 == 0;
    g.vec_v = a->dv % 8 == 0;
    return g;
}

int call(const sdm_gdr_args_t* a, bool backward, void* workspace, int64_t bytes, void* stream) {
    int st = check(a, backward), dev = 0;
    if (st) return st;
    if (!workspace) return SDM_GX_ERR_NULL;
    if (!aligned(workspace, 256)) return SDM_GX_ERR_ALIGN;
    if (bytes < lay_out(a, backward, nullptr, nullptr)) return SDM_GX_ERR_LIMIT;
    const int64_t scans = 8 * cdiv(scan_groups(*a, static_cast<int>(padded_dk(a->dk))), 8);
    if (slots_of(a) * (backward ? kGradThreads : kChunkThreads) >= kMaxThreads || scans * kScanThreads >= kMaxThreads)
        return SDM_GX_ERR_LIMIT;
    if ((st = current_gfx950(&dev))) return st;
    const void* both[] = {a->q.data, a->k.data, a->v.data, a->g.data, a->beta.data, a->cu_seqlens, a->s0, workspace};
    const void* fwd[] = {a->o.data, a->s_final};
    const void* bwd[] = {a->d_o.data, a->ds_final, a->d_q.data, a->d_k.data, a->d_v.data, a->d_g.data, a->d_beta.data,
                         a->ds0};
    for (const void* p : both)
        if (p && (st = pointer_on(p, dev))) return st;
    for (int i = 0; i < (backward ? 8 : 2); ++i)
        if (const void* p = backward ? bwd[i] : fwd[i])
            if ((st = pointer_on(p, dev))) return st;
    const GdrLaunch g = plan(a, backward, workspace);
    const hipError_t e = backward ? launch_gdr_backward(g, static_cast<hipStream_t>(stream))
                                  : launch_gdr_forward(g, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? SDM_GX_OK : record_hip_error(e);
}

int check_step(const sdm_gdr_step_args_t* a) {
    if (!a) return SDM_GX_ERR_ARG;
    if (int st = check_sizes(a->dtype, a->B, a->T, a->Hk, a->Hv, a->dk, a->dv)) return st;
    if (a->pool < 1 || a->pool >= (int64_t(1) << 31)) return SDM_GX_ERR_SHAPE;
    if (!a->slots && a->pool < a->B) return SDM_GX_ERR_SHAPE;
    if (!a->state) return SDM_GX_ERR_NULL;
    if (!aligned(a->state, 4) || !aligned(a->slots, 4)) return SDM_GX_ERR_ALIGN;
    const int64_t es = elem_size(a->dtype);
    const Operand in[] = {{&a->q, a->Hk, a->dk, es}, {&a->k, a->Hk, a->dk, es}, {&a->v, a->Hv, a->dv, es},
                          {&a->g, a->Hv, 1, 4},      {&a->beta, a->Hv, 1, 4}};
    const Operand o{&a->o, a->Hv, a->dv, es};
    Extent rd[6], wr[2];
    for (int i = 0; i < 5; ++i)
        if (int st = check_rows(in[i], a->B, a->T, &rd[i])) return st;
    if (int st = check_rows(o, a->B, a->T, &wr[0])) return st;
    if (int st = check_written(o, a->B, a->T)) return st;
    wr[1] = extent(a->state, a->pool * a->Hv * a->dk * a->dv * 4);
    rd[5] = extent(a->slots, a->slots ? a->B * 4 : 0);
    if (overlap(wr[0], wr[1])) return SDM_GX_ERR_OVERLAP;
    for (const Extent& w : wr)
        for (const Extent& r : rd)
            if (overlap(w, r)) return SDM_GX_ERR_OVERLAP;
    return SDM_GX_OK;
}

}  // namespace

extern "C" {

int sdm_gdr_check(const sdm_gdr_args_t* args, int32_t backward) { return check(args, backward != 0); }

int64_t sdm_gdr_workspace(const sdm_gdr_args_t* args, int32_t backward) {
    if (!args) return SDM_GX_ERR_ARG;
    if (int st = check_sizes(args->dtype, args->B, args->T, args->Hk, args->Hv, args->dk, args->dv)) return st;
    if (args->nseq < 1 || args->nseq >= (int64_t(1) << 20)) return SDM_GX_ERR_SHAPE;
    return lay_out(args, backward != 0, nullptr, nullptr);
}

int sdm_gdr_forward(const sdm_gdr_args_t* args, void* workspace, int64_t workspace_bytes, void* stream) {
    return call(args, false, workspace, workspace_bytes, stream);
}

int sdm_gdr_backward(const sdm_gdr_args_t* args, void* workspace, int64_t workspace_bytes, void* stream) {
    return call(args, true, workspace, workspace_bytes, stream);
}

int sdm_gdr_step_check(const sdm_gdr_step_args_t* args) { return check_step(args); }

int sdm_gdr_step(const sdm_gdr_step_args_t* a, void* stream) {
    int st = check_step(a), dev = 0;
    if (st || a->T == 0) return st;
    if (step_groups(*a) * kStepThreads >= kMaxThreads) return SDM_GX_ERR_LIMIT;
    if ((st = current_gfx950(&dev))) return st;
    const void* ps[] = {a->q.data, a->k.data, a->v.data, a->g.data, a->beta.data, a->o.data, a->state, a->slots};
    for (const void* p : ps)
        if (p && (st = pointer_on(p, dev))) return st;
    const bool vec = a->dv % 4 == 0 && aligned(a->state, 16);
    const hipError_t e = launch_gdr_step(*a, vec, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? SDM_GX_OK : record_hip_error(e);
}

const char* sdm_delta_strerror(int code) {
    switch (code) {
        case SDM_GX_OK: return "ok";
        case SDM_GX_ERR_NULL: return "a required pointer is NULL";
        case SDM_GX_ERR_SHAPE: return "sizes out of range (see the header's limits)";
        case SDM_GX_ERR_ALIGN: return "a pointer is not aligned to its elements, or a workspace to 256 (norm: 16) bytes";
        case SDM_GX_ERR_OVERLAP: return "an output overlaps an input or another output";
        case SDM_GX_ERR_STRIDE: return "stride out of range, or rows of an output that overlap each other";
        case SDM_GX_ERR_LIMIT: return "workspace too small, or the launch exceeds a device limit";
        case SDM_GX_ERR_HIP: return "HIP runtime error (see sdm_delta_last_hip_error)";
        case SDM_GX_ERR_DEVICE: return "no gfx950 device, or a pointer is not on the current device";
        case SDM_GX_ERR_ARG: return "invalid argument";
        default: return "unknown status";
    }
}

int sdm_delta_last_hip_error(void) { return t_last_hip_error; }

}  // extern "C"
