// Host entry points of the gated feed-forward product (sdm_ffn.h): argument checks, workspaces, the order of the launches.
// The arithmetic is in the ffn_*.hip files.
#include <algorithm>
#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/sdm_ffn.h"
#include "delta_host.h"
#include "ffn.h"

using namespace sdm_delta;

namespace {

constexpr int64_t kMaxRows = int64_t(1) << 21, kMaxWidth = int64_t(1) << 20;    // 256 rows of any operand stay below 2 GB
constexpr int64_t kMaxThreads = int64_t(1) << 32;

int64_t size_of(int dtype) { return dtype == SDM_E4M3 ? 1 : elem_size(dtype); }
int64_t up_to(int64_t n, int64_t m) { return cdiv(n, m) * m; }

struct Row {
    const void* p;
    int64_t ld, rows, cols, size;
};

int check(const sdm_ffn_args_t* a, bool backward) {
    if (!a) return SDM_GX_ERR_ARG;
    const bool bytes = a->dtype == SDM_E4M3;
    if (a->dtype < SDM_F32 || a->dtype > SDM_E4M3 || (bytes && backward)) return SDM_GX_ERR_ARG;
    if (bytes ? a->otype != SDM_BF16 && a->otype != SDM_F16 : a->otype != a->dtype) return SDM_GX_ERR_ARG;
    if (a->act < SDM_ACT_NONE || a->act > SDM_ACT_GELU) return SDM_GX_ERR_ARG;
    if (a->M < (backward ? 1 : 0) || a->M > kMaxRows || a->K < 1 || a->K > kMaxWidth || a->F < 1 || a->F > kMaxWidth) return SDM_GX_ERR_SHAPE;
    if (!a->x || !a->wg || !a->wu) return SDM_GX_ERR_NULL;
    if (bytes ? !a->sx || !a->sg || !a->su : a->sx || a->sg || a->su) return bytes ? SDM_GX_ERR_NULL : SDM_GX_ERR_ARG;
    const int64_t es = size_of(a->dtype), os = elem_size(a->otype), M = a->M, K = a->K, F = a->F;
    Row in[8], out[4];
    int ni = 0, no = 0;
    in[ni++] = {a->x, a->ld_x, M, K, es};
    in[ni++] = {a->wg, a->ld_wg, F, K, es};
    in[ni++] = {a->wu, a->ld_wu, F, K, es};
    if (bytes) {
        in[ni++] = {a->sx, 1, M, 1, 4};
        in[ni++] = {a->sg, 1, F, 1, 4};
        in[ni++] = {a->su, 1, F, 1, 4};
    }
    if (backward) {
        if (!a->dh || !a->gate || !a->up || !a->dx || !a->dwg || !a->dwu) return SDM_GX_ERR_NULL;
        in[ni++] = {a->dh, a->ld_dh, M, F, es};
        in[ni++] = {a->gate, a->ld_gate, M, F, 4};
        in[ni++] = {a->up, a->ld_up, M, F, 4};
        out[no++] = {a->dx, a->ld_dx, M, K, es};
        out[no++] = {a->dwg, a->ld_dwg, F, K, es};
        out[no++] = {a->dwu, a->ld_dwu, F, K, es};
    } else {
        if (!a->h || !a->gate != !a->up) return SDM_GX_ERR_NULL;
        out[no++] = {a->h, a->ld_h, M, F, os};
        if (a->gate) {
            out[no++] = {a->gate, a->ld_gate, M, F, 4};
            out[no++] = {a->up, a->ld_up, M, F, 4};
        }
    }
    for (int i = 0; i < ni + no; ++i) {
        const Row& r = i < ni ? in[i] : out[i - ni];
        if (r.ld < r.cols || r.ld >= SDM_GX_LD_LIMIT) return SDM_GX_ERR_STRIDE;
        if (!aligned(r.p, r.size)) return SDM_GX_ERR_ALIGN;
    }
    auto span = [](const Row& r) { return extent(r.p, r.rows ? ((r.rows - 1) * r.ld + r.cols) * r.size : 0); };     // below 2^55
    for (int i = 0; i < no; ++i) {
        for (int j = i + 1; j < no; ++j)
            if (overlap(span(out[i]), span(out[j]))) return SDM_GX_ERR_OVERLAP;
        for (int j = 0; j < ni; ++j)
            if (overlap(span(out[i]), span(in[j]))) return SDM_GX_ERR_OVERLAP;
    }
    return SDM_GX_OK;
}

// Workspace taken piece by piece; without a base it only counts.
struct Space {
    char* base;
    int64_t used;
    char* take(int64_t bytes) {
        char* p = base ? base + used : nullptr;
        used += up_to(bytes, 256);
        return p;
    }
};

// A product's operand from rows of `src`: where they lie, or laid out anew.
struct Laid {
    FfnOperand o;
    FfnLay lay;
    bool anew;
};
Laid operand(const void* src, int64_t ld, int64_t R, int64_t C, int dtype, Space* s) {
    const int64_t es = size_of(dtype);
    Laid l{};
    l.anew = !aligned(src, 16) || ld * es % 16 || C * es % 16 || ld * es >= (int64_t(1) << 22);
    if (!l.anew) {
        l.o = FfnOperand{static_cast<const char*>(src), ld * es};
        return l;
    }
    const int64_t pad = up_to(C, 16 / es), row = pad * es;
    char* p = s->take(R * row);
    l.o = FfnOperand{p, row};
    l.lay = FfnLay{src, ld, R, C, dtype, p, row, pad, 0};
    return l;
}

int product_type(int dtype) { return dtype == SDM_E4M3 ? kE4m3 : dtype == SDM_F32 ? kF32 : dtype == SDM_F16 ? kF16 : kBf16; }

// 256 x 256 tiles read half of what 128 x 128 ones do for each product, and these half of 64 x 64 ones: the largest of which
// there are enough for every CU, but where a second round of 256 x 256 ones would be half empty (one a CU, where two of 128 x 128
// fit). 4096 values a row, bfloat16 and 8 bits, tiles of 256 and of 128 in us: 256 tiles of 256 119 and 139, 65 and 75; 261 of
// them 187 and 162, 106 and 91; 320 194 and 172, 108 and 94; 416 205 and 230, 114 and 125; 512 231 and 267, 126 and 143. Tiles of
// 64 instead of 256 of 128: 69 and 42 (2048 rows of 2048 to 2048), instead of fewer 21 and 22 (1024 of 2048 to 1024). float32's six
// products a value are enough for 128 x 128 ones; their parts and the sums of larger ones would not fit the registers.
int64_t pair_tiles(int64_t M, int64_t F, int tile) { return cdiv(M, tile) * cdiv(F, tile / 2); }
int pair_tile(int64_t M, int64_t F, int dtype) {
    const int64_t large = dtype == SDM_F32 ? 0 : pair_tiles(M, F, 256);
    return large == 256 || large >= 384 ? 256 : pair_tiles(M, F, 128) >= 256 ? 128 : 64;
}
// dx and both weights' gradients: 400 tiles of 256 and more of 128 198 and 202 us, 608 319 and 348, 768 562 and 631
int64_t gradient_tiles(int64_t M, int64_t K, int64_t F, int tile) { return (cdiv(M, tile) + cdiv(2 * F, tile)) * cdiv(K, tile); }
int gradient_tile(int64_t M, int64_t K, int64_t F, int dtype) {
    return dtype != SDM_F32 && gradient_tiles(M, K, F, 256) >= 256 ? 256 : gradient_tiles(M, K, F, 128) >= 256 ? 128 : 64;
}

bool few(const sdm_ffn_args_t* a) { return a->M <= (a->dtype == SDM_F32 ? kFfnFewFloatRows : kFfnFewRows); }

struct Forward {
    int tile;
    Laid x, wg, wu;
    int64_t bytes;      // of the workspace
};
Forward forward_plan(const sdm_ffn_args_t* a, char* ws) {
    Space s{ws, 0};
    Forward f{};
    if (few(a)) return f;
    f.tile = pair_tile(a->M, a->F, a->dtype);
    f.x = operand(a->x, a->ld_x, a->M, a->K, a->dtype, &s);
    f.wg = operand(a->wg, a->ld_wg, a->F, a->K, a->dtype, &s);
    f.wu = operand(a->wu, a->ld_wu, a->F, a->K, a->dtype, &s);
    f.bytes = s.used;
    return f;
}

// Rounding dg and du to 16 bits adds to a gradient's error, on average over many values, what rounding the gradient itself does:
// sqrt(2) times the error of the rounded result alone. The fewer values there are of dg and du (M F) and of the gradients (M K, F
// K), the further a call is from that average: with 4096 of the fewest the errors of 500 random calls are up to 1.53 times the
// rounded result's, with 256 up to 1.7, with 4 up to 15. Up to 4096 dg and du come in two parts, and what they meet in the products
// twice: 1.0 (8192 rows of 64 to 64: 29 us, in one part 23). Above, as the caller has it (8192 rows of 4096 to 8192: 3800 us, in one part 2000).
int gradient_parts(const sdm_ffn_args_t* a) {
    if (a->dtype == SDM_F32) return 1;
    return a->precise || std::min(a->M, std::max(a->K, a->F)) * std::min(a->K, a->F) <= 4096 ? 2 : 1;
}

// A product of few tiles and a long sum is cut into parts along the sum, up to two workgroups a CU (tiles of 256: one), of 8
// steps of 128 bytes at the least, where that saves 40 steps: joining them is one more launch (333 rows of 1111 to 777 in
// float32, 36 steps saved: 80 us in parts and 78 without). bfloat16 training steps in parts and without: 100 rows of 1024 to 8192 73 and 281 us, 64 of 4096 to 8192 199 and 446, 8192 of
// 64 to 128 36 and 54.
struct Cut {
    int64_t part;
    int parts;
};
Cut cut(int64_t M, int64_t N, int64_t bytes, int tile) {
    const int64_t steps = cdiv(bytes, 128), have = cdiv(M, tile) * cdiv(N, tile);
    const int64_t most = std::min(steps / 8, (tile == 256 ? 256 : 512) / have);
    if (most < 2) return {up_to(bytes, 128), 1};
    const int64_t each = cdiv(steps, most);
    if (steps - each < 40) return {up_to(bytes, 128), 1};
    return {each * 128, static_cast<int>(cdiv(steps, each))};
}

struct Backward {
    int tile;
    Cut dx, dw;
    float *dx_parts, *dw_parts;
    FfnGrad grad;
    FfnLay wg, wu, x;
    FfnOperand rows, cols, w, xt;
    int64_t bytes;
};
Backward backward_plan(const sdm_ffn_args_t* a, char* ws) {
    Space s{ws, 0};
    Backward b{};
    b.tile = gradient_tile(a->M, a->K, a->F, a->dtype);
    const int64_t es = size_of(a->dtype);
    const int64_t M = a->M, K = a->K, F = a->F, Mp = up_to(M, 16 / es), Fp = up_to(F, 16 / es), parts = gradient_parts(a);
    auto area = [&](int64_t rows, int64_t cols, FfnOperand* o) {
        char* p = s.take(rows * cols * es);
        *o = FfnOperand{p, cols * es};
        return p;
    };
    char* rows = area(M, 2 * parts * Fp, &b.rows);
    char* cols = area(2 * F, parts * Mp, &b.cols);
    char* w = area(K, 2 * parts * Fp, &b.w);
    char* xt = area(K, parts * Mp, &b.xt);
    b.grad = FfnGrad{a->dh, a->gate, a->up, a->ld_dh, a->ld_gate, a->ld_up, M, F, Mp, Fp, a->dtype, a->act, static_cast<int>(parts), rows, cols};
    b.wg = FfnLay{a->wg, a->ld_wg, F, K, a->dtype, w, b.w.ld, Fp, parts == 2 ? 2 * Fp * es : 0};
    b.wu = b.wg;
    b.wu.src = a->wu;
    b.wu.ld = a->ld_wu;
    b.wu.dst = w + Fp * es;
    b.x = FfnLay{a->x, a->ld_x, M, K, a->dtype, xt, b.xt.ld, Mp, parts == 2 ? Mp * es : 0};
    const int64_t wide = up_to(K, 4);
    b.dx = cut(M, K, b.rows.ld, b.tile);
    b.dw = cut(2 * F, K, b.cols.ld, b.tile);
    if (b.dx.parts > 1) b.dx_parts = reinterpret_cast<float*>(s.take(b.dx.parts * M * wide * 4));
    if (b.dw.parts > 1) b.dw_parts = reinterpret_cast<float*>(s.take(b.dw.parts * 2 * F * wide * 4));
    b.bytes = s.used;
    return b;
}

int prepare(const sdm_ffn_args_t* a, bool backward, int64_t need, void* ws, int64_t ws_bytes) {
    if (need && !ws) return SDM_GX_ERR_NULL;
    if (!aligned(ws, 256)) return SDM_GX_ERR_ALIGN;
    if (ws_bytes < need) return SDM_GX_ERR_LIMIT;
    int dev = 0, st = current_gfx950(&dev);
    if (st) return st;
    const void* ps[] = {a->x, a->wg, a->wu, a->sx, a->sg, a->su, a->gate, a->up, need ? ws : nullptr, backward ? a->dh : a->h,
                        backward ? a->dx : nullptr, backward ? a->dwg : nullptr, backward ? a->dwu : nullptr};
    for (const void* p : ps)
        if (p && (st = pointer_on(p, dev))) return st;
    return SDM_GX_OK;
}

int status(hipError_t e) { return e == hipSuccess ? SDM_GX_OK : record_hip_error(e); }

}  // namespace

extern "C" {

int sdm_ffn_check(const sdm_ffn_args_t* args, int32_t backward) { return check(args, backward != 0); }

int64_t sdm_ffn_workspace(const sdm_ffn_args_t* a, int32_t backward) {
    if (int st = check(a, backward != 0)) return st;
    return backward ? backward_plan(a, nullptr).bytes : forward_plan(a, nullptr).bytes;
}

int sdm_ffn_forward(const sdm_ffn_args_t* a, void* ws, int64_t ws_bytes, void* stream) {
    int st = check(a, false);
    if (st || a->M == 0) return st;
    const Forward f = forward_plan(a, static_cast<char*>(ws));
    const hipStream_t s = static_cast<hipStream_t>(stream);
    FfnProduct p{};
    p.A = f.x.o;
    p.B = f.wg.o;
    p.B2 = f.wu.o;
    p.M = a->M;
    p.N = a->F;
    p.bytes = up_to(a->K * size_of(a->dtype), 16);
    p.type = product_type(a->dtype);
    p.act = a->act;
    p.otype = a->otype;
    p.sm = a->sx;
    p.sn = a->sg;
    p.sn2 = a->su;
    p.c = static_cast<char*>(a->h);
    p.ldc = a->ld_h;
    p.split = a->M;
    p.gate = a->gate;
    p.up = a->up;
    p.ld_gate = a->ld_gate;
    p.ld_up = a->ld_up;
    if (!few(a) && pair_tiles(a->M, a->F, f.tile) * 512 >= kMaxThreads) return SDM_GX_ERR_LIMIT;
    int64_t threads = 0;
    for (const Laid* l : {&f.x, &f.wg, &f.wu}) threads += l->lay.R * cdiv(l->lay.pad * size_of(a->dtype), 16) + 256;
    if (threads >= kMaxThreads) return SDM_GX_ERR_LIMIT;
    if ((st = prepare(a, false, f.bytes, ws, ws_bytes))) return st;
    if (few(a)) return status(launch_ffn_few(*a, s));
    // an operand used where it lies has no rows to lay out
    const FfnLay lay[3] = {f.x.lay, f.wg.lay, f.wu.lay};
    if (const hipError_t e = launch_ffn_lay(lay, s)) return status(e);
    return status(launch_ffn_pair(p, f.tile, s));
}

int sdm_ffn_backward(const sdm_ffn_args_t* a, void* ws, int64_t ws_bytes, void* stream) {
    int st = check(a, true);
    if (st) return st;
    const Backward b = backward_plan(a, static_cast<char*>(ws));
    const hipStream_t s = static_cast<hipStream_t>(stream);
    FfnProduct both[2] = {}, &dx = both[0], &dw = both[1];
    dx.A = b.rows;
    dx.B = b.w;
    dx.M = a->M;
    dx.N = a->K;
    dx.bytes = b.rows.ld;
    dx.c = static_cast<char*>(a->dx);
    dx.ldc = a->ld_dx;
    dx.split = a->M;
    dw.A = b.cols;
    dw.B = b.xt;
    dw.M = 2 * a->F;
    dw.N = a->K;
    dw.bytes = b.cols.ld;
    dw.c = static_cast<char*>(a->dwg);
    dw.c2 = static_cast<char*>(a->dwu);
    dw.ldc = a->ld_dwg;
    dw.ldc2 = a->ld_dwu;
    dw.split = a->F;
    FfnJoin join[2] = {};
    const Cut cuts[2] = {b.dx, b.dw};
    float* const areas[2] = {b.dx_parts, b.dw_parts};
    for (int i = 0; i < 2; ++i) {
        FfnProduct& p = both[i];
        p.type = product_type(a->dtype);
        p.otype = a->otype;
        p.part = cuts[i].part;
        p.parts = cuts[i].parts;
        if (p.parts == 1) continue;
        join[i] = FfnJoin{areas[i], p.M, p.N, up_to(p.N, 4), p.parts, p.otype, p.c, p.c2, p.ldc, p.ldc2, p.split};
        p.otype = SDM_F32;
        p.c = reinterpret_cast<char*>(areas[i]);
        p.ldc = join[i].ld;
        p.split = p.M;
    }
    if ((gradient_tiles(a->M, a->K, a->F, b.tile) + 1024) * 512 >= kMaxThreads) return SDM_GX_ERR_LIMIT;
    const int64_t gm = cdiv(b.grad.Mp, 64), gf = cdiv(b.grad.Fp, 64), gk = cdiv(a->K, 64);
    if ((gm * gf + (gm + 2 * gf) * gk) * 256 >= kMaxThreads) return SDM_GX_ERR_LIMIT;
    if ((st = prepare(a, true, b.bytes, ws, ws_bytes))) return st;
    const FfnLay lay[3] = {b.wg, b.wu, b.x};
    if (const hipError_t e = launch_ffn_grad(b.grad, lay, s)) return status(e);
    if (const hipError_t e = launch_ffn_products(both, b.tile, s)) return status(e);
    return status(launch_ffn_join(join, s));
}

}  // extern "C"
