// The norms after a block and before the next with the block's gate and residual scale (sdm_nrm.h), forward and
// backward, for gfx950.
//
// What bounds them is memory: the forward reads x, o, z and writes x', y, the backward reads dx', dy, x', o, z and
// writes dx, do, dz, each once. A row lives in the registers of one workgroup from its load to its store, so the two
// norms of a row, which depend on each other, cost two workgroup reductions and no second pass. Workgroups take many
// rows each: the weights stay in registers (in LDS in the backward), and in the backward so do their gradients' sums,
// which leave once per workgroup as partial sums that a second kernel adds in workgroup order.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "delta_types.h"
#include "nrm.h"

namespace sdm_delta {
namespace {

// Rows are read once: past the caches (16384 x 4096 rows, inputs in turn: in bfloat16 forward 133 -> 111 us, backward 201 ->
// 198; in float32 forward 247 -> 260, the other way).
constexpr bool kStream = true;

// The sum of v over the workgroup, in an order set by the lane and wavefront numbers alone. `buf` alternates between
// two LDS rows: a row is written again only after a barrier that follows its last read.
template <int NT>
__device__ __forceinline__ float row_sum(float v, float (*red)[16], int buf) {
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m, 64);
    if constexpr (NT > 64) {
        if ((threadIdx.x & 63) == 0) red[buf][threadIdx.x >> 6] = v;
        lds_barrier();
        v = 0.f;
#pragma unroll
        for (int i = 0; i < NT / 64; ++i)
            if (i < static_cast<int>(blockDim.x >> 6)) v += red[buf][i];
    }
    return v;
}

// act(z) and act'(z). With e = exp(-|z|) the sigmoid p and 1 - p are 1 / (1 + e) and e / (1 + e), in the order of z's sign:
// 1 - p taken as a difference would keep nothing of act' from z = 17 on. The 16-bit types take the hardware's exponential
// and reciprocal (1 ulp of float32), float32 the library's.
template <int DT>
__device__ __forceinline__ void gate(float z, int act, float& a, float& d) {
    float e, large;
    if constexpr (DT == 0) {
        e = expf(-fabsf(z));
        large = 1.f / (1.f + e);
    } else {
        e = __builtin_amdgcn_exp2f(-1.44269504f * fabsf(z));
        large = __builtin_amdgcn_rcpf(1.f + e);
    }
    const float small = e * large, p = z < 0.f ? small : large, q = z < 0.f ? large : small;
    if (act == SDM_ACT_SIGMOID) {
        a = p;
        d = p * q;
    } else {
        a = z * p;
        d = p * (1.f + z * q);
    }
}

// Weights as they lie in memory, and a weight's floats as of this use: left to itself the compiler converts 16-bit weights
// before the row loop and keeps twice the registers.
template <int WT>
__device__ __forceinline__ void load_weights(Raw<WT>& r, const void* w, int c, int D) {
    float f[8];
    load8<WT>(f, static_cast<const elem_t<WT>*>(w), c, D);
    if constexpr (WT == 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) r.w[i / 4][i % 4] = __float_as_uint(f[i]);
    } else {
        typedef elem_t<WT> t8 __attribute__((ext_vector_type(8)));
        t8 a;
#pragma unroll
        for (int i = 0; i < 8; ++i) a[i] = static_cast<elem_t<WT>>(f[i]);
        r.w[0] = __builtin_bit_cast(u32x4, a);
    }
}
template <int WT>
__device__ __forceinline__ void weight_floats(float (&f)[8], Raw<WT> r) {
    if constexpr (WT != 0) asm volatile("" : "+v"(r.w[0]));
    raw_floats<WT>(f, r);
}

// The next row's loads are in flight while a row is worked on (in bfloat16, inputs in turn: 16384 x 4096 rows 157 -> 109
// us, 6.1 TB/s; 8192 x 8192 197 -> 119; 2048 x 4096 29.6 -> 21.2). A row's end is loaded without a branch (load_row) and
// moved once it has come; with a branch its loads would wait for one another and for the row before them (20000 rows of
// 1111 in bfloat16: forward 110 -> 63 us and backward 277 -> 131, the wavefronts past the row left out too).
template <int DT, int WT, int NT, int NV>
__global__ __launch_bounds__(NT) void nrm_forward(const sdm_nrm_args_t a) {
    using T = elem_t<DT>;
    __shared__ float red[2][16];
    const int D = static_cast<int>(a.D), id = static_cast<int>(threadIdx.x), nt = static_cast<int>(blockDim.x);
    const float inv = 1.f / static_cast<float>(D);
    const bool has_o = a.o != nullptr, has_x = a.x != nullptr, has_y = a.w_pre != nullptr;
    const bool has_z = a.act != SDM_ACT_NONE;
    struct {
        Raw<DT> x[NV], o[NV], z[NV];
    } in;
    auto fetch = [&](int64_t r) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * nt + id) * 8;
            if (has_o) load_row<DT, kStream>(in.o[v], static_cast<const T*>(a.o) + r * a.ld_o, c, D);
            if (has_z) load_row<DT, kStream>(in.z[v], static_cast<const T*>(a.z) + r * a.ld_z, c, D);
            if (has_x) load_row<DT, kStream>(in.x[v], static_cast<const T*>(a.x) + r * a.ld_x, c, D);
        }
    };
    fetch(blockIdx.x);
    Raw<WT> w1[NV], w2[NV], sc[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int c = (v * nt + id) * 8;
        if (has_o) {
            load_weights<WT>(w1[v], a.w_post, c, D);
            load_weights<WT>(sc[v], a.scale, c, D);
        }
        if (has_y) load_weights<WT>(w2[v], a.w_pre, c, D);
    }
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        float x[NV][8], o[NV][8], z[NV][8];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            raw_floats<DT>(o[v], in.o[v]);
            raw_floats<DT>(z[v], in.z[v]);
            if (has_x) {
                raw_floats<DT>(x[v], in.x[v]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) x[v][i] = 0.f;
            }
            const int past = (v * nt + id) * 8 + 8 - D;
            if (__builtin_expect(past > 0 && D >= 8, 0)) {
                move_down(o[v], past);
                move_down(z[v], past);
                move_down(x[v], past);
            }
        }
        if (r + gridDim.x < a.rows) fetch(r + gridDim.x);
        float r1 = 0.f, r2 = 0.f;
        if (has_o) {
            float s = 0.f;
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int i = 0; i < 8; ++i) s = fmaf(o[v][i], o[v][i], s);
            r1 = 1.f / sqrtf(fmaf(row_sum<NT>(s, red, 0), inv, a.eps));
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                float w[8], s[8];
                weight_floats<WT>(w, w1[v]);
                weight_floats<WT>(s, sc[v]);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float g = 1.f, d;
                    if (has_z) gate<DT>(z[v][i], a.act, g, d);
                    // rounded to the residual's type here: the second norm is that of the stored row
                    x[v][i] = static_cast<float>(static_cast<T>(fmaf(s[i], o[v][i] * r1 * w[i] * g, x[v][i])));
                }
                store8(static_cast<T*>(a.x_new) + r * a.ld_xn, (v * nt + id) * 8, D, x[v]);
            }
        }
        if (has_y) {
            float s = 0.f;
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int i = 0; i < 8; ++i) s = fmaf(x[v][i], x[v][i], s);
            r2 = 1.f / sqrtf(fmaf(row_sum<NT>(s, red, 1), inv, a.eps));
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                float w[8];
                weight_floats<WT>(w, w2[v]);
#pragma unroll
                for (int i = 0; i < 8; ++i) x[v][i] = x[v][i] * r2 * w[i];
                store8(static_cast<T*>(a.y) + r * a.ld_y, (v * nt + id) * 8, D, x[v]);
            }
        }
        if (threadIdx.x == 0) {
            a.rstd[2 * r] = r1;
            a.rstd[2 * r + 1] = r2;
        }
        // a call with one norm reads and writes one LDS row only: keep a fast wavefront out of the next row's
        if (NT > 64 && has_o != has_y) lds_barrier();
    }
}

// The weights wait in LDS and the next row's loads are in flight while a row is worked on: a row's two dependent sums
// leave memory nothing to do otherwise.
template <int DT, int WT, int NT, int NV>
__global__ __launch_bounds__(NT) void nrm_backward(const sdm_nrm_args_t a, float* __restrict__ part) {
    using T = elem_t<DT>;
    using W = elem_t<WT>;
    __shared__ float red[2][16];
    // each thread's own columns: w_post, scale, w_pre; for long rows, whose values fill the registers, dw_pre's sum too
    __shared__ alignas(16) float wt[NV == 1 ? 3 : 4][NV][NT][8];
    const int D = static_cast<int>(a.D), id = static_cast<int>(threadIdx.x);
    const float inv = 1.f / static_cast<float>(D);
    const bool has_o = a.o != nullptr, has_y = a.w_pre != nullptr, has_up = a.dxn != nullptr;
    const bool has_z = a.act != SDM_ACT_NONE;
    // sums over this workgroup's rows: dx n act(z), which times scale is dw_post's and times w_post dscale's, and dw_pre's
    float s1[NV][8], s2[NV][8];
    struct {
        Raw<DT> dx[NV], y[NV], xn[NV], o[NV], z[NV];
        float r1, r2;
    } in;
    auto fetch = [&](int64_t r) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * NT + id) * 8;
            if (has_y) {
                load_row<DT, kStream>(in.y[v], static_cast<const T*>(a.dy) + r * a.ld_dy, c, D);
                load_row<DT, kStream>(in.xn[v], static_cast<const T*>(a.x_new) + r * a.ld_xn, c, D);
            }
            if (has_up) load_row<DT, kStream>(in.dx[v], static_cast<const T*>(a.dxn) + r * a.ld_dxn, c, D);
        }
        in.r1 = a.rstd[2 * r];
        in.r2 = a.rstd[2 * r + 1];
    };
    auto fetch_o = [&](int64_t r) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * NT + id) * 8;
            if (has_o) load_row<DT, kStream>(in.o[v], static_cast<const T*>(a.o) + r * a.ld_o, c, D);
            if (has_z) load_row<DT, kStream>(in.z[v], static_cast<const T*>(a.z) + r * a.ld_z, c, D);
        }
    };
    constexpr bool AHEAD = NV == 1;     // registers hold the next row beside this one
    int64_t r = blockIdx.x;
    if (AHEAD && r < a.rows) {
        fetch(r);
        fetch_o(r);
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int c = (v * NT + id) * 8;
        float f[8];
        auto keep = [&](int k, const void* w) {
            load8<WT>(f, static_cast<const W*>(w), c, D);
#pragma unroll
            for (int i = 0; i < 8; ++i) wt[k][v][id][i] = f[i];
        };
        if (has_o) {
            keep(0, a.w_post);
            keep(1, a.scale);
        }
        if (has_y) keep(2, a.w_pre);
#pragma unroll
        for (int i = 0; i < 8; ++i) s1[v][i] = s2[v][i] = 0.f;
        if constexpr (NV > 1)
            for (int i = 0; i < 8; ++i) wt[3][v][id][i] = 0.f;
    }
    for (; r < a.rows; r += gridDim.x) {
        if (!AHEAD) fetch(r);
        float dx[NV][8], y[NV][8], xn[NV][8], o[NV][8], z[NV][8];
        const float r1 = in.r1, r2 = in.r2;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            raw_floats<DT>(y[v], in.y[v]);
            raw_floats<DT>(xn[v], in.xn[v]);
            if (AHEAD) {
                raw_floats<DT>(o[v], in.o[v]);
                raw_floats<DT>(z[v], in.z[v]);
            }
            if (has_up) {
                raw_floats<DT>(dx[v], in.dx[v]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) dx[v][i] = 0.f;
            }
            const int past = (v * NT + id) * 8 + 8 - D;
            if (__builtin_expect(past > 0 && D >= 8, 0)) {
                move_down(y[v], past);
                move_down(xn[v], past);
                move_down(dx[v], past);
                if (AHEAD) {
                    move_down(o[v], past);
                    move_down(z[v], past);
                }
            }
        }
        if (AHEAD) {
            const int64_t next = r + gridDim.x < a.rows ? r + gridDim.x : r;    // the last row again: it costs little
            fetch(next);
            fetch_o(next);
        }
        if (has_y) {
            float s = 0.f;
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    xn[v][i] *= r2;
                    float& s2r = NV == 1 ? s2[v][i] : wt[NV == 1 ? 0 : 3][v][id][i];
                    s2r = fmaf(y[v][i], xn[v][i], s2r);
                    const float yw = y[v][i] * wt[2][v][id][i];
                    s = fmaf(yw, xn[v][i], s);
                    dx[v][i] = fmaf(r2, yw, dx[v][i]);
                }
            const float m = row_sum<NT>(s, red, 0) * inv * r2;
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int i = 0; i < 8; ++i) dx[v][i] = fmaf(-m, xn[v][i], dx[v][i]);
        }
        if (a.dx) {
#pragma unroll
            for (int v = 0; v < NV; ++v) store8(static_cast<T*>(a.dx) + r * a.ld_dx, (v * NT + id) * 8, D, dx[v]);
        }
        if (has_o) {
            float s = 0.f;
            if (!AHEAD) {
                fetch_o(r);
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    raw_floats<DT>(o[v], in.o[v]);
                    raw_floats<DT>(z[v], in.z[v]);
                    const int past = (v * NT + id) * 8 + 8 - D;
                    if (__builtin_expect(past > 0 && D >= 8, 0)) {
                        move_down(o[v], past);
                        move_down(z[v], past);
                    }
                }
            }
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float g = 1.f, d = 0.f;
                    if (has_z) gate<DT>(z[v][i], a.act, g, d);
                    const float w1 = wt[0][v][id][i], sc = wt[1][v][id][i];
                    const float n = o[v][i] * r1, u = dx[v][i] * n;
                    z[v][i] = u * sc * w1 * d;
                    s1[v][i] = fmaf(u, g, s1[v][i]);
                    dx[v][i] *= sc * g * w1;
                    o[v][i] = n;
                    s = fmaf(dx[v][i], n, s);
                }
            if (has_z) {
#pragma unroll
                for (int v = 0; v < NV; ++v) store8(static_cast<T*>(a.dz) + r * a.ld_dz, (v * NT + id) * 8, D, z[v]);
            }
            const float m = row_sum<NT>(s, red, 1) * inv;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int c = (v * NT + id) * 8;
#pragma unroll
                for (int i = 0; i < 8; ++i) dx[v][i] = r1 * fmaf(-m, o[v][i], dx[v][i]);
                store8(static_cast<T*>(a.d_o) + r * a.ld_do, c, D, dx[v]);
            }
        }
        if (NT > 64 && has_o != has_y) lds_barrier();
    }
    float* p = part + static_cast<int64_t>(blockIdx.x) * 2 * D;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int c = (v * NT + id) * 8;
        if (has_o) store8(p, c, D, s1[v]);
        if constexpr (NV > 1)
            for (int i = 0; i < 8; ++i) s2[v][i] = wt[3][v][id][i];
        if (has_y) store8(p + D, c, D, s2[v]);
    }
}

// The weights' gradients: column sums of the partial sums. 32 columns by 8 groups of consecutive workgroups; a
// group's sum runs in workgroup order and the eight are added in order.
template <int WT>
__global__ __launch_bounds__(256) void nrm_weights(const sdm_nrm_args_t a, const float* __restrict__ part, int groups) {
    using W = elem_t<WT>;
    __shared__ float red[8][33];
    const int D = static_cast<int>(a.D), which = blockIdx.y;
    if (!(which ? a.w_pre : a.o)) return;
    const int lane = threadIdx.x & 31, grp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    const int per = (groups + 7) / 8, lo = grp * per, hi = min(groups, lo + per);
    float s = 0.f;
    if (c < D) {
        const float* p = part + static_cast<int64_t>(which) * D + c;
#pragma unroll 8
        for (int i = lo; i < hi; ++i) s += p[static_cast<int64_t>(i) * 2 * D];
    }
    red[grp][lane] = s;
    lds_barrier();
    if (grp == 0 && c < D) {
#pragma unroll
        for (int i = 1; i < 8; ++i) s += red[i][lane];
        if (which) {
            static_cast<W*>(a.dw_pre)[c] = static_cast<W>(s);
        } else {
            static_cast<W*>(a.dw_post)[c] = static_cast<W>(s * static_cast<float>(static_cast<const W*>(a.scale)[c]));
            static_cast<W*>(a.dscale)[c] = static_cast<W>(s * static_cast<float>(static_cast<const W*>(a.w_post)[c]));
        }
    }
}

template <int DT, int WT, int NT, int NV>
hipError_t run_forward(const sdm_nrm_args_t& a, const NrmPlan& p, hipStream_t s) {
    nrm_forward<DT, WT, NT, NV><<<p.groups, p.threads, 0, s>>>(a);
    return hipGetLastError();
}
template <int DT, int WT, int NT, int NV>
hipError_t run_backward(const sdm_nrm_args_t& a, const NrmPlan& p, float* part, hipStream_t s) {
    nrm_backward<DT, WT, NT, NV><<<p.groups, p.threads, 0, s>>>(a, part);
    return hipGetLastError();
}

#define SDM_NRM_SHAPES(F, ...)                                                  \
    if (p.most == 64) return F<DT, WT, 64, 1>(__VA_ARGS__);                  \
    if (p.most == 128) return F<DT, WT, 128, 1>(__VA_ARGS__);                \
    if (p.most == 256 && p.vecs == 1) return F<DT, WT, 256, 1>(__VA_ARGS__);

template <int DT, int WT>
hipError_t forward_of(const sdm_nrm_args_t& a, const NrmPlan& p, hipStream_t s) {
    SDM_NRM_SHAPES(run_forward, a, p, s)
    if (p.most == 256) return run_forward<DT, WT, 256, 2>(a, p, s);
    return run_forward<DT, WT, 512, 2>(a, p, s);
}
template <int DT, int WT>
hipError_t backward_of(const sdm_nrm_args_t& a, const NrmPlan& p, float* part, hipStream_t s) {
    SDM_NRM_SHAPES(run_backward, a, p, part, s)
    if (p.vecs == 1) return run_backward<DT, WT, 512, 1>(a, p, part, s);
    return run_backward<DT, WT, 512, 2>(a, p, part, s);
}

}  // namespace

// wtype is dtype or float32 (the host checks)
hipError_t launch_nrm_forward(const sdm_nrm_args_t& a, const NrmPlan& p, hipStream_t s) {
    if (a.dtype == SDM_F32) return forward_of<0, 0>(a, p, s);
    if (a.dtype == SDM_BF16) return a.wtype == SDM_F32 ? forward_of<1, 0>(a, p, s) : forward_of<1, 1>(a, p, s);
    return a.wtype == SDM_F32 ? forward_of<2, 0>(a, p, s) : forward_of<2, 2>(a, p, s);
}

hipError_t launch_nrm_backward(const sdm_nrm_args_t& a, const NrmPlan& p, float* part, hipStream_t s) {
    hipError_t e;
    if (a.dtype == SDM_F32)
        e = backward_of<0, 0>(a, p, part, s);
    else if (a.dtype == SDM_BF16)
        e = a.wtype == SDM_F32 ? backward_of<1, 0>(a, p, part, s) : backward_of<1, 1>(a, p, part, s);
    else
        e = a.wtype == SDM_F32 ? backward_of<2, 0>(a, p, part, s) : backward_of<2, 2>(a, p, part, s);
    if (e != hipSuccess) return e;
    const dim3 grid(static_cast<unsigned>((a.D + 31) / 32), 2);
    if (a.wtype == SDM_F32)
        nrm_weights<0><<<grid, 256, 0, s>>>(a, part, p.groups);
    else if (a.wtype == SDM_BF16)
        nrm_weights<1><<<grid, 256, 0, s>>>(a, part, p.groups);
    else
        nrm_weights<2><<<grid, 256, 0, s>>>(a, part, p.groups);
    return hipGetLastError();
}

}  // namespace sdm_delta
