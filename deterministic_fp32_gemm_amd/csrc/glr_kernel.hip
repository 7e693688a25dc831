// The gated linear recurrence (sdm_glr.h), forward, backward and recurrent form, for gfx950.
//
//     h_t = a_t h_{t-1} + x_t,  a_t = exp(g_t);   y_t = h_t act(z_t)
//
// What bounds it is memory: x, g and z are read and y written once. A stretch of tokens maps the state that enters it as
// h -> A h + H, and two stretches after one another as A = A2 A1, H = A2 H1 + H2. A workgroup owns 64 channels (a lane
// each) of one run and walks it in tiles of 128 tokens: each of 8 wavefronts holds 16 of them in registers, finds its (A,
// H), and after one barrier each composes the maps before it, in order, and runs its own tokens from the state that enters.
// The next tile's loads are in flight meanwhile. The gradient walks the tiles from the last to the first: the states come
// from the tile's mark and the same maps, and D's recurrence, e -> a_t (u_t + e) from right to left, has the same A.
//
// Runs are cut into parts where 64 channels a workgroup give too few workgroups: a first kernel finds each part's map,
// which reads x and g (or dy, z and g) once more. It walks its part away from the end at which the second kernel starts, so
// that what it read last is what is wanted first and may still be in the last-level cache.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "block_device.h"
#include "glr.h"

namespace sdm_delta {
namespace {

constexpr int NW = kGlrWaves, KT = kGlrTokens, TILE = SDM_GLR_TILE;

struct Run {
    int64_t row;        // b
    int64_t start;      // first token
    int64_t mark;       // row of marks of its first tile
    int len;
};
__device__ __forceinline__ Run run_of(const sdm_glr_args_t& a, int i) {
    Run r;
    if (a.cu_seqlens == nullptr) {
        r.row = i;
        r.start = 0;
        r.len = static_cast<int>(a.T);
        r.mark = i * ((a.T + TILE - 1) / TILE);
    } else {
        const int T = static_cast<int>(a.T);
        const int s = min(max(a.cu_seqlens[i], 0), T), e = min(max(a.cu_seqlens[i + 1], 0), T);
        r.row = 0;
        r.start = s;
        r.len = max(e - s, 0);
        r.mark = s / TILE + i;      // at most T / TILE + nseq rows, whatever the entries are
    }
    return r;
}

// One token row's element of this lane's channel; `t` is the same for the whole wavefront.
template <class T>
__device__ __forceinline__ T at(const sdm_seq_t& s, int64_t row, int64_t t, int c) {
    return (static_cast<const T*>(s.data) + row * s.batch + t * s.token)[c];
}
template <class T>
__device__ __forceinline__ void put(const sdm_seq_t& s, int64_t row, int64_t t, int c, float v) {
    (static_cast<T*>(s.data) + row * s.batch + t * s.token)[c] = static_cast<T>(v);
}
// A h + H; from no state nothing comes, also where a growing A has left float32.
__device__ __forceinline__ float enter(float A, float H, float h) { return h == 0.f ? H : __builtin_fmaf(A, h, H); }

// The wavefront's KT tokens from t, read from inside the run whatever t is.
template <class T>
__device__ __forceinline__ void fetch(T (&o)[KT], const sdm_seq_t& s, const Run& r, int t, int c) {
#pragma unroll
    for (int i = 0; i < KT; ++i) o[i] = at<T>(s, r.row, r.start + min(t + i, r.len - 1), c);
}

// The map of each part of a run: BACK that of D's recurrence, from right to left, else that of the states.
template <int DT, int GT, bool Z, bool BACK>
__global__ __launch_bounds__(kGlrThreads) void glr_parts(const sdm_glr_args_t a, const int cblocks, const int segs, float* __restrict__ part) {
    using T = elem_t<DT>;
    using G = elem_t<GT>;
    __shared__ float ex[NW][2][64];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int cb = blockIdx.x % cblocks, rs = blockIdx.x / cblocks, seg = rs % segs, run = rs / segs;
    const Run r = run_of(a, run);
    const int D = static_cast<int>(a.D), c = cb * 64 + lane, cc = min(c, D - 1);
    const int seglen = ((r.len + segs - 1) / segs + TILE - 1) / TILE * TILE;
    const int64_t s0 = static_cast<int64_t>(seg) * seglen;
    if (s0 >= r.len) return;                                        // never asked for
    const int t0 = static_cast<int>(s0), t1 = min(r.len, t0 + seglen), each = seglen / NW;     // a multiple of KT
    const int lo = t0 + w * each, hi = min(t1, lo + each);
    float A = 1.f, H = 0.f;
    T x[KT], z[KT];
    G g[KT];
    const int n = hi > lo ? (hi - lo + KT - 1) / KT : 0;
    auto first = [&](int i) { return lo + (BACK ? i : n - 1 - i) * KT; };
    auto load = [&](int t) {
        fetch<T>(x, BACK ? a.dy : a.x, r, t, cc);
        fetch<G>(g, a.g, r, t, cc);
        if constexpr (BACK && Z) fetch<T>(z, a.z, r, t, cc);
    };
    if (n > 0) load(first(0));
    for (int i = 0; i < n; ++i) {
        const int t = first(i);
        float e[KT], u[KT];
#pragma unroll
        for (int k = 0; k < KT; ++k) {
            const bool in = t + k < hi;
            e[k] = in ? expf(static_cast<float>(g[k])) : 1.f;
            u[k] = in ? static_cast<float>(x[k]) : 0.f;
            if constexpr (BACK && Z) {
                float f, d;
                gate<DT != 0>(static_cast<float>(z[k]), a.act, f, d);
                u[k] = in ? u[k] * f : 0.f;
            }
        }
        if (i + 1 < n) load(first(i + 1));
        float P = 1.f, h = 0.f;
#pragma unroll
        for (int k = 0; k < KT; ++k) {
            const int j = BACK ? KT - 1 - k : k;
            h = BACK ? e[j] * (u[j] + h) : __builtin_fmaf(e[j], h, u[j]);
            P *= e[j];
        }
        // the new stretch is on the far side of those before it
        H = enter(A, H, h);
        A *= P;
    }
    ex[w][0][lane] = A;
    ex[w][1][lane] = H;
    __syncthreads();
    if (w == 0 && c < D) {
        A = 1.f;
        H = 0.f;
#pragma unroll
        for (int i = 0; i < NW; ++i) {
            const int j = BACK ? i : NW - 1 - i;
            H = enter(A, H, ex[j][1][lane]);
            A *= ex[j][0][lane];
        }
        float* p = part + (static_cast<int64_t>(run) * segs + seg) * 2 * a.D + c;
        p[0] = A;
        p[a.D] = H;
    }
}

template <int DT, int GT, bool Z>
__global__ __launch_bounds__(kGlrThreads) void glr_forward(const sdm_glr_args_t a, const int cblocks, const int segs, const float* __restrict__ part) {
    using T = elem_t<DT>;
    using G = elem_t<GT>;
    __shared__ float ex[2][NW][2][64];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int cb = blockIdx.x % cblocks, rs = blockIdx.x / cblocks, seg = rs % segs, run = rs / segs;
    const Run r = run_of(a, run);
    const int D = static_cast<int>(a.D), c = cb * 64 + lane, cc = min(c, D - 1);
    const int seglen = ((r.len + segs - 1) / segs + TILE - 1) / TILE * TILE;
    const int64_t s0 = static_cast<int64_t>(seg) * seglen;
    float h0 = a.h0 ? a.h0[run * a.D + cc] : 0.f;
    if (s0 >= r.len) {
        if (r.len == 0 && seg == 0 && w == 0 && c < D && a.h_final) a.h_final[run * a.D + c] = h0;
        return;
    }
    const int t0 = static_cast<int>(s0), t1 = min(r.len, t0 + seglen);
    T x[KT], z[KT];
    G g[KT];
    auto load = [&](int t) {
        fetch<T>(x, a.x, r, t, cc);
        fetch<G>(g, a.g, r, t, cc);
        if constexpr (Z) fetch<T>(z, a.z, r, t, cc);
    };
    load(t0 + w * KT);
    for (int s = 0; s < seg; ++s) {
        const float* p = part + (static_cast<int64_t>(run) * segs + s) * 2 * a.D + cc;
        h0 = enter(p[0], p[a.D], h0);
    }
    int buf = 0;
    for (int tile = t0; tile < t1; tile += TILE, buf ^= 1) {
        const int t = tile + w * KT;
        float e[KT], u[KT];
        T zz[KT];
        float A = 1.f, H = 0.f;
#pragma unroll
        for (int k = 0; k < KT; ++k) {
            const bool in = t + k < t1;
            e[k] = in ? expf(static_cast<float>(g[k])) : 1.f;
            u[k] = in ? static_cast<float>(x[k]) : 0.f;
            H = __builtin_fmaf(e[k], H, u[k]);
            A *= e[k];
            if constexpr (Z) zz[k] = z[k];
        }
        if (tile + TILE < t1) load(t + TILE);
        ex[buf][w][0][lane] = A;
        ex[buf][w][1][lane] = H;
        lds_barrier();      // the other buffer is written again only after the next one
        float h = h0, next = h0;
#pragma unroll
        for (int i = 0; i < NW; ++i) {
            h = i == w ? next : h;
            next = enter(ex[buf][i][0][lane], ex[buf][i][1][lane], next);
        }
        if (w == 0 && a.marks && c < D) a.marks[(r.mark + tile / TILE) * a.D + c] = h0;
        h0 = next;
#pragma unroll
        for (int k = 0; k < KT; ++k) {
            h = __builtin_fmaf(e[k], h, u[k]);
            float y = h;
            if constexpr (Z) {
                float f, d;
                gate<DT != 0>(static_cast<float>(zz[k]), a.act, f, d);
                y *= f;
            }
            if (t + k < t1 && c < D) put<T>(a.y, r.row, r.start + t + k, c, y);
        }
    }
    if (t1 == r.len && w == 0 && c < D && a.h_final) a.h_final[run * a.D + c] = h0;
}

template <int DT, int GT, bool Z>
__global__ __launch_bounds__(kGlrThreads) void glr_backward(const sdm_glr_args_t a, const int cblocks, const int segs, const float* __restrict__ part) {
    using T = elem_t<DT>;
    using G = elem_t<GT>;
    __shared__ float ex[2][NW][3][64];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int cb = blockIdx.x % cblocks, rs = blockIdx.x / cblocks, seg = rs % segs, run = rs / segs;
    const Run r = run_of(a, run);
    const int D = static_cast<int>(a.D), c = cb * 64 + lane, cc = min(c, D - 1);
    const int seglen = ((r.len + segs - 1) / segs + TILE - 1) / TILE * TILE;
    const int64_t s0 = static_cast<int64_t>(seg) * seglen;
    float e0 = a.dh_final ? a.dh_final[run * a.D + cc] : 0.f;       // what enters from the right
    if (s0 >= r.len) {
        if (r.len == 0 && seg == 0 && w == 0 && c < D && a.dh0) a.dh0[run * a.D + c] = e0;
        return;
    }
    const int t0 = static_cast<int>(s0), t1 = min(r.len, t0 + seglen);
    T x[KT], z[KT], dy[KT];
    G g[KT];
    float m;
    auto load = [&](int tile) {
        const int t = tile + w * KT;
        fetch<T>(x, a.x, r, t, cc);
        fetch<G>(g, a.g, r, t, cc);
        fetch<T>(dy, a.dy, r, t, cc);
        if constexpr (Z) fetch<T>(z, a.z, r, t, cc);
        m = a.marks[(r.mark + tile / TILE) * a.D + cc];
    };
    const int last = t0 + (t1 - t0 - 1) / TILE * TILE;
    load(last);
    const int used = (r.len - 1) / seglen;      // the last part that has tokens
    for (int s = used; s > seg; --s) {
        const float* p = part + (static_cast<int64_t>(run) * segs + s) * 2 * a.D + cc;
        e0 = enter(p[0], p[a.D], e0);
    }
    int buf = 0;
    for (int tile = last; tile >= t0; tile -= TILE, buf ^= 1) {
        const int t = tile + w * KT;
        float e[KT], u[KT], f[KT], v[KT], df[KT];     // a, x, dy act(z), and dy act'(z)
        float A = 1.f, H = 0.f, E = 0.f;
#pragma unroll
        for (int k = 0; k < KT; ++k) {
            const bool in = t + k < t1;
            e[k] = in ? expf(static_cast<float>(g[k])) : 1.f;
            u[k] = in ? static_cast<float>(x[k]) : 0.f;
            v[k] = in ? static_cast<float>(dy[k]) : 0.f;
            f[k] = v[k];
            if constexpr (Z) {
                float q, d;
                gate<DT != 0>(static_cast<float>(z[k]), a.act, q, d);
                f[k] = in ? v[k] * q : 0.f;
                df[k] = v[k] * d;
            }
            H = __builtin_fmaf(e[k], H, u[k]);
            A *= e[k];
        }
#pragma unroll
        for (int k = KT - 1; k >= 0; --k) E = e[k] * (f[k] + E);
        float h = m;
        if (tile > t0) load(tile - TILE);
        ex[buf][w][0][lane] = A;
        ex[buf][w][1][lane] = H;
        ex[buf][w][2][lane] = E;
        lds_barrier();      // the other buffer is written again only after the next one
#pragma unroll
        for (int i = 0; i < NW - 1; ++i)
            if (i < w) h = enter(ex[buf][i][0][lane], ex[buf][i][1][lane], h);
        float q = e0, next = e0;
#pragma unroll
        for (int i = NW - 1; i >= 0; --i) {
            q = i == w ? next : q;
            next = enter(ex[buf][i][0][lane], ex[buf][i][2][lane], next);
        }
        e0 = next;
        float met[KT];
#pragma unroll
        for (int k = 0; k < KT; ++k) {
            met[k] = h;
            h = __builtin_fmaf(e[k], h, u[k]);
        }
#pragma unroll
        for (int k = KT - 1; k >= 0; --k) {
            const float d = f[k] + q;
            q = e[k] * d;
            if (t + k < t1 && c < D) {
                const int64_t at = r.start + t + k;
                put<T>(a.dx, r.row, at, c, d);
                put<G>(a.dg, r.row, at, c, q * met[k]);
                if constexpr (Z) put<T>(a.dz, r.row, at, c, df[k] * __builtin_fmaf(e[k], met[k], u[k]));
            }
        }
    }
    if (seg == 0 && w == 0 && c < D && a.dh0) a.dh0[run * a.D + c] = e0;
}

// A thread has one channel of one stream.
template <int DT, int GT, bool Z>
__global__ __launch_bounds__(kGlrStepThreads) void glr_step(const sdm_glr_step_args_t a, const int cblocks) {
    using T = elem_t<DT>;
    using G = elem_t<GT>;
    const int64_t b = blockIdx.x / cblocks;
    const int c = blockIdx.x % cblocks * kGlrStepThreads + threadIdx.x;
    if (c >= a.D) return;
    const int64_t slot = a.slots ? a.slots[b] : b;
    if (slot < 0 || slot >= a.pool) {
        for (int64_t t = 0; t < a.T; ++t) put<T>(a.y, b, t, c, 0.f);
        return;
    }
    float h = a.state[slot * a.D + c];
    for (int64_t t = 0; t < a.T; ++t) {
        h = __builtin_fmaf(expf(static_cast<float>(at<G>(a.g, b, t, c))), h, static_cast<float>(at<T>(a.x, b, t, c)));
        float y = h;
        if constexpr (Z) {
            float f, d;
            gate<DT != 0>(static_cast<float>(at<T>(a.z, b, t, c)), a.act, f, d);
            y *= f;
        }
        put<T>(a.y, b, t, c, y);
    }
    a.state[slot * a.D + c] = h;
}

template <int DT, int GT, bool Z>
hipError_t forward_of(const sdm_glr_args_t& a, const GlrPlan& p, float* part, hipStream_t s) {
    const unsigned grid = static_cast<unsigned>(a.nseq * p.segs * p.cblocks);
    if (p.segs > 1) glr_parts<DT, GT, Z, false><<<grid, kGlrThreads, 0, s>>>(a, p.cblocks, p.segs, part);
    glr_forward<DT, GT, Z><<<grid, kGlrThreads, 0, s>>>(a, p.cblocks, p.segs, part);
    return hipGetLastError();
}
template <int DT, int GT, bool Z>
hipError_t backward_of(const sdm_glr_args_t& a, const GlrPlan& p, float* part, hipStream_t s) {
    const unsigned grid = static_cast<unsigned>(a.nseq * p.segs * p.cblocks);
    if (p.segs > 1) glr_parts<DT, GT, Z, true><<<grid, kGlrThreads, 0, s>>>(a, p.cblocks, p.segs, part);
    glr_backward<DT, GT, Z><<<grid, kGlrThreads, 0, s>>>(a, p.cblocks, p.segs, part);
    return hipGetLastError();
}
template <int DT, int GT, bool Z>
hipError_t step_of(const sdm_glr_step_args_t& a, hipStream_t s) {
    const int cblocks = static_cast<int>((a.D + kGlrStepThreads - 1) / kGlrStepThreads);
    glr_step<DT, GT, Z><<<static_cast<unsigned>(a.B * cblocks), kGlrStepThreads, 0, s>>>(a, cblocks);
    return hipGetLastError();
}

// gtype is dtype or float32 (the host checks)
#define SDM_GLR_TYPES(F, ...)                                                                                   \
    const bool z = a.act != SDM_ACT_NONE, wide = a.gtype == SDM_F32;                                            \
    if (a.dtype == SDM_F32) return z ? F<0, 0, true>(__VA_ARGS__) : F<0, 0, false>(__VA_ARGS__);                \
    if (a.dtype == SDM_BF16 && wide) return z ? F<1, 0, true>(__VA_ARGS__) : F<1, 0, false>(__VA_ARGS__);       \
    if (a.dtype == SDM_BF16) return z ? F<1, 1, true>(__VA_ARGS__) : F<1, 1, false>(__VA_ARGS__);               \
    if (wide) return z ? F<2, 0, true>(__VA_ARGS__) : F<2, 0, false>(__VA_ARGS__);                              \
    return z ? F<2, 2, true>(__VA_ARGS__) : F<2, 2, false>(__VA_ARGS__);

}  // namespace

hipError_t launch_glr_forward(const sdm_glr_args_t& a, const GlrPlan& p, float* part, hipStream_t s) {
    SDM_GLR_TYPES(forward_of, a, p, part, s)
}
hipError_t launch_glr_backward(const sdm_glr_args_t& a, const GlrPlan& p, float* part, hipStream_t s) {
    SDM_GLR_TYPES(backward_of, a, p, part, s)
}
hipError_t launch_glr_step(const sdm_glr_step_args_t& a, hipStream_t s) { SDM_GLR_TYPES(step_of, a, s) }

}  // namespace sdm_delta
