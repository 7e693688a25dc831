// The scans of the gated delta rule over a sequence's chunks: forward (o and the last state, or for the gradient every
// chunk's entering state and u) and backward (the gradient of every chunk's last state, dr and dv).
//
// Forward, per chunk with entering state S, G, T and P as in gdr_chunk.hip:
//     R = beta (V - exp(G) K S);  U = T R;  O = scale exp(G) Q S + P U;  S = exp(G_C) S + K^T (exp(G_C - G) U)
// Backward, with dS the gradient of the chunk's last state:
//     dU = P^T dO + exp(G_C - G) (K dS);  dR = T^T dU;  dV = beta dR
//     dS = exp(G_C) dS + Q^T (scale exp(G) dO) - K^T (beta exp(G) dR)
//
// The columns of S (of dv) never meet, so a workgroup owns 16 NT of them and walks all chunks of its sequence and
// head; the state stays in its accumulators in float32. The chunks of one head depend on each other: what bounds a
// scan of few heads is the time of one step, the chain S -> R -> U -> S. Four wavefronts, 16 tokens each, work on that
// chain; four more, the outputs' wavefronts, share their SIMDs and fill their waits with what the chain does not wait
// for (Q S and P U, a step late; P^T dO, a step early), and all eight share the update of S. S, R and U (16 columns
// each) pass through LDS as split parts, three barriers a step; everything else (K, Q, T, P and K^T fragments) comes
// straight from memory in operand layout, one chunk ahead of its use.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "gdr_device.h"

namespace sdm_delta {
namespace {

// Four consecutive tokens of one column as they lie in memory (past the chunk's tokens the last one's; a column past the
// head's is the caller's to leave out), and as floats, zero past the chunk's tokens. They are apart so that nothing
// waits for the load before the values are used.
template <int DT>
struct Tokens4 {
    elem_t<DT> x[4];
};
template <int DT>
__device__ __forceinline__ void load4(Tokens4<DT>& v, const elem_t<DT>* __restrict__ p, int64_t stride, int t, int n) {
#pragma unroll
    for (int e = 0; e < 4; ++e) v.x[e] = p[min(t + e, n - 1) * stride];
}
template <int DT>
__device__ __forceinline__ f32x4 floats4(const Tokens4<DT>& v, int t, int n) {
    f32x4 f;
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = t + e < n ? static_cast<float>(v.x[e]) : 0.f;
    return f;
}
// and back: tokens below n only
template <class T>
__device__ __forceinline__ void put4(T* __restrict__ p, int64_t stride, int t, int n, const f32x4& v) {
    if (t + 4 <= n) {
#pragma unroll
        for (int e = 0; e < 4; ++e) p[(t + e) * stride] = static_cast<T>(v[e]);
    } else {
#pragma unroll
        for (int e = 0; e < 3; ++e)
            if (t + e < n) p[(t + e) * stride] = static_cast<T>(v[e]);
    }
}

// What a workgroup of a scan works on.
struct Scan {
    int dk, dv, Hv, Hk, c0, hv, hk, chunks;
    int lane, row, grp, wave, part;     // part: which 16 tokens of a chunk
    bool chain;                         // a wavefront of the chain, not of the outputs
    int64_t head;
    Seq s;
};
__device__ __forceinline__ bool scan_of(Scan& w, const sdm_gdr_args_t& a, int total, int cols) {
    int id;
    if (!on_one_xcd(total, id)) return false;
    w.dk = static_cast<int>(a.dk), w.dv = static_cast<int>(a.dv), w.Hv = static_cast<int>(a.Hv);
    w.Hk = static_cast<int>(a.Hk);
    const int slices = (w.dv + cols - 1) / cols, seq = id / slices / w.Hv;
    w.c0 = id % slices * cols;
    w.hv = id / slices % w.Hv;
    w.hk = w.hv / (w.Hv / w.Hk);
    w.lane = threadIdx.x & 63;
    w.row = w.lane & 15;
    w.grp = w.lane >> 4;
    w.wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    w.chain = w.wave < 4;
    w.part = w.wave & 3;
    w.s = sequence(a, seq);
    w.chunks = (w.s.len + kChunk - 1) / kChunk;
    w.head = static_cast<int64_t>(seq) * w.Hv + w.hv;
    return true;
}

// The state tiles: tile m of a wavefront is rows (first + m) * 16 + 4 grp .. + 3, column c0 + 16 t + row.
template <int DKP>
struct Tiles {
    static constexpr int kOwners = DKP >= 128 ? 8 : 4, MT = DKP / 16 / kOwners;
    __device__ __forceinline__ static bool owner(const Scan& w) { return w.wave < kOwners; }
    static constexpr bool owns(bool chain) { return chain || kOwners == 8; }
    __device__ __forceinline__ static int first(const Scan& w) { return w.wave * MT; }
};
template <int DKP, int NT>
__device__ __forceinline__ void load_state(f32x4 (&S)[Tiles<DKP>::MT][NT], const Scan& w, const float* st) {
#pragma unroll
    for (int m = 0; m < Tiles<DKP>::MT; ++m)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int d = (Tiles<DKP>::first(w) + m) * 16 + w.grp * 4 + e, c = w.c0 + t * 16 + w.row;
                S[m][t][e] = st && d < w.dk && c < w.dv ? st[(w.head * w.dk + d) * w.dv + c] : 0.f;
            }
}
template <int DKP, int NT>
__device__ __forceinline__ void store_state(const f32x4 (&S)[Tiles<DKP>::MT][NT], const Scan& w, float* st) {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int c = w.c0 + t * 16 + w.row;
        if (c >= w.dv) continue;
#pragma unroll
        for (int m = 0; m < Tiles<DKP>::MT; ++m)
            put4(st + c, w.dv, (Tiles<DKP>::first(w) + m) * 16 + w.grp * 4, w.dk, S[m][t]);
    }
}

// A wavefront's fragments of one chunk, and its tokens' factors.
template <int NP, int DKP>
struct Operands {
    const GdrLaunch& g;
    const Scan& w;
    __device__ __forceinline__ int64_t sv(int chunk) const { return static_cast<int64_t>(w.s.slot + chunk) * w.Hv + w.hv; }
    __device__ __forceinline__ int64_t sk(int chunk) const { return static_cast<int64_t>(w.s.slot + chunk) * w.Hk + w.hk; }
    // K or Q: this wavefront's tokens
    __device__ __forceinline__ void rows(Frag<NP> (&f)[DKP / 32], uint16_t* from, int chunk) const {
#pragma unroll
        for (int kb = 0; kb < DKP / 32; ++kb)
            load_frag<NP>(f[kb], frag_at<NP>(from + sk(chunk) * (NP * 64 * DKP), w.part, kb, DKP / 32));
    }
    // K^T or Q^T: this wavefront's rows of the state
    template <bool CHAIN>
    __device__ __forceinline__ void cols(Frag<NP> (&f)[Tiles<DKP>::MT][2], uint16_t* from, int chunk) const {
        if constexpr (!Tiles<DKP>::owns(CHAIN)) return;
#pragma unroll
        for (int m = 0; m < Tiles<DKP>::MT; ++m)
#pragma unroll
            for (int kb = 0; kb < 2; ++kb)
                load_frag<NP>(f[m][kb], frag_at<NP>(from + sk(chunk) * (NP * 64 * DKP), Tiles<DKP>::first(w) + m, kb, 2));
    }
    // a 64 x 64 matrix: this wavefront's rows
    template <int N>
    __device__ __forceinline__ void square(Frag<N> (&f)[2], uint16_t* from, int chunk) const {
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) load_frag<N>(f[kb], frag_at<N>(from + sv(chunk) * (N * 4096), w.part, kb, 2));
    }
    __device__ __forceinline__ f32x4 token(int field, int chunk) const {
        return *reinterpret_cast<const f32x4*>(g.w.tok + (sv(chunk) * kTokFields + field) * 64 + w.part * 16 + w.grp * 4);
    }
    __device__ __forceinline__ float whole(int chunk) const { return g.w.tok[(sv(chunk) * kTokFields + kTokEg) * 64 + 63]; }
};

// The two kinds of wavefronts run loops of their own: where two paths of one loop meet, registers that loads are still
// on their way to would be moved, and the moves wait.
template <int DT, int DKP, int NT, bool STORE>
__global__ __launch_bounds__(512, 2) void gdr_scan(const GdrLaunch g, const int total) {
    constexpr int NP = kParts<DT>, PP = kOutParts<DT>, NKB = DKP / 32, MT = Tiles<DKP>::MT, COLS = 16 * NT;
    using T = elem_t<DT>;
    __shared__ Tile<3, COLS, DKP + 8> Sx;           // S, [column][dk]
    __shared__ Tile<3, COLS, 72> Rx, Dx;            // R and exp(G_C - G) U, [column][token]
    __shared__ Tile<PP, COLS, 72> Ux[STORE ? 1 : 2];    // U, of even and odd chunks
    const sdm_gdr_args_t& a = g.a;
    Scan w;
    if (!scan_of(w, a, total, COLS)) return;
    const int tok = w.part * 16, t4 = tok + w.grp * 4, hv = w.hv, dv = w.dv, chunks = w.chunks;
    const Operands<NP, DKP> from{g, w};
    f32x4 S[MT][NT];
    load_state<DKP, NT>(S, w, Tiles<DKP>::owner(w) ? a.s0 : nullptr);
    if (Tiles<DKP>::owner(w)) {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int t = 0; t < NT; ++t) Sx.put(t * 16, (Tiles<DKP>::first(w) + m) * 16, S[m][t]);
    }
    auto keep = [&](int chunk, auto chain) {
        if constexpr (STORE && Tiles<DKP>::owns(decltype(chain)::value))
            store_state<DKP, NT>(S, w, g.w.st + from.sv(chunk) * w.dk * dv);
    };
    auto update = [&](const Frag<NP> (&kt)[MT][2], float whole, auto chain) {
        if constexpr (!Tiles<DKP>::owns(decltype(chain)::value)) return;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            Frag<3> b[2];
            Dx.frag(b[0], t * 16, 0);
            Dx.frag(b[1], t * 16, 32);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                S[m][t] *= whole;
                mma<3>(S[m][t], kt[m][0], b[0]);
                mma<3>(S[m][t], kt[m][1], b[1]);
                Sx.put(t * 16, (Tiles<DKP>::first(w) + m) * 16, S[m][t]);
            }
        }
    };
    // Each operand's next chunk is fetched as soon as this one's is used (the last step fetches itself again).
    if (w.chain && chunks) {
        const T* vr = rows_at<const T>(a.v, w.s, hv);
        Frag<NP> kf[NKB], kt[MT][2];
        Frag<3> inv[2];
        Tokens4<DT> v[NT];
        f32x4 eg_n, last_n, beta_n;
        float whole_n;
        auto fetch_tok = [&](int chunk) {
            const int t0 = chunk * kChunk, n = min(kChunk, w.s.len - t0);
            eg_n = from.token(kTokEg, chunk);
            last_n = from.token(kTokLast, chunk);
            beta_n = from.token(kTokBeta, chunk);
            whole_n = from.whole(chunk);
#pragma unroll
            for (int c = 0; c < NT; ++c)
                load4<DT>(v[c], vr + t0 * a.v.token + min(w.c0 + c * 16 + w.row, dv - 1), a.v.token, t4, n);
        };
        from.rows(kf, g.w.kf, 0);
        fetch_tok(0);
        from.square(inv, g.w.inv, 0);
        from.template cols<true>(kt, g.w.kt, 0);
        loads_landed();
        for (int chunk = 0; chunk < chunks; ++chunk) {
            const int next = min(chunk + 1, chunks - 1), n = min(kChunk, w.s.len - chunk * kChunk);
            keep(chunk, std::bool_constant<true>{});
            const f32x4 eg = eg_n, last = last_n, beta = beta_n;
            const float whole = whole_n;
            lds_barrier();      // S is in LDS
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                f32x4 x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int kb = 0; kb < NKB; ++kb) {
                    Frag<3> b;
                    Sx.frag(b, t * 16, kb * 32);
                    mma<3>(x, kf[kb], b);
                }
                Rx.put(t * 16, tok, beta * (floats4<DT>(v[t], t4, n) - eg * x));
            }
            from.rows(kf, g.w.kf, next);
            fetch_tok(next);
            lds_barrier();
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                f32x4 u = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int kb = 0; kb < 2; ++kb) {
                    Frag<3> b;
                    Rx.frag(b, t * 16, kb * 32);
                    mma<3>(u, inv[kb], b);
                }
                Dx.put(t * 16, tok, last * u);
                if constexpr (!STORE) Ux[chunk & 1].put(t * 16, tok, u);
                if constexpr (STORE) {
                    if (w.c0 + t * 16 + w.row < dv)
                        put4(g.w.u + from.sv(chunk) * 64 * dv + w.c0 + t * 16 + w.row, dv, t4, kChunk, u);
                }
            }
            from.square(inv, g.w.inv, next);
            lds_barrier();
            update(kt, whole, std::bool_constant<true>{});
            from.template cols<true>(kt, g.w.kt, next);
        }
    }
    if (!w.chain && chunks) {
        T* orow = STORE ? nullptr : rows_at<T>(a.o, w.s, hv);
        Frag<NP> qf[NKB], kt[MT][2];
        Frag<PP> pm[2];
        f32x4 o[NT], eg_o = {0.f, 0.f, 0.f, 0.f}, eg_n;
        float whole_n;
        // the outputs of a chunk: P U on top of what Q S left
        auto finish = [&](int chunk) {
            const int t0 = chunk * kChunk, n = min(kChunk, w.s.len - t0);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                o[t] = o[t] * (eg_o * a.scale);
#pragma unroll
                for (int kb = 0; kb < 2; ++kb) {
                    Frag<PP> b;
                    Ux[STORE ? 0 : chunk & 1].frag(b, t * 16, kb * 32);
                    mma<PP>(o[t], pm[kb], b);
                }
                if (w.c0 + t * 16 + w.row < dv)
                    put4(orow + t0 * a.o.token + w.c0 + t * 16 + w.row, a.o.token, t4, n, o[t]);
            }
        };
        if constexpr (!STORE) {
            from.rows(qf, g.w.qf, 0);
            from.square(pm, g.w.pm, 0);
#pragma unroll
            for (int t = 0; t < NT; ++t) o[t] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
        eg_n = from.token(kTokEg, 0);
        whole_n = from.whole(0);
        from.template cols<false>(kt, g.w.kt, 0);
        loads_landed();
        for (int chunk = 0; chunk < chunks; ++chunk) {
            const int next = min(chunk + 1, chunks - 1);
            keep(chunk, std::bool_constant<false>{});
            const f32x4 eg = eg_n;
            const float whole = whole_n;
            lds_barrier();
            f32x4 x[NT];
            if constexpr (!STORE) {
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    x[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int kb = 0; kb < NKB; ++kb) {
                        Frag<PP> b;
#pragma unroll
                        for (int p = 0; p < PP; ++p)
                            b.p[p] = *reinterpret_cast<const bf16x8*>(&Sx.v[p][t * 16 + w.row][kb * 32 + 8 * w.grp]);
                        mma<PP>(x[t], qf[kb], b);
                    }
                }
                from.rows(qf, g.w.qf, next);
            }
            eg_n = from.token(kTokEg, next);
            whole_n = from.whole(next);
            lds_barrier();
            if constexpr (!STORE) {
                if (chunk) finish(chunk - 1);
                from.square(pm, g.w.pm, chunk);
#pragma unroll
                for (int t = 0; t < NT; ++t) o[t] = x[t];
                eg_o = eg;
            }
            lds_barrier();
            update(kt, whole, std::bool_constant<false>{});
            from.template cols<false>(kt, g.w.kt, next);
        }
        if constexpr (!STORE) finish(chunks - 1);
    }
    if constexpr (!STORE)
        if (a.s_final && Tiles<DKP>::owner(w)) store_state<DKP, NT>(S, w, a.s_final + w.head * w.dk * dv);
}

template <int DT, int DKP, int NT>
__global__ __launch_bounds__(512, 2) void gdr_scan_back(const GdrLaunch g, const int total) {
    constexpr int NP = kParts<DT>, NKB = DKP / 32, MT = Tiles<DKP>::MT, COLS = 16 * NT;
    using T = elem_t<DT>;
    __shared__ Tile<3, COLS, DKP + 8> Sx;           // dS, [column][dk]
    __shared__ Tile<3, COLS, 72> Ox, Qx, Ux, Rx;    // the next chunk's dO, scale exp(G) dO, dU and -beta exp(G) dR
    __shared__ f32x4 Wx[NT][4][64];                 // P^T dO, as the chain's wavefronts hold dU
    const sdm_gdr_args_t& a = g.a;
    Scan w;
    if (!scan_of(w, a, total, COLS)) return;
    const int tok = w.part * 16, t4 = tok + w.grp * 4, hv = w.hv, dv = w.dv, top = w.chunks - 1;
    const Operands<NP, DKP> from{g, w};
    f32x4 S[MT][NT];
    load_state<DKP, NT>(S, w, Tiles<DKP>::owner(w) ? a.ds_final : nullptr);
    if (Tiles<DKP>::owner(w)) {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int t = 0; t < NT; ++t) Sx.put(t * 16, (Tiles<DKP>::first(w) + m) * 16, S[m][t]);
    }
    Frag<NP> kt[MT][2], qt[MT][2];
    auto keep = [&](int chunk, auto chain) {
        if constexpr (Tiles<DKP>::owns(decltype(chain)::value))
            store_state<DKP, NT>(S, w, g.w.dst + from.sv(chunk) * w.dk * dv);
    };
    auto update = [&](float whole, auto chain) {
        if constexpr (!Tiles<DKP>::owns(decltype(chain)::value)) return;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            Frag<3> bq[2], br[2];
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) {
                Qx.frag(bq[kb], t * 16, kb * 32);
                Rx.frag(br[kb], t * 16, kb * 32);
            }
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                S[m][t] *= whole;
#pragma unroll
                for (int kb = 0; kb < 2; ++kb) {
                    mma<3>(S[m][t], qt[m][kb], bq[kb]);
                    mma<3>(S[m][t], kt[m][kb], br[kb]);
                }
                Sx.put(t * 16, (Tiles<DKP>::first(w) + m) * 16, S[m][t]);
            }
        }
    };
    if (w.chain && top >= 0) {
        T* dvr = rows_at<T>(a.d_v, w.s, hv);
        Frag<NP> kf[NKB];
        Frag<3> inv[2];
        f32x4 eg_n, last_n, beta_n;
        float whole_n;
        auto fetch_tok = [&](int chunk) {
            eg_n = from.token(kTokEg, chunk);
            last_n = from.token(kTokLast, chunk);
            beta_n = from.token(kTokBeta, chunk);
            whole_n = from.whole(chunk);
        };
        from.rows(kf, g.w.kf, top);
        fetch_tok(top);
        from.square(inv, g.w.invt, top);
        from.template cols<true>(kt, g.w.kt, top);
        from.template cols<true>(qt, g.w.qt, top);
        loads_landed();
        lds_barrier();
        for (int chunk = top; chunk >= 0; --chunk) {
            const int t0 = chunk * kChunk, n = min(kChunk, w.s.len - t0), next = max(chunk - 1, 0);
            keep(chunk, std::bool_constant<true>{});
            const f32x4 eg = eg_n, last = last_n, beta = beta_n;
            const float whole = whole_n;
            lds_barrier();      // dS and P^T dO are in LDS
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                f32x4 u = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int kb = 0; kb < NKB; ++kb) {
                    Frag<3> b;
                    Sx.frag(b, t * 16, kb * 32);
                    mma<3>(u, kf[kb], b);
                }
                Ux.put(t * 16, tok, u * last + Wx[t][w.part][w.lane]);
            }
            from.rows(kf, g.w.kf, next);
            fetch_tok(next);
            lds_barrier();
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                f32x4 d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int kb = 0; kb < 2; ++kb) {
                    Frag<3> b;
                    Ux.frag(b, t * 16, kb * 32);
                    mma<3>(d, inv[kb], b);
                }
                Rx.put(t * 16, tok, -(beta * eg) * d);
                const int c = w.c0 + t * 16 + w.row;
                if (c < dv) {
                    put4(g.w.dr + from.sv(chunk) * 64 * dv + c, dv, t4, kChunk, d);
                    put4(dvr + t0 * a.d_v.token + c, a.d_v.token, t4, n, beta * d);
                }
            }
            from.square(inv, g.w.invt, next);
            lds_barrier();
            update(whole, std::bool_constant<true>{});
            from.template cols<true>(kt, g.w.kt, next);
            from.template cols<true>(qt, g.w.qt, next);
        }
    }
    if (!w.chain && top >= 0) {
        const T* dor = rows_at<const T>(a.d_o, w.s, hv);
        Frag<3> pm[2];                  // P^T of the next chunk
        Tokens4<DT> raw[NT];            // dO of the chunk after the next
        f32x4 o1[NT], eg_n;             // dO of this chunk
        float whole_n;
        auto fetch_do = [&](int chunk) {
            const int t0 = chunk * kChunk, n = min(kChunk, w.s.len - t0);
#pragma unroll
            for (int c = 0; c < NT; ++c)
                load4<DT>(raw[c], dor + t0 * a.d_o.token + min(w.c0 + c * 16 + w.row, dv - 1), a.d_o.token, t4, n);
        };
        auto p_do = [&]() {     // P^T dO of the chunk in Ox, for the chain's next step
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                f32x4 x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int kb = 0; kb < 2; ++kb) {
                    Frag<3> b;
                    Ox.frag(b, t * 16, kb * 32);
                    mma<3>(x, pm[kb], b);
                }
                Wx[t][w.part][w.lane] = x;
            }
        };
        eg_n = from.token(kTokEg, top);
        whole_n = from.whole(top);
        from.square(pm, g.w.pm, top);
        fetch_do(top);
        from.template cols<false>(kt, g.w.kt, top);
        from.template cols<false>(qt, g.w.qt, top);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            o1[t] = floats4<DT>(raw[t], t4, min(kChunk, w.s.len - top * kChunk));
            Ox.put(t * 16, tok, o1[t]);
        }
        lds_barrier();
        p_do();
        from.square(pm, g.w.pm, max(top - 1, 0));
        fetch_do(max(top - 1, 0));
        loads_landed();
        for (int chunk = top; chunk >= 0; --chunk) {
            const int next = max(chunk - 1, 0), n = min(kChunk, w.s.len - next * kChunk);
            keep(chunk, std::bool_constant<false>{});
            const f32x4 eg = eg_n;
            const float whole = whole_n;
            lds_barrier();
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                Qx.put(t * 16, tok, o1[t] * (eg * a.scale));
                o1[t] = floats4<DT>(raw[t], t4, n);
                Ox.put(t * 16, tok, o1[t]);
            }
            eg_n = from.token(kTokEg, next);
            whole_n = from.whole(next);
            fetch_do(max(chunk - 2, 0));
            lds_barrier();
            p_do();
            from.square(pm, g.w.pm, max(chunk - 2, 0));
            lds_barrier();
            update(whole, std::bool_constant<false>{});
            from.template cols<false>(kt, g.w.kt, next);
            from.template cols<false>(qt, g.w.qt, next);
        }
    }
    if (a.ds0 && Tiles<DKP>::owner(w)) store_state<DKP, NT>(S, w, a.ds0 + w.head * w.dk * dv);
}

template <int DT, int DKP>
hipError_t scan(const GdrLaunch& g, int mode, hipStream_t s) {
    const int total = static_cast<int>((g.a.dv + 15) / 16 * g.a.Hv * g.a.nseq), grid = 8 * ((total + 7) / 8);
    if (mode == 0)
        gdr_scan<DT, DKP, 1, false><<<grid, 512, 0, s>>>(g, total);
    else if (mode == 1)
        gdr_scan<DT, DKP, 1, true><<<grid, 512, 0, s>>>(g, total);
    else
        gdr_scan_back<DT, DKP, 1><<<grid, 512, 0, s>>>(g, total);
    return hipGetLastError();
}

template <int DT>
hipError_t run(const GdrLaunch& g, int mode, hipStream_t s) {
    if (g.dkp == 64) return scan<DT, 64>(g, mode, s);
    if (g.dkp == 128) return scan<DT, 128>(g, mode, s);
    return scan<DT, 256>(g, mode, s);
}

}  // namespace

// mode 0: forward; 1: forward for the gradient (states and u); 2: backward
hipError_t launch_gdr_scan(const GdrLaunch& g, int mode, hipStream_t s) {
    switch (g.a.dtype) {
        case SDM_F32: return run<0>(g, mode, s);
        case SDM_BF16: return run<1>(g, mode, s);
        default: return run<2>(g, mode, s);
    }
}

}  // namespace sdm_delta
