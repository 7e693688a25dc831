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
// scan of few heads is the time of one step. Four wavefronts split the 64 tokens and the dk rows of a step; what they
// exchange (S, R, U: 16 columns each) goes through LDS as split parts, three barriers a step; everything else (K, Q,
// T, P and K^T fragments) comes straight from memory in operand layout, one chunk ahead of its use.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdr_device.h"

namespace sdm_delta {
namespace {

// Four consecutive tokens of one column (the row of token t + e, or the chunk's last where there is none and the value
// is dropped; a column past the head's is the caller's to leave out).
template <int DT>
__device__ __forceinline__ f32x4 tokens4(const elem_t<DT>* __restrict__ p, int64_t stride, int t, int n) {
    f32x4 v;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float x = static_cast<float>(p[min(t + e, n - 1) * stride]);
        v[e] = t + e < n ? x : 0.f;
    }
    return v;
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

template <int DT, int DKP, int NT, bool STORE>
__global__ __launch_bounds__(256, 1) void gdr_scan(const GdrLaunch g, const int total) {
    constexpr int NP = kParts<DT>, PP = kOutParts<DT>, NKB = DKP / 32, MT = DKP / 64, COLS = 16 * NT;
    using T = elem_t<DT>;
    __shared__ Tile<3, COLS, DKP + 8> Sx;       // S, [column][dk]
    __shared__ Tile<3, COLS, 72> Rx, Ux, Dx;    // R, U and exp(G_C - G) U, [column][token]
    const sdm_gdr_args_t& a = g.a;
    int id;
    if (!on_one_xcd(total, id)) return;
    const int dk = static_cast<int>(a.dk), dv = static_cast<int>(a.dv), Hv = static_cast<int>(a.Hv);
    const int slices = (dv + COLS - 1) / COLS;
    const int c0 = id % slices * COLS, hv = id / slices % Hv, seq = id / slices / Hv;
    const int r = Hv / static_cast<int>(a.Hk), hk = hv / r;
    const int lane = threadIdx.x & 63, row = lane & 15, grp = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Seq s = sequence(a, seq);
    const int chunks = (s.len + kChunk - 1) / kChunk;
    const int64_t head = static_cast<int64_t>(seq) * Hv + hv;
    const T* vr = rows_at<const T>(a.v, s, hv);
    T* orow = STORE ? nullptr : rows_at<T>(a.o, s, hv);

    // state tile m of this wavefront: rows (wave * MT + m) * 16 + 4 grp .. + 3, column c0 + 16 t + row
    f32x4 S[MT][NT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int d = (wave * MT + m) * 16 + grp * 4, c = c0 + t * 16 + row;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                S[m][t][e] = a.s0 && d + e < dk && c < dv ? a.s0[(head * dk + d + e) * dv + c] : 0.f;
            Sx.put(t * 16, d - grp * 4, S[m][t]);
        }

    Frag<NP> kf[NKB], qf[STORE ? 1 : NKB], kt[MT][2];
    Frag<3> inv[2];
    Frag<PP> pm[2];
    f32x4 eg, last, beta, v[NT];
    float whole = 0.f;
    const int tok = wave * 16;      // this wavefront's tokens of a chunk
    auto fetch_kq = [&](int chunk) {
        const int64_t sk = (static_cast<int64_t>(s.slot + chunk) * a.Hk + hk) * (NP * 64 * DKP);
#pragma unroll
        for (int kb = 0; kb < NKB; ++kb) {
            load_frag<NP>(kf[kb], frag_at<NP>(g.w.kf + sk, wave, kb, NKB));
            if constexpr (!STORE) load_frag<NP>(qf[kb], frag_at<NP>(g.w.qf + sk, wave, kb, NKB));
        }
    };
    auto fetch_inv = [&](int chunk) {
        const int64_t sv = static_cast<int64_t>(s.slot + chunk) * Hv + hv;
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) load_frag<3>(inv[kb], frag_at<3>(g.w.inv + sv * (3 * 4096), wave, kb, 2));
    };
    auto fetch_rest = [&](int chunk) {
        const int64_t slot = s.slot + chunk, sv = slot * Hv + hv, sk = slot * a.Hk + hk;
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            if constexpr (!STORE) load_frag<PP>(pm[kb], frag_at<PP>(g.w.pm + sv * (PP * 4096), wave, kb, 2));
#pragma unroll
            for (int m = 0; m < MT; ++m)
                load_frag<NP>(kt[m][kb], frag_at<NP>(g.w.kt + sk * (NP * 64 * DKP), wave * MT + m, kb, 2));
        }
    };
    f32x4 eg_n, last_n, beta_n;
    float whole_n = 0.f;
    auto fetch_tok = [&](int chunk) {
        const int t0 = chunk * kChunk, n = min(kChunk, s.len - t0);
        const float* t = g.w.tok + (static_cast<int64_t>(s.slot + chunk) * Hv + hv) * (kTokFields * 64);
        eg_n = *reinterpret_cast<const f32x4*>(t + kTokEg * 64 + tok + grp * 4);
        last_n = *reinterpret_cast<const f32x4*>(t + kTokLast * 64 + tok + grp * 4);
        beta_n = *reinterpret_cast<const f32x4*>(t + kTokBeta * 64 + tok + grp * 4);
        whole_n = t[kTokEg * 64 + 63];
#pragma unroll
        for (int c = 0; c < NT; ++c)
            v[c] = tokens4<DT>(vr + t0 * a.v.token + min(c0 + c * 16 + row, dv - 1), a.v.token, tok + grp * 4, n);
    };
    if (chunks) {
        fetch_kq(0);
        fetch_tok(0);
        fetch_inv(0);
        fetch_rest(0);
        loads_landed();
    }
    for (int chunk = 0; chunk < chunks; ++chunk) {
        const int t0 = chunk * kChunk, n = min(kChunk, s.len - t0);
        const int64_t sv = static_cast<int64_t>(s.slot + chunk) * Hv + hv;
        if constexpr (STORE) {
            float* st = g.w.st + sv * dk * dv;
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int d = (wave * MT + m) * 16 + grp * 4 + e, c = c0 + t * 16 + row;
                        if (d < dk && c < dv) st[static_cast<int64_t>(d) * dv + c] = S[m][t][e];
                    }
        }
        // each operand's next chunk is fetched as soon as this one's is used (the last step fetches itself again)
        const int next = min(chunk + 1, chunks - 1);
        eg = eg_n;
        last = last_n;
        beta = beta_n;
        whole = whole_n;
        lds_barrier();      // S of all wavefronts is in LDS
        f32x4 x[NT], o[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) x[t] = o[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int kb = 0; kb < NKB; ++kb) {
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                Frag<3> b;
                Sx.frag(b, t * 16, kb * 32);
                mma<3>(x[t], kf[kb], b);
                if constexpr (!STORE) mma<PP>(o[t], qf[kb], b);
            }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) Rx.put(t * 16, tok, beta * (v[t] - eg * x[t]));
        fetch_kq(next);
        fetch_tok(next);
        lds_barrier();
        f32x4 u[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            u[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) {
                Frag<3> b;
                Rx.frag(b, t * 16, kb * 32);
                mma<3>(u[t], inv[kb], b);
            }
            if constexpr (!STORE) Ux.put(t * 16, tok, u[t]);
            Dx.put(t * 16, tok, last * u[t]);
        }
        fetch_inv(next);
        lds_barrier();
        if constexpr (STORE) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
                if (c0 + t * 16 + row < dv)
                    put4(g.w.u + sv * 64 * dv + c0 + t * 16 + row, dv, tok + grp * 4, kChunk, u[t]);
        }
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
                Sx.put(t * 16, (wave * MT + m) * 16, S[m][t]);
            }
        }
        if constexpr (!STORE) {
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                o[t] = o[t] * (eg * a.scale);
#pragma unroll
                for (int kb = 0; kb < 2; ++kb) {
                    Frag<PP> b;
#pragma unroll
                    for (int p = 0; p < PP; ++p)
                        b.p[p] = *reinterpret_cast<const bf16x8*>(&Ux.v[p][t * 16 + row][kb * 32 + 8 * grp]);
                    mma<PP>(o[t], pm[kb], b);
                }
                if (c0 + t * 16 + row < dv)
                    put4(orow + t0 * a.o.token + c0 + t * 16 + row, a.o.token, tok + grp * 4, n, o[t]);
            }
        }
        fetch_rest(next);
    }
    float* out = STORE ? nullptr : a.s_final;
    if (!out) return;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int d = (wave * MT + m) * 16 + grp * 4 + e, c = c0 + t * 16 + row;
                if (d < dk && c < dv) out[(head * dk + d) * dv + c] = S[m][t][e];
            }
}

template <int DT, int DKP, int NT>
__global__ __launch_bounds__(256, 1) void gdr_scan_back(const GdrLaunch g, const int total) {
    constexpr int NP = kParts<DT>, NKB = DKP / 32, MT = DKP / 64, COLS = 16 * NT;
    using T = elem_t<DT>;
    __shared__ Tile<3, COLS, DKP + 8> Sx;       // dS, [column][dk]
    __shared__ Tile<3, COLS, 72> Ox, Qx, Ux, Rx;    // dO, scale exp(G) dO, dU and -beta exp(G) dR, [column][token]
    const sdm_gdr_args_t& a = g.a;
    int id;
    if (!on_one_xcd(total, id)) return;
    const int dk = static_cast<int>(a.dk), dv = static_cast<int>(a.dv), Hv = static_cast<int>(a.Hv);
    const int slices = (dv + COLS - 1) / COLS;
    const int c0 = id % slices * COLS, hv = id / slices % Hv, seq = id / slices / Hv;
    const int r = Hv / static_cast<int>(a.Hk), hk = hv / r;
    const int lane = threadIdx.x & 63, row = lane & 15, grp = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Seq s = sequence(a, seq);
    const int chunks = (s.len + kChunk - 1) / kChunk;
    const int64_t head = static_cast<int64_t>(seq) * Hv + hv;
    const T* dor = rows_at<const T>(a.d_o, s, hv);
    T* dvr = rows_at<T>(a.d_v, s, hv);

    f32x4 S[MT][NT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int d = (wave * MT + m) * 16 + grp * 4, c = c0 + t * 16 + row;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                S[m][t][e] = a.ds_final && d + e < dk && c < dv ? a.ds_final[(head * dk + d + e) * dv + c] : 0.f;
            Sx.put(t * 16, d - grp * 4, S[m][t]);
        }
    const int tok = wave * 16;
    Frag<NP> kf[NKB];
    Frag<3> invt[2], pmt[2];
    Frag<NP> kt[MT][2], qt[MT][2];
    f32x4 eg, last, beta, dof[NT];
    float whole = 0.f;
    auto fetch_kp = [&](int chunk) {
        const int64_t slot = s.slot + chunk, sv = slot * Hv + hv, sk = (slot * a.Hk + hk) * (NP * 64 * DKP);
#pragma unroll
        for (int kb = 0; kb < NKB; ++kb) load_frag<NP>(kf[kb], frag_at<NP>(g.w.kf + sk, wave, kb, NKB));
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) load_frag<3>(pmt[kb], frag_at<3>(g.w.pm + sv * (3 * 4096), wave, kb, 2));
    };
    auto fetch_inv = [&](int chunk) {
        const int64_t sv = static_cast<int64_t>(s.slot + chunk) * Hv + hv;
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) load_frag<3>(invt[kb], frag_at<3>(g.w.invt + sv * (3 * 4096), wave, kb, 2));
    };
    auto fetch_t = [&](int chunk) {
        const int64_t sk = static_cast<int64_t>(s.slot + chunk) * a.Hk + hk;
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                load_frag<NP>(kt[m][kb], frag_at<NP>(g.w.kt + sk * (NP * 64 * DKP), wave * MT + m, kb, 2));
                load_frag<NP>(qt[m][kb], frag_at<NP>(g.w.qt + sk * (NP * 64 * DKP), wave * MT + m, kb, 2));
            }
    };
    f32x4 eg_n, last_n, beta_n;
    float whole_n = 0.f;
    auto fetch_tok = [&](int chunk) {
        const int t0 = chunk * kChunk, n = min(kChunk, s.len - t0);
        const float* t = g.w.tok + (static_cast<int64_t>(s.slot + chunk) * Hv + hv) * (kTokFields * 64);
        eg_n = *reinterpret_cast<const f32x4*>(t + kTokEg * 64 + tok + grp * 4);
        last_n = *reinterpret_cast<const f32x4*>(t + kTokLast * 64 + tok + grp * 4);
        beta_n = *reinterpret_cast<const f32x4*>(t + kTokBeta * 64 + tok + grp * 4);
        whole_n = t[kTokEg * 64 + 63];
#pragma unroll
        for (int c = 0; c < NT; ++c)
            dof[c] = tokens4<DT>(dor + t0 * a.d_o.token + min(c0 + c * 16 + row, dv - 1), a.d_o.token, tok + grp * 4, n);
    };
    if (chunks) {
        fetch_tok(chunks - 1);
        fetch_kp(chunks - 1);
        fetch_inv(chunks - 1);
        fetch_t(chunks - 1);
        loads_landed();
    }
    for (int chunk = chunks - 1; chunk >= 0; --chunk) {
        const int t0 = chunk * kChunk, n = min(kChunk, s.len - t0);
        const int64_t sv = static_cast<int64_t>(s.slot + chunk) * Hv + hv;
        const int next = max(chunk - 1, 0);
        float* st = g.w.dst + sv * dk * dv;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int d = (wave * MT + m) * 16 + grp * 4 + e, c = c0 + t * 16 + row;
                    if (d < dk && c < dv) st[static_cast<int64_t>(d) * dv + c] = S[m][t][e];
                }
#pragma unroll
        for (int t = 0; t < NT; ++t) Ox.put(t * 16, tok, dof[t]);
        eg = eg_n;
        last = last_n;
        beta = beta_n;
        whole = whole_n;
        lds_barrier();
#pragma unroll
        for (int t = 0; t < NT; ++t) Qx.put(t * 16, tok, dof[t] * (eg * a.scale));
        fetch_tok(next);
        f32x4 u[NT], d[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            u[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int kb = 0; kb < NKB; ++kb) {
                Frag<3> b;
                Sx.frag(b, t * 16, kb * 32);
                mma<3>(u[t], kf[kb], b);
            }
            u[t] *= last;
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) {
                Frag<3> b;
                Ox.frag(b, t * 16, kb * 32);
                mma<3>(u[t], pmt[kb], b);
            }
            Ux.put(t * 16, tok, u[t]);
        }
        fetch_kp(next);
        lds_barrier();
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            d[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) {
                Frag<3> b;
                Ux.frag(b, t * 16, kb * 32);
                mma<3>(d[t], invt[kb], b);
            }
            Rx.put(t * 16, tok, -(beta * eg) * d[t]);
        }
        fetch_inv(next);
        lds_barrier();
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
                Sx.put(t * 16, (wave * MT + m) * 16, S[m][t]);
            }
            const int c = c0 + t * 16 + row;
            if (c < dv) {
                put4(g.w.dr + sv * 64 * dv + c, dv, tok + grp * 4, kChunk, d[t]);
                put4(dvr + t0 * a.d_v.token + c, a.d_v.token, tok + grp * 4, n, beta * d[t]);
            }
        }
        fetch_t(next);
    }
    if (!a.ds0) return;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int d = (wave * MT + m) * 16 + grp * 4 + e, c = c0 + t * 16 + row;
                if (d < dk && c < dv) a.ds0[(head * dk + d) * dv + c] = S[m][t][e];
            }
}

int workgroups(const GdrLaunch& g) { return static_cast<int>((g.a.dv + g.cols - 1) / g.cols * g.a.Hv * g.a.nseq); }

#define SDM_GDR_LAUNCH(KERNEL, ...)                                                                       \
    do {                                                                                                  \
        const int total = workgroups(g);                                                                  \
        KERNEL<__VA_ARGS__><<<8 * ((total + 7) / 8), 256, 0, s>>>(g, total);                              \
        return hipGetLastError();                                                                         \
    } while (0)

template <int DT, int DKP>
hipError_t forward_of(const GdrLaunch& g, bool store, hipStream_t s) {
    if (store) {
        if (g.cols == 32) SDM_GDR_LAUNCH(gdr_scan, DT, DKP, 2, true);
        SDM_GDR_LAUNCH(gdr_scan, DT, DKP, 1, true);
    }
    if (g.cols == 32) SDM_GDR_LAUNCH(gdr_scan, DT, DKP, 2, false);
    SDM_GDR_LAUNCH(gdr_scan, DT, DKP, 1, false);
}
template <int DT, int DKP>
hipError_t back_of(const GdrLaunch& g, hipStream_t s) {
    if (g.cols == 32) SDM_GDR_LAUNCH(gdr_scan_back, DT, DKP, 2);
    SDM_GDR_LAUNCH(gdr_scan_back, DT, DKP, 1);
}

template <int DT>
hipError_t run(const GdrLaunch& g, int mode, hipStream_t s) {
    if (g.dkp == 64) return mode == 2 ? back_of<DT, 64>(g, s) : forward_of<DT, 64>(g, mode == 1, s);
    if (g.dkp == 128) return mode == 2 ? back_of<DT, 128>(g, s) : forward_of<DT, 128>(g, mode == 1, s);
    return mode == 2 ? back_of<DT, 256>(g, s) : forward_of<DT, 256>(g, mode == 1, s);
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
