// The gradient of the gated delta rule within a chunk, all chunks at once, from what the two scans left: each chunk's
// entering state S, the gradient dE of its last state, U and dR.
//
//     dP = (dO U^T) decay scale (j <= i);   dA = -(dR U^T) decay (j < i)
//     dq = scale exp(G) dO S^T + dP K
//     dkr = dA K - exp(G) dR S^T            (beta dkr is the part of dk_i from i's own row of the triangular system)
//     dkc = exp(G_C - G) U dE^T + dP^T Q + (beta dA)^T K
//     dk = beta dkr + dkc;   dbeta = dR . V + k . dkr
//     dG = q . dq + k . (beta dkr - dkc), and at the chunk's last token also k . exp(G_C - G) U dE^T over all tokens
//     and exp(G_C) <S, dE>: every factor exp(G_i ..) of a product is differentiated by the product itself
//     dg = the sums of dG from each token to the chunk's end
//
// One workgroup per chunk and value head. Each wavefront owns dk columns of dq and dk for all 64 tokens, so S and dE
// are read and split once; dO, U and dR are staged in LDS by 64 columns of dv at a time. About 18 x 64 dk dv flops on
// up to six steps each: bounded by the matrix cores and the LDS reads that feed them.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdr_device.h"

namespace sdm_delta {
namespace {

template <int DT, int DKP>
__global__ __launch_bounds__(256, DKP <= 128 ? 2 : 1) void gdr_grad(const GdrLaunch g) {
    constexpr int NP = kParts<DT>, MT = DKP / 64;
    using T = elem_t<DT>;
    struct Staged {
        Tile<NP, 64, 64> o;
        Tile<3, 64, 64> u, r;
    };
    struct Pairs {
        Tile<3, 64, 64> m, t;     // a 64 x 64 matrix by rows and by columns
    };
    union Shared {
        Staged s;
        Pairs p;
        __device__ Shared() {}
    };
    __shared__ Shared L;
    __shared__ alignas(16) float Gh[64], Gl[64], Eg[64], La[64], Be[64], Rv[64], red[4][2][64], tot[4][2];
    const sdm_gdr_args_t& a = g.a;
    int seq, chunk;
    Seq s;
    const int slot = blockIdx.x, hv = blockIdx.y, rr = static_cast<int>(a.Hv / a.Hk), hk = hv / rr;
    if (!owner(a, slot, seq, chunk, s)) return;
    const int t0 = chunk * kChunk, n = min(kChunk, s.len - t0);
    const int dk = static_cast<int>(a.dk), dv = static_cast<int>(a.dv);
    const int lane = threadIdx.x & 63, row = lane & 15, grp = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t sv = static_cast<int64_t>(slot) * a.Hv + hv, sk = static_cast<int64_t>(slot) * a.Hk + hk;
    const bool vst = (dv & 7) == 0;

    if (threadIdx.x < 64) {
        const float* t = g.w.tok + sv * (kTokFields * 64) + threadIdx.x;
        Gh[threadIdx.x] = t[kTokG * 64];
        Gl[threadIdx.x] = t[kTokGlo * 64];
        Eg[threadIdx.x] = t[kTokEg * 64];
        La[threadIdx.x] = t[kTokLast * 64];
        Be[threadIdx.x] = t[kTokBeta * 64];
    }
    const T* dor = rows_at<const T>(a.d_o, s, hv) + t0 * a.d_o.token;
    const T* vr = rows_at<const T>(a.v, s, hv) + t0 * a.v.token;
    const float* ur = g.w.u + sv * 64 * dv;
    const float* rp = g.w.dr + sv * 64 * dv;
    const float* st = g.w.st + sv * dk * dv;
    const float* de = g.w.dst + sv * dk * dv;

    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
    f32x4 dp[4], da[4], aq[MT][4], ar[MT][4], as[MT][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        dp[j] = da[j] = zero;
#pragma unroll
        for (int m = 0; m < MT; ++m) aq[m][j] = ar[m][j] = as[m][j] = zero;
    }
    float rv[2] = {0.f, 0.f}, sde = 0.f;
    for (int c0 = 0; c0 < dv; c0 += 64) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int i = h * 32 + (threadIdx.x >> 3), cc = (threadIdx.x & 7) * 8, c = c0 + cc;
            float x[8], y[8];
            Frag<3> f;
            Raw<DT> raw;
            Frag<NP> fo;
            const int at = min(i, n - 1);
            if (g.vec_v)
                load_raw<DT, true>(raw, dor + at * a.d_o.token, c, dv, i < n);
            else
                load_raw<DT, false>(raw, dor + at * a.d_o.token, c, dv, i < n);
            raw_frag<DT>(fo, raw);
            load8(x, ur + i * dv, c, dv, vst);
            split8(f, x);
#pragma unroll
            for (int p = 0; p < NP; ++p) *reinterpret_cast<bf16x8*>(L.s.o.at(p, i, cc)) = fo.p[p];
#pragma unroll
            for (int p = 0; p < 3; ++p) *reinterpret_cast<bf16x8*>(L.s.u.at(p, i, cc)) = f.p[p];
            load8(x, rp + i * dv, c, dv, vst);
            split8(f, x);
#pragma unroll
            for (int p = 0; p < 3; ++p) *reinterpret_cast<bf16x8*>(L.s.r.at(p, i, cc)) = f.p[p];
            if (g.vec_v)
                load_raw<DT, true>(raw, vr + at * a.v.token, c, dv, i < n);
            else
                load_raw<DT, false>(raw, vr + at * a.v.token, c, dv, i < n);
            raw_floats<DT>(y, raw);
#pragma unroll
            for (int e = 0; e < 8; ++e) rv[h] = fmaf(x[e], y[e], rv[h]);
        }
        lds_barrier();
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            Frag<NP> fo;
            Frag<3> fr, fu;
            L.s.o.frag(fo, wave * 16, kb * 32);
            L.s.r.frag(fr, wave * 16, kb * 32);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                L.s.u.frag(fu, j * 16, kb * 32);
                mma<3>(dp[j], fo, fu);
                mma<3>(da[j], fr, fu);
            }
            Frag<3> fs[MT], fe[MT];
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const int d = (wave * MT + m) * 16 + row, c = c0 + kb * 32 + grp * 8;
                float x[8], y[8];
                load8(x, st + static_cast<int64_t>(d) * dv, c, d < dk ? dv : 0, vst);
                load8(y, de + static_cast<int64_t>(d) * dv, c, d < dk ? dv : 0, vst);
#pragma unroll
                for (int e = 0; e < 8; ++e) sde = fmaf(x[e], y[e], sde);
                split8(fs[m], x);
                split8(fe[m], y);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                L.s.o.frag(fo, j * 16, kb * 32);
                L.s.r.frag(fr, j * 16, kb * 32);
                L.s.u.frag(fu, j * 16, kb * 32);
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    mma<3>(aq[m][j], fo, fs[m]);
                    mma<3>(ar[m][j], fr, fs[m]);
                    mma<3>(as[m][j], fu, fe[m]);
                }
            }
        }
        lds_barrier();
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int m = 1; m < 8; m <<= 1) rv[h] += __shfl_xor(rv[h], m, 64);
        if ((threadIdx.x & 7) == 0) Rv[h * 32 + (threadIdx.x >> 3)] = rv[h];
    }

    const T* kr = rows_at<const T>(a.k, s, hk) + t0 * a.k.token;
    const T* qr = rows_at<const T>(a.q, s, hk) + t0 * a.q.token;
    // the state's part of each sum, and k . dks
    float ks = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const f32x4 eg = *reinterpret_cast<const f32x4*>(&Eg[j * 16 + grp * 4]);
        const f32x4 la = *reinterpret_cast<const f32x4*>(&La[j * 16 + grp * 4]);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            aq[m][j] *= eg * a.scale;
            ar[m][j] *= -eg;
            as[m][j] *= la;
            const int d = (wave * MT + m) * 16 + row;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = j * 16 + grp * 4 + e;
                if (i < n && d < dk) ks = fmaf(static_cast<float>(kr[i * a.k.token + d]), as[m][j][e], ks);
            }
        }
    }
    // dP, then dA: by rows against K, by columns against Q and K
    const uint16_t* kt = g.w.kt + sk * (NP * 64 * DKP);
    const uint16_t* qt = g.w.qt + sk * (NP * 64 * DKP);
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        if (which) lds_barrier();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f32x4 x = zero, y = zero;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = wave * 16 + grp * 4 + e, c = j * 16 + row;
                if (j <= wave && (which ? c < i : c <= i)) {
                    const float d = expf((Gh[i] - Gh[c]) + (Gl[i] - Gl[c]));
                    x[e] = which ? -da[j][e] * d : dp[j][e] * d * a.scale;
                    y[e] = which ? Be[i] * x[e] : x[e];
                }
            }
            bf16x4 xs[3];
            split4<3>(xs, x);
#pragma unroll
            for (int p = 0; p < 3; ++p)
#pragma unroll
                for (int e = 0; e < 4; ++e) *L.p.m.at(p, wave * 16 + grp * 4 + e, j * 16 + row) = xs[p][e];
            L.p.t.put(j * 16, wave * 16, y);
        }
        lds_barrier();
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            Frag<NP> fk[MT], fq[MT];
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                load_frag<NP>(fk[m], kt + static_cast<int64_t>((wave * MT + m) * 2 + kb) * NP * 512);
                if (!which) load_frag<NP>(fq[m], qt + static_cast<int64_t>((wave * MT + m) * 2 + kb) * NP * 512);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                Frag<3> fm, ft;
                if (kb * 2 <= j) {
                    L.p.m.frag(fm, j * 16, kb * 32);
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        if (which)
                            mma<3>(ar[m][j], fm, fk[m]);
                        else
                            mma<3>(aq[m][j], fm, fk[m]);
                    }
                }
                if (kb * 2 + 1 >= j) {
                    L.p.t.frag(ft, j * 16, kb * 32);
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        if (which)
                            mma<3>(as[m][j], ft, fk[m]);
                        else
                            mma<3>(as[m][j], ft, fq[m]);
                    }
                }
            }
        }
    }

    // write dq and dk; the row sums of dG and dbeta
    const bool parts = rr > 1;
    T* dqr = rows_at<T>(a.d_q, s, hk) + t0 * a.d_q.token;
    T* dkr = rows_at<T>(a.d_k, s, hk) + t0 * a.d_k.token;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float dG[4] = {0.f, 0.f, 0.f, 0.f}, dB[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const int d = (wave * MT + m) * 16 + row;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = j * 16 + grp * 4 + e;
                if (i >= n || d >= dk) continue;
                const float q = static_cast<float>(qr[i * a.q.token + d]), k = static_cast<float>(kr[i * a.k.token + d]);
                const float own_row = Be[i] * ar[m][j][e];
                dG[e] = fmaf(q, aq[m][j][e], fmaf(k, own_row - as[m][j][e], dG[e]));
                dB[e] = fmaf(k, ar[m][j][e], dB[e]);
                const float dkv = own_row + as[m][j][e];
                if (parts) {
                    g.w.dqp[(sv * 64 + i) * dk + d] = aq[m][j][e];
                    g.w.dkp[(sv * 64 + i) * dk + d] = dkv;
                } else {
                    dqr[i * a.d_q.token + d] = static_cast<T>(aq[m][j][e]);
                    dkr[i * a.d_k.token + d] = static_cast<T>(dkv);
                }
            }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
#pragma unroll
            for (int x = 1; x < 16; x <<= 1) {
                dG[e] += __shfl_xor(dG[e], x, 64);
                dB[e] += __shfl_xor(dB[e], x, 64);
            }
            if (row == 0) {
                red[wave][0][j * 16 + grp * 4 + e] = dG[e];
                red[wave][1][j * 16 + grp * 4 + e] = dB[e];
            }
        }
    }
#pragma unroll
    for (int x = 1; x < 64; x <<= 1) {
        ks += __shfl_xor(ks, x, 64);
        sde += __shfl_xor(sde, x, 64);
    }
    if (lane == 0) {
        tot[wave][0] = ks;
        tot[wave][1] = sde;
    }
    lds_barrier();
    if (wave == 0) {
        double x = 0.0;
        float db = Rv[lane];
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            x += red[w][0][lane];
            db += red[w][1][lane];
        }
        if (lane == 63) {
#pragma unroll
            for (int w = 0; w < 4; ++w) x += static_cast<double>(tot[w][0]) + static_cast<double>(Eg[63]) * tot[w][1];
        }
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const double y = __shfl_down(x, d, 64);
            if (lane + d < 64) x += y;
        }
        if (lane < n) {
            rows_at<float>(a.d_g, s, hv)[(t0 + lane) * a.d_g.token] = static_cast<float>(x);
            rows_at<float>(a.d_beta, s, hv)[(t0 + lane) * a.d_beta.token] = db;
        }
    }
}

// dq and dk of shared q/k heads: the value heads' parts, added in head order.
template <int DT>
__global__ __launch_bounds__(256) void gdr_shared(const GdrLaunch g) {
    using T = elem_t<DT>;
    const sdm_gdr_args_t& a = g.a;
    int seq, chunk;
    Seq s;
    const int slot = blockIdx.x, hk = blockIdx.y, rr = static_cast<int>(a.Hv / a.Hk), dk = static_cast<int>(a.dk);
    if (!owner(a, slot, seq, chunk, s)) return;
    const int t0 = chunk * kChunk, n = min(kChunk, s.len - t0);
    const float* src = blockIdx.z ? g.w.dkp : g.w.dqp;
    const sdm_rows_t& to = blockIdx.z ? a.d_k : a.d_q;
    T* out = rows_at<T>(to, s, hk) + t0 * to.token;
    const int64_t head = static_cast<int64_t>(64) * dk;
    src += (static_cast<int64_t>(slot) * a.Hv + hk * rr) * head;
    for (int i = threadIdx.x; i < n * dk; i += 256) {
        float x = src[i];
        for (int h = 1; h < rr; ++h) x += src[h * head + i];
        out[i / dk * to.token + i % dk] = static_cast<T>(x);
    }
}

template <int DT>
hipError_t run(const GdrLaunch& g, hipStream_t s) {
    const dim3 grid(static_cast<unsigned>(g.slots), static_cast<unsigned>(g.a.Hv));
    if (g.dkp == 64)
        gdr_grad<DT, 64><<<grid, 256, 0, s>>>(g);
    else if (g.dkp == 128)
        gdr_grad<DT, 128><<<grid, 256, 0, s>>>(g);
    else
        gdr_grad<DT, 256><<<grid, 256, 0, s>>>(g);
    if (g.a.Hv != g.a.Hk) {
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        gdr_shared<DT><<<dim3(grid.x, static_cast<unsigned>(g.a.Hk), 2), 256, 0, s>>>(g);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_gdr_chunk(const GdrLaunch& g, bool backward, hipStream_t s);
hipError_t launch_gdr_scan(const GdrLaunch& g, int mode, hipStream_t s);

hipError_t launch_gdr_forward(const GdrLaunch& g, hipStream_t s) {
    if (g.slots) {
        const hipError_t e = launch_gdr_chunk(g, false, s);
        if (e != hipSuccess) return e;
    }
    return launch_gdr_scan(g, 0, s);
}

hipError_t launch_gdr_backward(const GdrLaunch& g, hipStream_t s) {
    hipError_t e;
    if (g.slots && (e = launch_gdr_chunk(g, true, s)) != hipSuccess) return e;
    if (g.slots && (e = launch_gdr_scan(g, 1, s)) != hipSuccess) return e;
    if ((e = launch_gdr_scan(g, 2, s)) != hipSuccess || !g.slots) return e;
    switch (g.a.dtype) {
        case SDM_F32: return run<0>(g, s);
        case SDM_BF16: return run<1>(g, s);
        default: return run<2>(g, s);
    }
}

}  // namespace sdm_delta
