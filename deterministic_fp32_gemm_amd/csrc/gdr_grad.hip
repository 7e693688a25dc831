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
// One workgroup per chunk and value head. Each of eight wavefronts owns dk columns of dq and dk for all 64 tokens (half
// of them for dk <= 64), so S and dE are read and split once; dO, U and dR are staged in LDS by 64 columns of dv at a
// time. About 18 x 64 dk dv flops on up to six steps each. One workgroup a CU (104 KB of LDS, and some 240 registers at
// two wavefronts a SIMD; either alone would allow no second) leaves its waits open: for the loads of a block of 64
// columns, which are used as soon as they are asked for, and for the LDS reads that feed the matrix cores. 2 x 4096 tokens
// of 16 heads of 128 in bfloat16 take 191 us, 578 MB at 3.0 TB/s, the matrix cores busy for 24% of it.
//
// Token order. A result tile's lane holds rows 4 p .. 4 p + 3 (p = lane / 16), a fragment's lane elements 8 p .. 8 p + 7.
// Row r of token tile j is token 32 (j / 2) + 8 (r / 4) + 4 (j % 2) + r % 4: then the four tokens of a result lane are
// four of the eight in the same lane's fragment of K^T and Q^T, and the row sums with k and q need no further read.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdr_device.h"

namespace sdm_delta {
namespace {

// The sum over the 16 lanes of a row.
template <int CTRL>
__device__ __forceinline__ float dpp_add(float x) {
    return x + __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float row_sum16(float x) {
    x = dpp_add<0xb1>(x);       // lanes 1, 0, 3, 2 of each four
    x = dpp_add<0x4e>(x);       // 2, 3, 0, 1
    x = dpp_add<0x141>(x);      // 7 .. 0 of each eight
    return dpp_add<0x140>(x);   // 15 .. 0
}

__device__ __forceinline__ constexpr int token_of(int j, int r) { return 32 * (j >> 1) + 8 * (r >> 2) + 4 * (j & 1) + (r & 3); }

template <int DT, int DKP>
__global__ __launch_bounds__(kGradThreads, 2) void gdr_grad(const GdrLaunch g, const int heads) {
    constexpr int NP = kParts<DT>;
    constexpr int MT = 1, PASSES = DKP == 256 ? 2 : 1;  // dk tiles of a wavefront at a time; times
    constexpr int NJ = DKP >= 128 ? 4 : 2;              // its token tiles
    using T = elem_t<DT>;
    struct Staged {
        Tile<NP, 64, 64> o;
        Tile<3, 64, 64> u, r;
    };
    struct Pairs {
        Tile<3, 64, 64> m[2], t[2];     // dP and dA by rows and by columns
    };
    union Shared {
        Staged s;
        Pairs p;
        __device__ Shared() {}
    };
    __shared__ Shared L;
    __shared__ alignas(16) float Gh[64], Gl[64], Eg[64], La[64], Be[64], Rv[64], red[8][2][64], tot[8][2];
    const sdm_gdr_args_t& a = g.a;
    int seq, chunk;
    Seq s;
    const int slot = blockIdx.x, rr = static_cast<int>(a.Hv / a.Hk), hk = blockIdx.y * heads / rr;
    if (!owner(a, slot, seq, chunk, s)) return;
    const int t0 = chunk * kChunk, n = min(kChunk, s.len - t0);
    const int dk = static_cast<int>(a.dk), dv = static_cast<int>(a.dv);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int j0 = DKP >= 128 ? 0 : (wave >> 2) * 2;
    const int64_t sk = static_cast<int64_t>(slot) * a.Hk + hk;
    const int dvp = g.dvp;
    const uint16_t* kt = g.w.kt + sk * (NP * 64 * DKP);
    const uint16_t* qt = g.w.qt + sk * (NP * 64 * DKP);
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
    // the value heads of this workgroup: all that share the q/k head, whose dq and dk are summed here, or one of them
    constexpr bool SUM = PASSES == 1;
    f32x4 sq[SUM ? NJ : 1], sk4[SUM ? NJ : 1];
#pragma unroll
    for (int j = 0; j < (SUM ? NJ : 1); ++j) sq[j] = sk4[j] = zero;
#pragma unroll 1
    for (int h = 0; h < heads; ++h) {
    const int hv = blockIdx.y * heads + h;
    const int64_t sv = static_cast<int64_t>(slot) * a.Hv + hv;
    // not the same for every head (and pass) as far as the compiler knows: it would keep every address of one across the
    // loop, in scratch memory
    int id = threadIdx.x;
    asm volatile("" : "+v"(id));
    const int lane = id & 63;
    if (h) lds_barrier();
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
    const float* ur = g.w.u + sv * 64 * dvp;
    const float* rp = g.w.dr + sv * 64 * dvp;
    const float* st = g.w.st + sv * dk * dvp;
    const float* de = g.w.dst + sv * dk * dvp;

#pragma unroll 1
    for (int pass = 0; pass < PASSES; ++pass) {     // more than 128 columns of dk: the second half after the first
    const int tile0 = DKP >= 128 ? pass * 8 + wave : wave & 3;
    if (pass) lds_barrier();
    int row = lane & 15, grp = lane >> 4;
    if constexpr (PASSES > 1) asm volatile("" : "+v"(row), "+v"(grp));
    f32x4 dpa[4], aq[MT][NJ], ar[MT][NJ], as[MT][NJ];       // dpa: a row tile of dP (wavefronts 0 .. 3) or of dA
#pragma unroll
    for (int j = 0; j < 4; ++j) dpa[j] = zero;
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int m = 0; m < MT; ++m) aq[m][j] = ar[m][j] = as[m][j] = zero;
    float rv = 0.f, sde = 0.f;
    // staging: this thread's row and its token, 8 columns
    const int si = id >> 3, sc = (id & 7) * 8, stok = token_of(si >> 4, si & 15);
    struct {
        Raw<DT> o, v;
        Raw<0> u, r;
    } in;
    auto fetch = [&](int c0) {
        const int c = c0 + sc, at = min(stok, n - 1);
        if (g.vec_v) {
            load_raw<DT, true>(in.o, dor + at * a.d_o.token, c, dv, stok < n);
            load_raw<DT, true>(in.v, vr + at * a.v.token, c, dv, stok < n);
        } else {
            load_raw<DT, false>(in.o, dor + at * a.d_o.token, c, dv, stok < n);
            load_raw<DT, false>(in.v, vr + at * a.v.token, c, dv, stok < n);
        }
        load_raw<0, true>(in.u, ur + stok * dvp, c, dvp, true);
        load_raw<0, true>(in.r, rp + stok * dvp, c, dvp, true);
    };
    for (int c0 = 0; c0 < dv; c0 += 64) {
        fetch(c0);
        {
            float x[8], y[8];
            Frag<NP> fo;
            Frag<3> f;
            raw_frag<DT>(fo, in.o);
#pragma unroll
            for (int p = 0; p < NP; ++p) *reinterpret_cast<bf16x8*>(L.s.o.at(p, si, sc)) = fo.p[p];
            raw_floats<0>(x, in.u);
            split8(f, x);
#pragma unroll
            for (int p = 0; p < 3; ++p) *reinterpret_cast<bf16x8*>(L.s.u.at(p, si, sc)) = f.p[p];
            raw_floats<0>(y, in.r);
            split8(f, y);
#pragma unroll
            for (int p = 0; p < 3; ++p) *reinterpret_cast<bf16x8*>(L.s.r.at(p, si, sc)) = f.p[p];
            raw_floats<DT>(x, in.v);
#pragma unroll
            for (int e = 0; e < 8; ++e) rv = fmaf(x[e], y[e], rv);
        }
        lds_barrier();
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            Raw<0> xs[MT], ys[MT];
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const int d = (tile0 + m) * 16 + row, c = c0 + kb * 32 + grp * 8;
                const int64_t at = static_cast<int64_t>(min(d, dk - 1)) * dvp;
                load_raw<0, true>(xs[m], st + at, c, dvp, d < dk);
                load_raw<0, true>(ys[m], de + at, c, dvp, d < dk);
            }
            Frag<NP> fo;
            Frag<3> fr, fu;
            if (wave < 4) {
                L.s.o.frag(fo, wave * 16, kb * 32);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    L.s.u.frag(fu, j * 16, kb * 32);
                    mma(dpa[j], fo, fu);
                }
            } else {
                L.s.r.frag(fr, (wave - 4) * 16, kb * 32);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    L.s.u.frag(fu, j * 16, kb * 32);
                    mma(dpa[j], fr, fu);
                }
            }
            Frag<3> fs[MT];
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                float x[8], y[8];
                raw_floats<0>(x, xs[m]);
                raw_floats<0>(y, ys[m]);
#pragma unroll
                for (int e = 0; e < 8; ++e) sde = fmaf(x[e], y[e], sde);
                split8(fs[m], x);
            }
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                L.s.o.frag(fo, (j0 + j) * 16, kb * 32);
                L.s.r.frag(fr, (j0 + j) * 16, kb * 32);
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    mma(aq[m][j], fo, fs[m]);
                    mma(ar[m][j], fr, fs[m]);
                }
            }
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                float y[8];
                raw_floats<0>(y, ys[m]);
                split8(fs[m], y);
            }
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                L.s.u.frag(fu, (j0 + j) * 16, kb * 32);
#pragma unroll
                for (int m = 0; m < MT; ++m) mma(as[m][j], fu, fs[m]);
            }
        }
        lds_barrier();
    }
#pragma unroll
    for (int m = 1; m < 8; m <<= 1) rv += __shfl_xor(rv, m, 64);
    if ((id & 7) == 0) Rv[stok] = rv;
    if (DKP < 128 && wave >= 4) sde = 0.f;      // wavefronts 0 .. 3 have summed the same

    Frag<NP> fk[MT][2], fq[MT][2];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            load_frag<NP>(fk[m][kb], kt + static_cast<int64_t>((tile0 + m) * 2 + kb) * NP * 512);
            load_frag<NP>(fq[m][kb], qt + static_cast<int64_t>((tile0 + m) * 2 + kb) * NP * 512);
        }
    auto value = [](const Frag<NP>& f, int e) {
        float x = static_cast<float>(f.p[NP - 1][e]);
#pragma unroll
        for (int p = NP - 2; p >= 0; --p) x += static_cast<float>(f.p[p][e]);
        return x;
    };
    // the state's part of each sum, and k . dks
    float ks = 0.f;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        const int i0 = token_of(j0 + j, grp * 4);
        const f32x4 eg = *reinterpret_cast<const f32x4*>(&Eg[i0]);
        const f32x4 la = *reinterpret_cast<const f32x4*>(&La[i0]);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            aq[m][j] *= eg * a.scale;
            ar[m][j] *= -eg;
            as[m][j] *= la;
            const Frag<NP>& f = NJ == 4 || j0 == 0 ? fk[m][NJ == 4 ? j >> 1 : 0] : fk[m][1];
#pragma unroll
            for (int e = 0; e < 4; ++e) ks = fmaf(value(f, 4 * (j & 1) + e), as[m][j][e], ks);
        }
    }
    // dP and dA with their decays, half the wavefronts each: by rows against K, by columns against Q and, times beta, K
    {
        const int which = wave >> 2, wi = wave & 3, i0 = token_of(wi, grp * 4);
        const f32x4 gh = *reinterpret_cast<const f32x4*>(&Gh[i0]), gl = *reinterpret_cast<const f32x4*>(&Gl[i0]);
        const f32x4 one = {1.f, 1.f, 1.f, 1.f};
        const f32x4 be = which ? *reinterpret_cast<const f32x4*>(&Be[i0]) : one;
        const float sign = which ? -1.f : a.scale;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int c = token_of(j, row);
            const float ch = Gh[c], cl = Gl[c];
            f32x4 x;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const bool in = c < i0 + e + 1 - which;
                x[e] = in ? dpa[j][e] * sign * exp_of((gh[e] - ch) + (gl[e] - cl)) : 0.f;
            }
            bf16x4 xs[3];
            split4<3>(xs, x);
#pragma unroll
            for (int p = 0; p < 3; ++p)
#pragma unroll
                for (int e = 0; e < 4; ++e) *L.p.m[which].at(p, wi * 16 + grp * 4 + e, c) = xs[p][e];
            if (which) split4<3>(xs, x * be);
#pragma unroll
            for (int p = 0; p < 3; ++p) *reinterpret_cast<bf16x4*>(L.p.t[which].at(p, j * 16 + row, i0)) = xs[p];
        }
    }
    lds_barrier();
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            Frag<3> f;
            if (NJ < 4 || kb <= j >> 1) {       // a token's row reaches back, its column forward, by blocks of 32
                L.p.m[0].frag(f, (j0 + j) * 16, kb * 32);
#pragma unroll
                for (int m = 0; m < MT; ++m) mma(aq[m][j], f, fk[m][kb]);
                L.p.m[1].frag(f, (j0 + j) * 16, kb * 32);
#pragma unroll
                for (int m = 0; m < MT; ++m) mma(ar[m][j], f, fk[m][kb]);
            }
            if (NJ < 4 || kb >= j >> 1) {
                L.p.t[0].frag(f, (j0 + j) * 16, kb * 32);
#pragma unroll
                for (int m = 0; m < MT; ++m) mma(as[m][j], f, fq[m][kb]);
                L.p.t[1].frag(f, (j0 + j) * 16, kb * 32);
#pragma unroll
                for (int m = 0; m < MT; ++m) mma(as[m][j], f, fk[m][kb]);
            }
        }

    // write dq and dk; the row sums of dG and dbeta
    const bool parts = rr > heads, write = h + 1 == heads;
    T* dqr = rows_at<T>(a.d_q, s, hk) + t0 * a.d_q.token;
    T* dkr = rows_at<T>(a.d_k, s, hk) + t0 * a.d_k.token;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        f32x4 dG = zero, dB = zero;
        const int i0 = token_of(j0 + j, grp * 4);
        const f32x4 be = *reinterpret_cast<const f32x4*>(&Be[i0]);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const int d = (tile0 + m) * 16 + row;
            const Frag<NP>& k8 = NJ == 4 || j0 == 0 ? fk[m][NJ == 4 ? j >> 1 : 0] : fk[m][1];
            const Frag<NP>& q8 = NJ == 4 || j0 == 0 ? fq[m][NJ == 4 ? j >> 1 : 0] : fq[m][1];
            const f32x4 own = be * ar[m][j];
            f32x4 dqv = aq[m][j], dkv = own + as[m][j];
            if constexpr (SUM) {
                dqv = sq[j] += dqv;
                dkv = sk4[j] += dkv;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float q = value(q8, 4 * (j & 1) + e), k = value(k8, 4 * (j & 1) + e);
                dG[e] = fmaf(q, aq[m][j][e], fmaf(k, own[e] - as[m][j][e], dG[e]));
                dB[e] = fmaf(k, ar[m][j][e], dB[e]);
            }
            if (d < dk && write) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int i = i0 + e;
                    if (i >= n) continue;
                    if (parts) {
                        g.w.dqp[(sv * 64 + i) * dk + d] = dqv[e];
                        g.w.dkp[(sv * 64 + i) * dk + d] = dkv[e];
                    } else {
                        dqr[i * a.d_q.token + d] = static_cast<T>(dqv[e]);
                        dkr[i * a.d_k.token + d] = static_cast<T>(dkv[e]);
                    }
                }
            }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            dG[e] = row_sum16(dG[e]);
            dB[e] = row_sum16(dB[e]);
        }
        if (row == 0) {
            f32x4 &g4 = *reinterpret_cast<f32x4*>(&red[wave][0][i0]), &b4 = *reinterpret_cast<f32x4*>(&red[wave][1][i0]);
            g4 = pass ? g4 + dG : dG;
            b4 = pass ? b4 + dB : dB;
        }
    }
#pragma unroll
    for (int x = 1; x < 64; x <<= 1) {
        ks += __shfl_xor(ks, x, 64);
        sde += __shfl_xor(sde, x, 64);
    }
    if (lane == 0) {
        tot[wave][0] = pass ? tot[wave][0] + ks : ks;
        tot[wave][1] = pass ? tot[wave][1] + sde : sde;
    }
    }
    lds_barrier();
    if (wave == 0) {
        double x = 0.0;
        float db = Rv[lane];
        const int w0 = DKP >= 128 ? 0 : (lane >> 5) * 4;        // the wavefronts that hold this token
#pragma unroll
        for (int w = 0; w < (DKP >= 128 ? 8 : 4); ++w) {
            x += red[w0 + w][0][lane];
            db += red[w0 + w][1][lane];
        }
        if (lane == 63) {
#pragma unroll
            for (int w = 0; w < 8; ++w) x += static_cast<double>(tot[w][0]) + static_cast<double>(Eg[63]) * tot[w][1];
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
    // One workgroup for all value heads of a q/k head saves their parts of dq and dk a way through memory and a kernel;
    // few chunks go by one head each, for time (sequences of one chunk with two q/k heads, two value heads each, 128 wide
    // in bfloat16, the whole gradient by chunks x q/k heads: 32: 71 us together, 67 apart; 128: 109 and 111; 256: 182 and
    // 206; 1024: 720 and 775).
    const int rr = static_cast<int>(g.a.Hv / g.a.Hk);
    const int heads = g.dkp <= 128 && static_cast<int64_t>(g.slots) * g.a.Hk >= 256 ? rr : 1;
    const dim3 grid(static_cast<unsigned>(g.slots), static_cast<unsigned>(g.a.Hv / heads));
    if (g.dkp == 64)
        gdr_grad<DT, 64><<<grid, kGradThreads, 0, s>>>(g, heads);
    else if (g.dkp == 128)
        gdr_grad<DT, 128><<<grid, kGradThreads, 0, s>>>(g, heads);
    else
        gdr_grad<DT, 256><<<grid, kGradThreads, 0, s>>>(g, heads);
    if (heads != rr) {
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
