// What a chunk's tokens alone determine: the decays, P = scale (Q K^T) decay, the inverse of I + A, and K and Q
// transposed, all laid out as matrix-core fragments for the scans.
//
// With G the running sum of g in a chunk, u of the chunk solves (I + A) U = R, A_ij = beta_i exp(G_i - G_j) k_i . k_j
// for j < i, R = beta (V - exp(G) K S). T = (I + A)^-1 is unit lower triangular. The 16 x 16 blocks on its diagonal
// come from forward substitution, one wavefront each; two levels of T21 = -T22 A21 T11 give the rest on the float32
// matrix cores. (Products of powers of A would need no substitution, but lose everything when keys repeat: the powers
// grow to 10^17 before they cancel.)
//
// G is summed in float64 and kept as two float32: a token that forgets almost everything (g = -100, or -inf, which is
// held at -1000: exp gives 0 either way) leaves the differences after it exact.
//
// One workgroup per chunk and value head. Few chunks are bounded by latency, about 1 MFLOP of matrix work against two
// chains of 16 substitution steps (10 us for 16 of them); 4 workgroups share a CU and fill each other's gaps, and many
// are bounded by memory (16384 tokens of 32 heads of 128 in bfloat16: 144 us, 720 MB, 5.0 TB/s).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "gdr_device.h"

namespace sdm_delta {
namespace {

constexpr int kLd = 68;     // row of a 64 x 64 float32 matrix in LDS

template <int DT, int DKP, bool BWD>
__global__ __launch_bounds__(kChunkThreads, DT == 0 && DKP == 128 ? 3 : DKP < 256 || DT == 1 ? 4 : 1) void gdr_chunk(const GdrLaunch g) {
    constexpr int NP = kParts<DT>, NKB = DKP / 32;
    using T = elem_t<DT>;
    // K's (or Q's) fragments, then A and the matrix that P, and after it T, are laid out in
    constexpr int kFragBytes = 64 * DKP * NP * 2, kMatBytes = 2 * 64 * kLd * 4;
    __shared__ alignas(16) char buf[kFragBytes > kMatBytes ? kFragBytes : kMatBytes];
    auto& As = *reinterpret_cast<float(*)[64][kLd]>(buf);
    auto& Ts = *reinterpret_cast<float(*)[64][kLd]>(buf + 64 * kLd * 4);
    uint16_t* const Kf = reinterpret_cast<uint16_t*>(buf);
    __shared__ alignas(16) float Gh[64], Gl[64], Be[64];
    const sdm_gdr_args_t& a = g.a;
    int seq, chunk;
    Seq s;
    const int slot = blockIdx.x, hv = blockIdx.y, r = static_cast<int>(a.Hv / a.Hk), hk = hv / r;
    if (!owner(a, slot, seq, chunk, s)) return;
    const int t0 = chunk * kChunk, n = min(kChunk, s.len - t0), dk = static_cast<int>(a.dk);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), row = lane & 15, grp = lane >> 4;
    const int64_t sv = static_cast<int64_t>(slot) * a.Hv + hv;

    // This wavefront's 16 tokens of K and Q as fragments: to LDS for the others, to memory for the scans
    const bool first = hv % r == 0;
    const int64_t sk = static_cast<int64_t>(slot) * a.Hk + hk, frag = sk * (NP * 64 * DKP);
    const T* kr = rows_at<const T>(a.k, s, hk) + t0 * a.k.token;
    const T* qr = rows_at<const T>(a.q, s, hk) + t0 * a.q.token;
    Frag<NP> kf[NKB], qf[NKB];
    {
        const int ti = wave * 16 + row, at = min(ti, n - 1);
        Raw<DT> xk[NKB], xq[NKB];
        float gt = 0.f, be = 0.f;
        if (wave == 0) {
            const int l = min(lane, n - 1);
            gt = rows_at<const float>(a.g, s, hv)[(t0 + l) * a.g.token];
            be = rows_at<const float>(a.beta, s, hv)[(t0 + l) * a.beta.token];
        }
        auto fetch = [&](auto vec) {
#pragma unroll
            for (int kb = 0; kb < NKB; ++kb) {
                load_raw<DT, decltype(vec)::value>(xk[kb], kr + at * a.k.token, kb * 32 + grp * 8, dk, ti < n);
                load_raw<DT, decltype(vec)::value>(xq[kb], qr + at * a.q.token, kb * 32 + grp * 8, dk, ti < n);
            }
        };
        if (g.vec_qk)
            fetch(std::true_type{});
        else
            fetch(std::false_type{});
        // the decays, while K and Q are on their way
        if (wave == 0) {
            double x = lane < n ? (gt < -1000.f ? -1000.f : gt) : 0.f;
            be = lane < n ? be : 0.f;
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const double y = __shfl_up(x, d, 64);
                if (lane >= d) x += y;
            }
            const double last = __shfl(x, 63, 64);
            const float hi = static_cast<float>(x), lo = static_cast<float>(x - hi);
            Gh[lane] = hi;
            Gl[lane] = lo;
            Be[lane] = be;
            float* tok = g.w.tok + sv * (kTokFields * 64);
            tok[kTokG * 64 + lane] = hi;
            tok[kTokGlo * 64 + lane] = lo;
            tok[kTokEg * 64 + lane] = exp_of(hi) * (1.f + lo);
            tok[kTokLast * 64 + lane] = exp_of(static_cast<float>(last - x));
            tok[kTokBeta * 64 + lane] = be;
        }
#pragma unroll
        for (int kb = 0; kb < NKB; ++kb) {
            raw_frag<DT>(kf[kb], xk[kb]);
            raw_frag<DT>(qf[kb], xq[kb]);
            store_frag<NP>(frag_at<NP>(Kf, wave, kb, NKB), kf[kb]);
            if (first) {
                store_frag<NP>(frag_at<NP>(g.w.kf + frag, wave, kb, NKB), kf[kb]);
                if constexpr (!BWD) store_frag<NP>(frag_at<NP>(g.w.qf + frag, wave, kb, NKB), qf[kb]);
            }
        }
    }
    lds_barrier();
    // K K^T and Q K^T, row tile `wave`. All column tiles, also those above the diagonal: the last wavefront needs them
    // all, so leaving them out of the others saves no time
    f32x4 kk[4], qk[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        kk[j] = qk[j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int kb = 0; kb < NKB; ++kb) {
            Frag<NP> bf;
            load_frag<NP>(bf, frag_at<NP>(Kf, j, kb, NKB));
            mma(kk[j], kf[kb], bf);
            mma(qk[j], qf[kb], bf);
        }
    }
    // K^T, and Q^T in the backward, once per q/k head: a fragment's eight tokens are eight 2-byte LDS reads
    auto transposed = [&](uint16_t* out) {
#pragma unroll 2
        for (int i = wave; i < DKP / 16 * 2; i += 4) {
            const int t = i >> 1, kb = i & 1, c = t * 16 + row;
            Frag<NP> f;
#pragma unroll
            for (int p = 0; p < NP; ++p)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int j = kb * 32 + grp * 8 + e;
                    const uint16_t x = frag_at<NP>(Kf, j >> 4, c >> 5, NKB)[p * 512 + ((j & 15) + (c >> 3 & 3) * 16) * 8 + (c & 7)];
                    f.p[p][e] = __builtin_bit_cast(__bf16, x);
                }
            store_frag<NP>(frag_at<NP>(out, t, kb, 2), f);
        }
    };
    if (first) transposed(g.w.kt + frag);
    lds_barrier();
    if constexpr (BWD) {
        if (first) {
#pragma unroll
            for (int kb = 0; kb < NKB; ++kb) store_frag<NP>(frag_at<NP>(Kf, wave, kb, NKB), qf[kb]);
            lds_barrier();
            transposed(g.w.qt + frag);
            lds_barrier();
        }
    }

    const f32x4 gh = *reinterpret_cast<const f32x4*>(&Gh[wave * 16 + grp * 4]);
    const f32x4 gl = *reinterpret_cast<const f32x4*>(&Gl[wave * 16 + grp * 4]);
    const f32x4 be = *reinterpret_cast<const f32x4*>(&Be[wave * 16 + grp * 4]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int i0 = wave * 16 + grp * 4, c = j * 16 + row;
        if (j > wave) {     // above the diagonal: A is not read there
#pragma unroll
            for (int e = 0; e < 4; ++e) Ts[i0 + e][c] = 0.f;
            continue;
        }
        const float ch = Gh[c], cl = Gl[c];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float d = c <= i0 + e ? exp_of((gh[e] - ch) + (gl[e] - cl)) : 0.f;
            As[i0 + e][c] = be[e] * kk[j][e] * d;
            Ts[i0 + e][c] = a.scale * qk[j][e] * d;
        }
    }
    lds_barrier();

    // P, row tiles in order; the backward's P^T, of columns
    {
        uint16_t* out = g.w.pm + sv * (3 * 4096);
        Frag<3> f;
        float v[8];
        const int t = wave;
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            if (kSkipZero<DT, DKP> && (BWD ? kb * 2 + 1 < t : kb * 2 > t)) continue;    // all zero: nothing reads it
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int m = t * 16 + row, k = kb * 32 + grp * 8 + e;
                v[e] = BWD ? Ts[k][m] : Ts[m][k];
            }
            split8(f, v);
            store_frag<3>(frag_at<3>(out, t, kb, 2), f);
        }
    }
    lds_barrier();

    // the diagonal blocks of T: lane c solves column c (the four lane groups repeat each other)
    {
        float t[16];
        const int b = wave * 16;
        int from = b;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            // A's rows are read four at a time, once the four before are nearly used: all at once are 120 registers
            if (i % 4 == 0 && i) asm volatile("" : "+v"(from) : "v"(t[i - 2]));
            float v = i == row ? 1.f : 0.f;
#pragma unroll
            for (int j = 0; j < i; ++j) v = fmaf(-As[from + i][b + j], t[j], v);
            t[i] = v;
        }
        // this wavefront's 16 rows of T, zero off the diagonal block until the levels below fill them
#pragma unroll
        for (int i = 0; i < 16; ++i) Ts[b + i][lane] = 0.f;
        if (grp == 0) {
#pragma unroll
            for (int i = 0; i < 16; ++i) Ts[b + i][b + row] = t[i];
        }
    }
    lds_barrier();
    // 16 -> 32: wavefronts 0 and 1, one 32 x 32 block each
    if (wave < 2) {
        const int b = wave * 32;
        f32x4 x = {0.f, 0.f, 0.f, 0.f}, y = x;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            x = __builtin_amdgcn_mfma_f32_16x16x4f32(As[b + 16 + row][b + grp * 4 + e], Ts[b + grp * 4 + e][b + row], x, 0, 0, 0);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            y = __builtin_amdgcn_mfma_f32_16x16x4f32(-Ts[b + 16 + row][b + 16 + grp * 4 + e], x[e], y, 0, 0, 0);
#pragma unroll
        for (int e = 0; e < 4; ++e) Ts[b + 16 + grp * 4 + e][b + row] = y[e];
    }
    lds_barrier();
    // 32 -> 64: wavefront (tile row, tile column) of the lower left 32 x 32; the blocks above the diagonal are zero
    {
        const int tr = wave >> 1, tc = wave & 1;
        f32x4 y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            f32x4 x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < 2; ++k) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    x = __builtin_amdgcn_mfma_f32_16x16x4f32(As[32 + m * 16 + row][k * 16 + grp * 4 + e],
                                                             Ts[k * 16 + grp * 4 + e][tc * 16 + row], x, 0, 0, 0);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e)
                y = __builtin_amdgcn_mfma_f32_16x16x4f32(-Ts[32 + tr * 16 + row][32 + m * 16 + grp * 4 + e], x[e], y, 0, 0, 0);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) Ts[32 + tr * 16 + grp * 4 + e][tc * 16 + row] = y[e];
    }
    lds_barrier();
    {
        Frag<3> f;
        float v[8];
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            const int m = wave * 16 + row, k = kb * 32 + grp * 8;
            if (!kSkipZero<DT, DKP> || kb * 2 <= wave) {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = Ts[m][k + e];
                split8(f, v);
                store_frag<3>(frag_at<3>(g.w.inv + sv * (3 * 4096), wave, kb, 2), f);
            }
            if (BWD && (!kSkipZero<DT, DKP> || kb * 2 + 1 >= wave)) {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = Ts[k + e][m];
                split8(f, v);
                store_frag<3>(frag_at<3>(g.w.invt + sv * (3 * 4096), wave, kb, 2), f);
            }
        }
    }
}

template <int DT, bool BWD>
hipError_t run(const GdrLaunch& g, hipStream_t s) {
    const dim3 grid(static_cast<unsigned>(g.slots), static_cast<unsigned>(g.a.Hv));
    if (g.dkp == 64)
        gdr_chunk<DT, 64, BWD><<<grid, kChunkThreads, 0, s>>>(g);
    else if (g.dkp == 128)
        gdr_chunk<DT, 128, BWD><<<grid, kChunkThreads, 0, s>>>(g);
    else
        gdr_chunk<DT, 256, BWD><<<grid, kChunkThreads, 0, s>>>(g);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_gdr_chunk(const GdrLaunch& g, bool backward, hipStream_t s) {
    switch (g.a.dtype) {
        case SDM_F32: return backward ? run<0, true>(g, s) : run<0, false>(g, s);
        case SDM_BF16: return backward ? run<1, true>(g, s) : run<1, false>(g, s);
        default: return backward ? run<2, true>(g, s) : run<2, false>(g, s);
    }
}

}  // namespace sdm_delta
