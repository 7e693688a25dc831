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
// straight from memory in operand layout, ahead of its use. Heads of 128 in bfloat16: a step takes 1.22 us alone and 1.90 us
// with 256 workgroups, each of which reads some 86 KB of operands a step (16384 tokens of 32 heads: 487 us).
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
__device__ __forceinline__ void load4(Tokens4<DT>& v, const elem_t<DT>* __restrict__ p, int stride, int t, int n) {
#pragma unroll
    for (int e = 0; e < 4; ++e) v.x[e] = p[static_cast<int64_t>(min(t + e, n - 1)) * stride];
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
__device__ __forceinline__ void put4(T* __restrict__ p, int stride, int t, int n, const f32x4& v) {
    p += static_cast<int64_t>(t) * stride;
    if (t + 4 <= n) {
#pragma unroll
        for (int e = 0; e < 4; ++e) p[static_cast<int64_t>(e) * stride] = static_cast<T>(v[e]);
    } else {
#pragma unroll
        for (int e = 0; e < 3; ++e)
            if (t + e < n) p[static_cast<int64_t>(e) * stride] = static_cast<T>(v[e]);
    }
}

// Sums of products of fragments over k blocks, in two accumulators that take turns: a product that waits for the one
// before takes half as long again.
template <int KBS, int NA, int NB>
__device__ __forceinline__ void products(f32x4 (&x)[2], const Frag<NA>* a, const Frag<NB>* b) {
    int i = 0;
#pragma unroll
    for (int k = 0; k < KBS; ++k)
#pragma unroll
        for (int s = 2; s >= 0; --s)
#pragma unroll
            for (int p = 0; p < NA; ++p)
                if (s - p >= 0 && s - p < NB) {
                    x[i & 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[k].p[p], b[k].p[s - p], x[i & 1], 0, 0, 0);
                    ++i;
                }
}
template <int KBS, class TileT, int N>
__device__ __forceinline__ void read(Frag<N>* b, const TileT& B, int row0, int k0) {
#pragma unroll
    for (int k = 0; k < KBS; ++k) B.frag(b[k], row0, k0 + k * 32);
}
// LDS reads above are issued before anything below
__device__ __forceinline__ void reads_first() { __builtin_amdgcn_sched_barrier(0); }

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
__device__ __forceinline__ void store_state(const f32x4 (&S)[Tiles<DKP>::MT][NT], const Scan& w, float* st, int dv) {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int c = w.c0 + t * 16 + w.row;
        if (c >= dv) continue;
#pragma unroll
        for (int m = 0; m < Tiles<DKP>::MT; ++m)
            put4(st + c, dv, (Tiles<DKP>::first(w) + m) * 16 + w.grp * 4, w.dk, S[m][t]);
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
    // a 64 x 64 matrix: this wavefront's rows, the k blocks K0 .. K0 + KN - 1 that are not all zero
    template <int K0, int KN, int N>
    __device__ __forceinline__ void square(Frag<N> (&f)[KN], uint16_t* from, int chunk) const {
#pragma unroll
        for (int k = 0; k < KN; ++k) load_frag<N>(f[k], frag_at<N>(from + sv(chunk) * (N * 4096), w.part, K0 + k, 2));
    }
    __device__ __forceinline__ f32x4 token(int field, int chunk) const {
        return *reinterpret_cast<const f32x4*>(g.w.tok + (sv(chunk) * kTokFields + field) * 64 + w.part * 16 + w.grp * 4);
    }
    __device__ __forceinline__ float whole(int chunk) const { return g.w.tok[(sv(chunk) * kTokFields + kTokEg) * 64 + 63]; }
};

// Operands are fetched one chunk ahead; in the backward scan two where the registers hold two chunks (bfloat16, the whole
// gradient: 4096 tokens x 2 heads of 128 231 us with one and 222 with two, 2 x 4096 x 16 heads 562 and 566; the forward
// scans take as long or longer with two, 4 x 2048 tokens x 32 heads 250 us with one and 264); with wide float32 heads not
// even one: K^T (and Q^T) come in the middle of their own step.
template <int DT, int DKP, int NT> constexpr int kBackDepth = DT == 1 && DKP <= 128 && NT == 1 ? 2 : 1;
template <int DT, int DKP, int NT> constexpr bool kLate = (DT != 1 && DKP > 128) || (DT == 0 && DKP * NT >= 256);
// k blocks of S in registers at once
template <int DT, int DKP, int NT> constexpr int kHalf = DT == 0 ? (DKP * NT >= 256 ? 1 : 2) : DKP == 128 ? 4 : 2;

// step(chunk, set), sets of operands taking turns. Where two paths meet inside a scan's loop, registers that loads are
// still on their way to would be moved, and the moves wait: hence no branch in it, and a loop of its own for each kind of
// wavefront.
template <int DEPTH, class F>
__device__ __forceinline__ void in_turn(int chunks, F step) {
    if constexpr (DEPTH == 1) {
        for (int i = 0; i < chunks; ++i) step(i, std::integral_constant<int, 0>{}, std::integral_constant<int, 0>{});
    } else {
        int i = 0;
        for (; i + 1 < chunks; i += 2) {
            step(i, std::integral_constant<int, 0>{}, std::integral_constant<int, 1>{});
            step(i + 1, std::integral_constant<int, 1>{}, std::integral_constant<int, 0>{});
        }
        if (i < chunks) step(i, std::integral_constant<int, 0>{}, std::integral_constant<int, 1>{});
    }
}

template <int DT, int DKP, int NT, bool STORE>
__global__ __launch_bounds__(kScanThreads, 2) void gdr_scan(const GdrLaunch g, const int total) {
    constexpr int NP = kParts<DT>, NKB = DKP / 32, MT = Tiles<DKP>::MT, COLS = 16 * NT;
    constexpr int HALF = kHalf<DT, DKP, NT>;
    constexpr bool LATE = kLate<DT, DKP, NT>;
    using T = elem_t<DT>;
    __shared__ Tile<3, COLS, DKP> Sx;           // S, [column][dk]
    __shared__ Tile<3, COLS, 64> Rx, Dx;            // R and exp(G_C - G) U, [column][token]
    __shared__ Tile<3, COLS, 64> Ux[STORE ? 1 : 2];    // U, of even and odd chunks
    const sdm_gdr_args_t& a = g.a;
    Scan w;
    if (!scan_of(w, a, total, COLS)) return;
    const int tok = w.part * 16, t4 = tok + w.grp * 4, hv = w.hv, dv = w.dv, chunks = w.chunks;
    const Operands<NP, DKP> from{g, w};
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
    // tokens with a value in this lane's column: none in a column past dv, whose state stays zero
    auto held = [&](int t, int n) { return w.c0 + t * 16 + w.row < dv ? n : 0; };
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
            store_state<DKP, NT>(S, w, g.w.st + from.sv(chunk) * w.dk * g.dvp, g.dvp);
    };
    auto update = [&](const Frag<NP> (&kt)[MT][2], float whole, auto chain, auto meanwhile) {
        if constexpr (!Tiles<DKP>::owns(decltype(chain)::value)) return;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            Frag<3> b[2];
            read<2>(b, Dx, t * 16, 0);
            reads_first();
            if (t == 0) meanwhile();
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                f32x4 y[2] = {S[m][t] * whole, zero};
                products<2>(y, kt[m], b);
                S[m][t] = y[0] + y[1];
                Sx.put(t * 16, (Tiles<DKP>::first(w) + m) * 16, S[m][t]);
            }
        }
    };
    // Each operand's next chunk is fetched as soon as this one's is used (the last steps fetch the last chunk again).
    // T and P are lower triangular: the first 32 tokens' rows have one k block
    auto run_chain = [&](auto kn) {
        constexpr int KN = decltype(kn)::value;
        const T* vr = rows_at<const T>(a.v, w.s, hv);
        struct {
            Frag<NP> kf[NKB], kt[MT][2];
            Frag<3> inv[KN];
            Tokens4<DT> v[NT];
            f32x4 eg, last, beta;
            float whole;
        } f;
        auto fetch_r = [&](int chunk) {
            const int t0 = chunk * kChunk, n = min(kChunk, w.s.len - t0);
            from.rows(f.kf, g.w.kf, chunk);
            f.eg = from.token(kTokEg, chunk);
            f.beta = from.token(kTokBeta, chunk);
#pragma unroll
            for (int c = 0; c < NT; ++c)
                load4<DT>(f.v[c], vr + t0 * a.v.token + min(w.c0 + c * 16 + w.row, dv - 1), static_cast<int>(a.v.token), t4, n);
        };
        auto fetch_u = [&](int chunk) {
            from.template square<0, KN>(f.inv, g.w.inv, chunk);
            f.last = from.token(kTokLast, chunk);
        };
        auto fetch_s = [&](int chunk) {
            from.template cols<true>(f.kt, g.w.kt, chunk);
            f.whole = from.whole(chunk);
        };
        fetch_r(0);
        fetch_u(0);
        if constexpr (!LATE) fetch_s(0);
        loads_landed();
        __builtin_amdgcn_s_setprio(2);      // over the outputs' wavefronts
        for (int chunk = 0; chunk < chunks; ++chunk) {
            const int next = min(chunk + 1, chunks - 1), n = min(kChunk, w.s.len - chunk * kChunk);
            keep(chunk, std::true_type{});
            lds_barrier();      // S is in LDS
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                f32x4 x[2] = {zero, zero};
#pragma unroll
                for (int k0 = 0; k0 < NKB; k0 += HALF) {
                    Frag<3> b[HALF];
                    read<HALF>(b, Sx, t * 16, k0 * 32);
                    reads_first();
                    products<HALF>(x, f.kf + k0, b);
                }
                Rx.put(t * 16, tok, f.beta * (floats4<DT>(f.v[t], t4, held(t, n)) - f.eg * (x[0] + x[1])));
            }
            lds_barrier();
            f32x4 u[NT];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                Frag<3> b[KN];
                read<KN>(b, Rx, t * 16, 0);
                reads_first();
                if (t == 0) {
                    if constexpr (LATE) fetch_s(chunk);
                    else fetch_r(next);
                }
                f32x4 y[2] = {zero, zero};
                products<KN>(y, f.inv, b);
                u[t] = y[0] + y[1];
                Dx.put(t * 16, tok, f.last * u[t]);
            }
            lds_barrier();
            update(f.kt, f.whole, std::true_type{}, [&] {
                fetch_u(next);
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    if constexpr (!STORE) Ux[chunk & 1].put(t * 16, tok, u[t]);
            });
            if constexpr (STORE) {
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    if (w.c0 + t * 16 + w.row < g.dvp)
                        put4(g.w.u + from.sv(chunk) * 64 * g.dvp + w.c0 + t * 16 + w.row, g.dvp, t4, kChunk, u[t]);
            }
            if constexpr (LATE) fetch_r(next);
            else fetch_s(next);
        }
        if constexpr (!STORE) lds_barrier();    // the last chunk's U
    };
    auto run_outputs = [&](auto kn) {
        // Float16 heads of 128 hold two parts of Q and three of P: no more than two k blocks of S beside them, and with two
        // column tiles Q of the next chunk comes after the update (a lone head of 4096 tokens: 121 us so, 132 with Q late
        // and four k blocks; neither spills, all four at once with Q early do)
        constexpr int KN = decltype(kn)::value, OUT = DT == 2 && HALF > 2 ? 2 : HALF;
        constexpr bool QLATE = DT == 2 && DKP * NT >= 256;
        T* orow = STORE ? nullptr : rows_at<T>(a.o, w.s, hv);
        struct {
            Frag<NP> qf[STORE ? 1 : NKB], kt[MT][2];
            Frag<3> pm[KN];
            f32x4 eg;
            float whole;
        } f;
        f32x4 o[NT];
        // the outputs of a chunk: P U on top of what Q S left
        auto finish = [&](int chunk) {
            const int t0 = chunk * kChunk, n = min(kChunk, w.s.len - t0);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                Frag<3> b[KN];
                read<KN>(b, Ux[STORE ? 0 : chunk & 1], t * 16, 0);
                reads_first();
                f32x4 y[2] = {o[t], zero};
                products<KN>(y, f.pm, b);
                y[0] += y[1];
                if (w.c0 + t * 16 + w.row < dv)
                    put4(orow + t0 * a.o.token + w.c0 + t * 16 + w.row, static_cast<int>(a.o.token), t4, n, y[0]);
            }
        };
        auto fetch_q = [&](int chunk) {
            if constexpr (!STORE) {
                from.rows(f.qf, g.w.qf, chunk);
                f.eg = from.token(kTokEg, chunk);
            }
        };
        auto fetch_s = [&](int chunk) {
            from.template cols<false>(f.kt, g.w.kt, chunk);
            f.whole = from.whole(chunk);
        };
        fetch_q(0);
        if constexpr (!STORE) from.template square<0, KN>(f.pm, g.w.pm, 0);
        if constexpr (!LATE) fetch_s(0);
        loads_landed();
        for (int chunk = 0; chunk < chunks; ++chunk) {
            const int next = min(chunk + 1, chunks - 1);
            keep(chunk, std::false_type{});
            lds_barrier();
            if constexpr (!STORE) {
                if (chunk) {
                    finish(chunk - 1);
                    from.template square<0, KN>(f.pm, g.w.pm, chunk);
                }
            }
            lds_barrier();
            if constexpr (LATE) fetch_s(chunk);
            if constexpr (!STORE) {
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    f32x4 x[2] = {zero, zero};
#pragma unroll
                    for (int k0 = 0; k0 < NKB; k0 += OUT) {
                        Frag<3> b[OUT];
                        read<OUT>(b, Sx, t * 16, k0 * 32);
                        reads_first();
                        products<OUT>(x, f.qf + k0, b);
                    }
                    o[t] = (x[0] + x[1]) * (f.eg * a.scale);
                }
            }
            if constexpr (!LATE && !QLATE) fetch_q(next);
            lds_barrier();
            update(f.kt, f.whole, std::false_type{}, [] {});
            if constexpr (LATE || QLATE) fetch_q(next);
            if constexpr (!LATE) fetch_s(next);
        }
        if constexpr (!STORE) {
            lds_barrier();
            finish(chunks - 1);
        }
    };
    using One = std::integral_constant<int, kSkipZero<DT, DKP> ? 1 : 2>;
    using Two = std::integral_constant<int, 2>;
    if (chunks) {
        const bool one = kSkipZero<DT, DKP> && w.part < 2;
        if (w.chain && one)
            run_chain(One{});
        else if (w.chain)
            run_chain(Two{});
        else if (one)
            run_outputs(One{});
        else
            run_outputs(Two{});
    }
    if constexpr (!STORE)
        if (a.s_final && Tiles<DKP>::owner(w)) store_state<DKP, NT>(S, w, a.s_final + w.head * w.dk * dv, dv);
}

template <int DT, int DKP, int NT>
__global__ __launch_bounds__(kScanThreads, 2) void gdr_scan_back(const GdrLaunch g, const int total) {
    constexpr int NP = kParts<DT>, NKB = DKP / 32, MT = Tiles<DKP>::MT, COLS = 16 * NT;
    constexpr int HALF = kHalf<DT, DKP, NT>, DEPTH = kBackDepth<DT, DKP, NT>;
    constexpr bool LATE = kLate<DT, DKP, NT>;
    using T = elem_t<DT>;
    __shared__ Tile<3, COLS, DKP> Sx;           // dS, [column][dk]
    __shared__ Tile<3, COLS, 64> Ox, Qx, Ux, Rx;    // the next chunk's dO, scale exp(G) dO, dU and -beta exp(G) dR
    __shared__ f32x4 Wx[NT][4][64];                 // P^T dO, as the chain's wavefronts hold dU
    const sdm_gdr_args_t& a = g.a;
    Scan w;
    if (!scan_of(w, a, total, COLS)) return;
    const int tok = w.part * 16, t4 = tok + w.grp * 4, hv = w.hv, dv = w.dv, top = w.chunks - 1;
    const Operands<NP, DKP> from{g, w};
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
    // tokens with a value in this lane's column: none in a column past dv, whose state stays zero
    auto held = [&](int t, int n) { return w.c0 + t * 16 + w.row < dv ? n : 0; };
    f32x4 S[MT][NT];
    load_state<DKP, NT>(S, w, Tiles<DKP>::owner(w) ? a.ds_final : nullptr);
    if (Tiles<DKP>::owner(w)) {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int t = 0; t < NT; ++t) Sx.put(t * 16, (Tiles<DKP>::first(w) + m) * 16, S[m][t]);
    }
    auto keep = [&](int chunk, auto chain) {
        if constexpr (Tiles<DKP>::owns(decltype(chain)::value))
            store_state<DKP, NT>(S, w, g.w.dst + from.sv(chunk) * w.dk * g.dvp, g.dvp);
    };
    auto update = [&](const Frag<NP> (&qt)[MT][2], const Frag<NP> (&kt)[MT][2], float whole, auto chain, auto meanwhile) {
        if constexpr (!Tiles<DKP>::owns(decltype(chain)::value)) return;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            Frag<3> bq[2], br[2];
            read<2>(bq, Qx, t * 16, 0);
            read<2>(br, Rx, t * 16, 0);
            reads_first();
            if (t == 0) meanwhile();
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                f32x4 y[2] = {S[m][t] * whole, zero};
                products<2>(y, qt[m], bq);
                products<2>(y, kt[m], br);
                S[m][t] = y[0] + y[1];
                Sx.put(t * 16, (Tiles<DKP>::first(w) + m) * 16, S[m][t]);
            }
        }
    };
    const auto back = [&](int i) { return max(top - i, 0); };       // the i-th chunk from the end
    // T^T and P^T are upper triangular: the last 32 tokens' rows have one k block
    auto run_chain = [&](auto kn) {
        constexpr int KN = decltype(kn)::value, K0 = 2 - KN;
        T* dvr = rows_at<T>(a.d_v, w.s, hv);
        struct Set {
            Frag<NP> kf[NKB], kt[MT][2], qt[MT][2];
            Frag<3> inv[KN];
            f32x4 eg, last, beta;
            float whole;
        } set[DEPTH];
        auto fetch_u = [&](Set& f, int chunk) {
            from.rows(f.kf, g.w.kf, chunk);
            f.last = from.token(kTokLast, chunk);
        };
        auto fetch_r = [&](Set& f, int chunk) {
            from.template square<K0, KN>(f.inv, g.w.invt, chunk);
        };
        auto fetch_s = [&](Set& f, int chunk) {
            from.template cols<true>(f.kt, g.w.kt, chunk);
            from.template cols<true>(f.qt, g.w.qt, chunk);
            f.whole = from.whole(chunk);
        };
        auto fetch_v = [&](Set& f, int chunk) {
            f.eg = from.token(kTokEg, chunk);
            f.beta = from.token(kTokBeta, chunk);
        };
#pragma unroll
        for (int i = 0; i < DEPTH; ++i) {
            fetch_u(set[i], back(i));
            fetch_r(set[i], back(i));
            fetch_v(set[i], back(i));
            if constexpr (!LATE) fetch_s(set[i], back(i));
        }
        loads_landed();
        __builtin_amdgcn_s_setprio(2);
        lds_barrier();
        in_turn<DEPTH>(top + 1, [&](int i, auto turn, auto other) {
            Set &f = set[turn], &before = set[other];
            const int chunk = top - i, next = back(i + DEPTH), t0 = chunk * kChunk, n = min(kChunk, w.s.len - t0);
            keep(chunk, std::true_type{});
            lds_barrier();      // dS and P^T dO are in LDS
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                f32x4 x[2] = {zero, zero};
#pragma unroll
                for (int k0 = 0; k0 < NKB; k0 += HALF) {
                    Frag<3> b[HALF];
                    read<HALF>(b, Sx, t * 16, k0 * 32);
                    reads_first();
                    if (DEPTH == 2 && t == 0 && k0 == 0) {
                        fetch_r(before, back(i + 1));
                        fetch_s(before, back(i + 1));
                    }
                    products<HALF>(x, f.kf + k0, b);
                }
                Ux.put(t * 16, tok, (x[0] + x[1]) * f.last + Wx[t][w.part][w.lane]);
            }
            lds_barrier();
            f32x4 d[NT];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                Frag<3> b[KN];
                read<KN>(b, Ux, t * 16, K0 * 32);
                reads_first();
                if (t == 0) {
                    if constexpr (LATE) fetch_s(f, chunk);
                    else fetch_u(f, next);
                }
                f32x4 y[2] = {zero, zero};
                products<KN>(y, f.inv, b);
                d[t] = y[0] + y[1];
                Rx.put(t * 16, tok, -(f.beta * f.eg) * d[t]);
            }
            lds_barrier();
            const f32x4 beta = f.beta;
            update(f.qt, f.kt, f.whole, std::true_type{}, [&] {
                if constexpr (DEPTH == 1) fetch_r(f, next);
                fetch_v(f, next);
            });
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const int c = w.c0 + t * 16 + w.row;
                if (c < g.dvp) put4(g.w.dr + from.sv(chunk) * 64 * g.dvp + c, g.dvp, t4, kChunk, d[t]);
                if (c < dv) {
                    put4(dvr + t0 * a.d_v.token + c, static_cast<int>(a.d_v.token), t4, n, beta * d[t]);
                }
            }
            if constexpr (LATE) fetch_u(f, next);
            else if constexpr (DEPTH == 1) fetch_s(f, next);
        });
    };
    auto run_outputs = [&](auto kn) {
        constexpr int KN = decltype(kn)::value, K0 = 2 - KN;
        const T* dor = rows_at<const T>(a.d_o, w.s, hv);
        struct Set {
            Frag<NP> kt[MT][2], qt[MT][2];
            Frag<3> pm[KN];                 // P^T of the next chunk
            Tokens4<DT> raw[NT];            // dO of the next chunk
            f32x4 eg;
            float whole;
        } set[DEPTH];
        f32x4 o1[NT];                       // dO of this chunk
        auto fetch_do = [&](Set& f, int chunk) {
            const int t0 = chunk * kChunk, n = min(kChunk, w.s.len - t0);
#pragma unroll
            for (int c = 0; c < NT; ++c)
                load4<DT>(f.raw[c], dor + t0 * a.d_o.token + min(w.c0 + c * 16 + w.row, dv - 1), static_cast<int>(a.d_o.token), t4, n);
        };
        auto fetch_s = [&](Set& f, int chunk) {
            from.template cols<false>(f.kt, g.w.kt, chunk);
            from.template cols<false>(f.qt, g.w.qt, chunk);
            f.whole = from.whole(chunk);
        };
        auto p_do = [&](const Frag<3>* pm) {    // P^T dO of the chunk in Ox, for the chain's next step
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                Frag<3> b[KN];
                read<KN>(b, Ox, t * 16, K0 * 32);
                reads_first();
                f32x4 y[2] = {zero, zero};
                products<KN>(y, pm, b);
                Wx[t][w.part][w.lane] = y[0] + y[1];
            }
        };
        from.template square<K0, KN>(set[0].pm, g.w.pm, top);
        fetch_do(set[0], top);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            o1[t] = floats4<DT>(set[0].raw[t], t4, held(t, min(kChunk, w.s.len - top * kChunk)));
            Ox.put(t * 16, tok, o1[t]);
        }
        lds_barrier();
        p_do(set[0].pm);
#pragma unroll
        for (int i = 0; i < DEPTH; ++i) {
            from.template square<K0, KN>(set[i].pm, g.w.pm, back(i + 1));
            fetch_do(set[i], back(i + 1));
            set[i].eg = from.token(kTokEg, back(i));
            if constexpr (!LATE) fetch_s(set[i], back(i));
        }
        loads_landed();
        in_turn<DEPTH>(top + 1, [&](int i, auto turn, auto) {
            Set& f = set[turn];
            const int chunk = top - i, n = min(kChunk, w.s.len - back(i + 1) * kChunk);
            keep(chunk, std::false_type{});
            lds_barrier();
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                Qx.put(t * 16, tok, o1[t] * (f.eg * a.scale));
                o1[t] = floats4<DT>(f.raw[t], t4, held(t, n));
                Ox.put(t * 16, tok, o1[t]);
            }
            f.eg = from.token(kTokEg, back(i + DEPTH));
            fetch_do(f, back(i + 1 + DEPTH));
            lds_barrier();
            if constexpr (LATE) fetch_s(f, chunk);
            p_do(f.pm);
            from.template square<K0, KN>(f.pm, g.w.pm, back(i + 1 + DEPTH));
            lds_barrier();
            update(f.qt, f.kt, f.whole, std::false_type{}, [] {});
            if constexpr (!LATE) fetch_s(f, back(i + DEPTH));
        });
    };
    using One = std::integral_constant<int, kSkipZero<DT, DKP> ? 1 : 2>;
    using Two = std::integral_constant<int, 2>;
    if (top >= 0) {
        const bool one = kSkipZero<DT, DKP> && w.part >= 2;
        if (w.chain && one)
            run_chain(One{});
        else if (w.chain)
            run_chain(Two{});
        else if (one)
            run_outputs(One{});
        else
            run_outputs(Two{});
    }
    if (a.ds0 && Tiles<DKP>::owner(w)) store_state<DKP, NT>(S, w, a.ds0 + w.head * w.dk * dv, dv);
}

template <int DT, int DKP, int NT>
hipError_t scan(const GdrLaunch& g, int mode, hipStream_t s) {
    const int total = static_cast<int>(scan_groups(g.a, g.dkp)), grid = 8 * ((total + 7) / 8);
    if (mode == 0)
        gdr_scan<DT, DKP, NT, false><<<grid, kScanThreads, 0, s>>>(g, total);
    else if (mode == 1)
        gdr_scan<DT, DKP, NT, true><<<grid, kScanThreads, 0, s>>>(g, total);
    else
        gdr_scan_back<DT, DKP, NT><<<grid, kScanThreads, 0, s>>>(g, total);
    return hipGetLastError();
}
template <int DT, int DKP>
hipError_t scan(const GdrLaunch& g, int mode, hipStream_t s) {
    if constexpr (DKP <= 128)
        if (scan_tiles(g.a, DKP) == 2) return scan<DT, DKP, 2>(g, mode, s);
    return scan<DT, DKP, 1>(g, mode, s);
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
