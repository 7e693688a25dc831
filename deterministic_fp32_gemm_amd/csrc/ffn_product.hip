// Products of the gated feed-forward on the matrix cores (sdm_ffn.h), for gfx950: C = A B^T from rows of A and B, and, as a
// pair, h = act(A Bg^T) * (A Bu^T) with both products' tiles in one wavefront's registers.
//
// Bounded by the matrix cores where M, N and K are large; a tile's operands go through LDS. All element types are laid out
// alike, by bytes: a step takes 128 bytes of each row, of which a lane holds 32 of row l % 32 for each half of the step
// (lanes 0 .. 31 the first 32 bytes of 64, lanes 32 .. 63 the other), two 16-byte pieces. Which element of a row meets which
// place of the instruction's summed axis does not matter as long as A and B agree, so the same pieces feed two
// v_mfma_f32_32x32x16 of 16-bit elements or one v_mfma_f32_32x32x64 of 8-bit ones, 64 clocks either way.
//
// 8-bit products: the instruction aligns 8 adjacent elements' products and cuts each off below 2^-13 of the largest (measured;
// the groups' sums have float32's bits). 16-bit instructions would not, at half the rate; for operands rounded to 2^-4 and a
// result of 16 bits the full rate is taken.
//
// Memory to LDS by buffer_load_dwordx4 ... lds, no registers between: 16 bytes of a lane go to 16 consecutive bytes a lane,
// so the order that keeps reads off one another's banks (piece c of row r at place c ^ (r % 8)) is made by the choice of each
// lane's source. Rows past M or N and pieces past the row's end read as zero by the buffer's bounds.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "block_device.h"
#include "ffn.h"

namespace sdm_delta {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kStep = 128;                      // bytes of a row a step
constexpr uint32_t kNowhere = 0x80000000u;      // an offset past every buffer: they are below 2 GB
constexpr uint32_t kBufferWord = 0x00027000u;   // a raw buffer of 32-bit data

struct Piece {
    u32x4 w[2];
};

template <int ET>
__device__ __forceinline__ void mma(f32x16& acc, const Piece& a, const Piece& b) {
    if constexpr (ET == kE4m3) {
        const i32x8 x = __builtin_bit_cast(i32x8, a), y = __builtin_bit_cast(i32x8, b);
        acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, y, acc, 0, 0, 0, 0, 0, 0);     // e4m3, no scales
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if constexpr (ET == kBf16)
                acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a.w[i]), __builtin_bit_cast(bf16x8, b.w[i]), acc, 0, 0, 0);
            else
                acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a.w[i]), __builtin_bit_cast(f16x8, b.w[i]), acc, 0, 0, 0);
    }
}

struct Buffer {
    const char* p;
    uint32_t n;
};
__device__ __forceinline__ u32x4 resource(const Buffer& b) {
    const uint64_t a = reinterpret_cast<uint64_t>(b.p);
    return u32x4{static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(a))),
                 static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(a >> 32))) & 0xffffu,
                 static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(b.n))), kBufferWord};
}
// 16 bytes a lane from offset `off` into LDS at `lds` + 16 lane. In assembly, since the compiler would otherwise wait for
// every load in flight before each read of LDS; wait_loads() below counts them.
__device__ __forceinline__ void load_lds(const u32x4& r, uint32_t lds, uint32_t off) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(lds), "v"(off), "s"(r) : "memory");
}
// All but this wavefront's last N loads have landed, every read of LDS has come back; then all wavefronts meet.
template <int N>
__device__ __forceinline__ void meet() {
    static_assert(N < 64, "the counter's 6 bits");
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// The workgroup's tile: workgroups go to the XCDs in turn, so each XCD takes a contiguous stretch of tiles, and a stretch
// goes through groups of 8 rows of tiles column by column: the 32 tiles that an XCD works on share A's and B's rows in its L2.
__device__ __forceinline__ void tile_of(int id, int tm, int tn, int& m, int& n) {
    const int total = tm * tn, q = total / 8, r = total % 8, xcd = id % 8, t = xcd * q + min(xcd, r) + id / 8;
    const int g = t / (8 * tn), first = g * 8, rows = min(8, tm - first), in = t - g * 8 * tn;
    m = first + in % rows;
    n = in / rows;
}

// Four consecutive columns of one row, of which `n` exist.
template <class T>
__device__ __forceinline__ void store4(T* p, int64_t n, const float (&v)[4]) {
    if (n >= 4) {
        if constexpr (sizeof(T) == 4) {
            typedef uint32_t u32x4a __attribute__((ext_vector_type(4), aligned(4)));
            *reinterpret_cast<u32x4a*>(p) = u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
        } else {
            typedef T t4 __attribute__((ext_vector_type(4)));
            typedef uint32_t u32x2u __attribute__((ext_vector_type(2), aligned(2)));
            const t4 x = {static_cast<T>(v[0]), static_cast<T>(v[1]), static_cast<T>(v[2]), static_cast<T>(v[3])};
            *reinterpret_cast<u32x2u*>(p) = __builtin_bit_cast(u32x2, x);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 3; ++i)
        if (i < n) p[i] = static_cast<T>(v[i]);
}
__device__ __forceinline__ void store4(int otype, char* base, int64_t at, int64_t n, const float (&v)[4]) {
    if (otype == SDM_F32)
        store4(reinterpret_cast<float*>(base) + at, n, v);
    else if (otype == SDM_BF16)
        store4(reinterpret_cast<__bf16*>(base) + at, n, v);
    else
        store4(reinterpret_cast<_Float16*>(base) + at, n, v);
}

struct Both {
    FfnProduct p[2];
    int tm[2], tn[2], first;       // tiles of each; workgroups of the first
};

// Tiles of T x T (as a pair: T rows and T / 2 columns of either product), four wavefronts of T/2 x T/2. A wavefront's part of
// B's tile is its columns of Bg, then the same of Bu. S steps of LDS: S - 1 of them in flight, or one and a half where S is 2.
// P parts of each operand a step: 3 for the small tiles of float32, whose six products then come from one step's reads (a
// sixth of the steps, half of the loads; 333 rows of 1111 to 777: 39 -> 17 us); the large tiles take a part of each a step.
template <int ET, int T, int S, int P, bool PAIR>
__global__ __launch_bounds__(256, T == 256 || P > 1 ? 1 : 2) void ffn_product(const Both both) {
    constexpr int W = T / 2, NB = W / 32, LOADS = 2 * T / 32;       // a wavefront's rows, blocks of 32, loads a step and part
    constexpr int PLACE = 2 * T * kStep;        // bytes of a step's part
    __shared__ __attribute__((aligned(1024))) char lds[S][P * PLACE];
    const int second = static_cast<int>(blockIdx.x) >= both.first ? 1 : 0;
    const FfnProduct& p = both.p[second];
    const int tm = both.tm[second], tn = both.tn[second];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wm = w >> 1, wn = w & 1;
    __builtin_assume(w >= 0 && w < 4);
    int ti, tj;
    tile_of(static_cast<int>(blockIdx.x) - (second ? both.first : 0), tm, tn, ti, tj);
    const int64_t m0 = static_cast<int64_t>(ti) * T, n0 = static_cast<int64_t>(tj) * (PAIR ? W : T);
    constexpr int BR = PAIR ? W : T;            // rows of a B that the tile takes
    auto rows_of = [&](const FfnOperand& o, int64_t first, int64_t all, int most) {
        const int64_t n = min(all - first, static_cast<int64_t>(most));
        return Buffer{o.p + first * o.ld, static_cast<uint32_t>((n - 1) * o.ld + p.bytes)};
    };
    const Buffer ba = rows_of(p.A, m0, p.M, T), bb = rows_of(p.B, n0, p.N, BR), bc = PAIR ? rows_of(p.B2, n0, p.N, BR) : bb;

    // Load j of wavefront w fills rows (4 j + w) 8 .. + 7 of the tile's A, then B: a lane's row and piece.
    const int r8 = lane >> 3, piece = (lane & 7) ^ r8;
    uint32_t off[LOADS];
#pragma unroll
    for (int j = 0; j < LOADS; ++j) {
        const int r = ((j % (LOADS / 2)) * 4 + w) * 8 + r8;
        if (j < LOADS / 2)
            off[j] = static_cast<uint32_t>(r * p.A.ld) + piece * 16;
        else if constexpr (PAIR)
            off[j] = static_cast<uint32_t>((r / W * (W / 2) + r % (W / 2)) * (r / (W / 2) % 2 ? p.B2.ld : p.B.ld)) + piece * 16;
        else
            off[j] = static_cast<uint32_t>(r * p.B.ld) + piece * 16;
    }
    const uint32_t base = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) char*)&lds[0][0]));
    const int segments = P > 1 ? 1 : p.segments, steps = static_cast<int>((p.bytes + kStep - 1) / kStep), total = steps * segments;
    // The next step's buffers; past the last step nothing is read.
    int seg = 0, at = 0;
    u32x4 ra[P], rb[P], rc[P];
    uint32_t none;
    auto next_step = [&]() {
        const int64_t from = static_cast<int64_t>(at) * kStep;
        auto part = [&](const Buffer& b, int64_t plane, uint32_t which) {
            return resource(Buffer{b.p + plane * which + from, b.n - static_cast<uint32_t>(from)});
        };
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const uint32_t ia = P > 1 ? i : p.aparts >> (2 * seg) & 3, ib = P > 1 ? i : p.bparts >> (2 * seg) & 3;
            ra[i] = part(ba, p.A.plane, ia);
            rb[i] = part(bb, p.B.plane, ib);
            rc[i] = PAIR ? part(bc, p.B2.plane, ib) : rb[i];
        }
        none = seg >= segments || from + piece * 16 >= p.bytes ? kNowhere : 0u;       // the row has ended
        if (++at == steps) {
            at = 0;
            ++seg;
        }
    };
    auto load = [&](int buf, int n) {
        const int i = n / LOADS, j = n % LOADS;
        const uint32_t to = base + buf * (P * PLACE) + i * PLACE + (j * 4 + w) * 1024;
        if (j < LOADS / 2)
            load_lds(ra[i], to, off[j] | none);
        else
            load_lds(PAIR && (j - LOADS / 2) * 32 + w * 8 & W / 2 ? rc[i] : rb[i], to, off[j] | none);
    };
    f32x16 acc[NB][NB];                         // [columns][rows]
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j) acc[i][j] = (f32x16){0};
    Piece fa[2][P][NB], fb[2][P][NB];
    const int lr = lane & 31, lh = lane >> 5, sw = lr & 7;
    constexpr int READS = 4 * NB * P, BLOCKS = NB * NB, AHEAD = BLOCKS > 1 ? BLOCKS / 2 : 1;
    // Read n of a half step, in the order in which the products want them: B's first block, A's, B's others.
    auto read = [&](int buf, int half, int n) {
        const int part = P - 1 - n / (4 * NB), k = n % (4 * NB), c = ((half * 4 + lh * 2 + k % 2) ^ sw) * 16, i = k / 2;
        const char* a = &lds[buf][part * PLACE + (wm * W + lr) * kStep + c];
        const char* b = &lds[buf][part * PLACE + (T + wn * W + lr) * kStep + c];
        if (i >= 1 && i <= NB)
            fa[half][part][i - 1].w[k % 2] = *reinterpret_cast<const u32x4*>(a + (i - 1) * 32 * kStep);
        else
            fb[half][part][i ? i - NB : 0].w[k % 2] = *reinterpret_cast<const u32x4*>(b + (i ? i - NB : 0) * 32 * kStep);
    };
    // the part products of a block, smallest first
    auto products = [&](int half, int i, int j) {
#pragma unroll
        for (int order = P - 1; order >= 0; --order)
#pragma unroll
            for (int x = order; x >= 0; --x) mma<ET>(acc[i][j], fb[half][order - x][i], fa[half][x][j]);
    };
    // A step's second half is read while its first is multiplied, and the next step's first half while the second is. Between
    // the two the wavefronts meet: all reads of this step are back, so its place takes the loads of the step S later, which
    // have S - 1 whole steps to land. Blocks of 64 clocks of products, with the reads behind the first half of them and the
    // loads spread over all, in the order written here (the compiler would gather the products behind the barrier).
    auto blocks = [&](int half, int from, bool loads, int to) {
#pragma unroll
        for (int n = 0; n < BLOCKS; ++n) {
            constexpr int kReads = READS / AHEAD, kLoads = P * LOADS / BLOCKS;
#pragma unroll
            for (int k = 0; k < kReads; ++k)
                if (n * kReads + k < READS) read(from, 1 - half, n * kReads + k);
            if (loads) {
#pragma unroll
                for (int k = 0; k < kLoads; ++k) load(to, n * kLoads + k);
            }
            products(half, n / NB, n % NB);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
#pragma unroll
    for (int s = 0; s < S; ++s) {
        next_step();
#pragma unroll
        for (int j = 0; j < P * LOADS; ++j) load(s, j);
    }
    meet<(S - 1) * P * LOADS>();
#pragma unroll
    for (int k = 0; k < READS; ++k) read(0, 0, k);
    for (int t = 0; t < total; ++t) {
        const int buf = t % S;
        blocks(0, buf, false, 0);
        next_step();
        meet<(S - 2) * P * LOADS>();
        __builtin_amdgcn_sched_barrier(0);
        blocks(1, (t + 1) % S, true, buf);
    }

    // Lane l holds columns 8 (i / 4) + 4 (l / 32) + i % 4 of row l % 32 of each block. 32 rows at a time go through the
    // wavefront's own part of LDS, so that its lanes store whole stretches of a row; rows there are 4 banks apart.
    meet<0>();
    constexpr int kRow = W * 4 + 16, kLanes = (PAIR ? W / 2 : W) / 4, kRows = 64 / kLanes;
    static_assert(4 * 32 * kRow <= sizeof(lds), "the wavefronts' rows fit");
    char* mine = &lds[0][0] + w * 32 * kRow;
    const int col = lane % kLanes * 4;
    const int64_t n = n0 + wn * (PAIR ? W / 2 : W) + col, left = p.N - n;
    float sg[4], su[4];
    if constexpr (ET == kE4m3) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int64_t c = min(n + e, p.N - 1);
            sg[e] = p.sn[c];
            su[e] = p.sn2[c];
        }
    }
#pragma unroll
    for (int j = 0; j < NB; ++j) {
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                *reinterpret_cast<f32x4*>(mine + lr * kRow + (i * 32 + q * 8 + lh * 4) * 4) =
                    f32x4{acc[i][j][q * 4], acc[i][j][q * 4 + 1], acc[i][j][q * 4 + 2], acc[i][j][q * 4 + 3]};
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
        for (int r = lane / kLanes; r < 32; r += kRows) {
            const int64_t m = m0 + wm * W + j * 32 + r;
            const f32x4* from = reinterpret_cast<const f32x4*>(mine + r * kRow + col * 4);
            if (m >= p.M || left <= 0) continue;
            const f32x4 x = from[0];
            float g[4] = {x[0], x[1], x[2], x[3]};
            if constexpr (!PAIR) {
                char* c = m < p.split ? p.c : p.c2;
                store4(p.otype, c, (m < p.split ? m * p.ldc : (m - p.split) * p.ldc2) + n, left, g);
            } else {
                const f32x4 y = from[W / 8];
                float u[4] = {y[0], y[1], y[2], y[3]}, h[4];
                if constexpr (ET == kE4m3) {
                    const float sm = p.sm[m];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        g[e] *= sm * sg[e];
                        u[e] *= sm * su[e];
                    }
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float f, d;
                    if (p.otype == SDM_F32)
                        gate<false>(g[e], p.act, f, d);
                    else
                        gate<true>(g[e], p.act, f, d);
                    h[e] = f * u[e];
                }
                store4(p.otype, p.c, m * p.ldc + n, left, h);
                if (p.gate) {
                    store4(p.gate + m * p.ld_gate + n, left, g);
                    store4(p.up + m * p.ld_up + n, left, u);
                }
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
    }
}

template <int ET, int T, int S, int P, bool PAIR>
hipError_t run(const FfnProduct* p, int n, hipStream_t s) {
    Both b{};
    int64_t total = 0;
    for (int i = 0; i < n; ++i) {
        b.p[i] = p[i];
        b.tm[i] = static_cast<int>((p[i].M + T - 1) / T);
        b.tn[i] = static_cast<int>((p[i].N + (PAIR ? T / 2 : T) - 1) / (PAIR ? T / 2 : T));
        total += static_cast<int64_t>(b.tm[i]) * b.tn[i];
        if (i == 0) b.first = static_cast<int>(total);
    }
    ffn_product<ET, T, S, P, PAIR><<<static_cast<unsigned>(total), 256, 0, s>>>(b);
    return hipGetLastError();
}
template <int ET, bool PAIR>
hipError_t tiled(const FfnProduct* p, int n, int tile, hipStream_t s) {
    if (tile == 256) return run<ET, 256, 2, 1, PAIR>(p, n, s);
    if (tile == 128) return run<ET, 128, 2, 1, PAIR>(p, n, s);
    if constexpr (ET == kBf16)
        if (p[0].segments > 1) return run<ET, 64, 3, 3, PAIR>(p, n, s);
    return run<ET, 64, 4, 1, PAIR>(p, n, s);
}

}  // namespace

// 8-bit operands come as a pair only (the host has no other call)
hipError_t launch_ffn_pair(const FfnProduct& p, int tile, hipStream_t s) {
    if (p.type == kE4m3) return tiled<kE4m3, true>(&p, 1, tile, s);
    return p.type == kBf16 ? tiled<kBf16, true>(&p, 1, tile, s) : tiled<kF16, true>(&p, 1, tile, s);
}
hipError_t launch_ffn_products(const FfnProduct (&p)[2], int tile, hipStream_t s) {
    return p[0].type == kBf16 ? tiled<kBf16, false>(p, 2, tile, s) : tiled<kF16, false>(p, 2, tile, s);
}

}  // namespace sdm_delta
