// Products of the gated feed-forward on the matrix cores (sdm_ffn.h), for gfx950: C = A B^T from rows of A and B, and, as a
// pair, h = act(A Bg^T) * (A Bu^T) with both products' tiles in one wavefront's registers.
//
// Bounded by the matrix cores where M, N and K are large; a tile's operands go through LDS. All element types are laid out
// alike, by bytes: a step takes 128 bytes of each row, of which a lane holds 32 of row l % 32 for each half of the step
// (lanes 0 .. 31 the first 32 bytes of 64, lanes 32 .. 63 the other), two 16-byte pieces. Which element of a row meets which
// place of the instruction's summed axis does not matter as long as A and B agree, so the same pieces feed two
// v_mfma_f32_32x32x16 of 16-bit elements or one v_mfma_f32_32x32x64 of 8-bit ones, 64 clocks either way. Eight float32 are
// split into bfloat16 parts on their way from LDS and take six v_mfma_f32_32x32x16, 192 clocks, where float32's own matrix
// instructions would take 512; the vector instructions of the split run beside another wavefront's products.
//
// 8-bit products: the instruction aligns 8 adjacent elements' products and cuts each off below 2^-13 of the largest (measured;
// the groups' sums have float32's bits). 16-bit instructions would not, at half the rate; for operands rounded to 2^-4 and a
// result of 16 bits the full rate is taken.
//
// Memory to LDS by buffer_load_dwordx4 ... lds, no registers between: 16 bytes of a lane go to 16 consecutive bytes a lane,
// so the order that keeps reads off one another's banks is made by the choice of each lane's source: piece c of row r is at
// place c ^ (r / 2 % 8). A 16-byte read serves 16 lanes at once from 64 banks, two rows' worth, and not 16 neighbouring lanes:
// with c ^ (r % 8) half of all LDS cycles were conflicts.
//
// 8192 rows of 4096 to 8192: 8 bits 505 us, 2.18 PFLOP/s (the library's product of 8192^3 2.72); bfloat16 as a pair with g and u
// kept 905 us, 1.21, and the gradient's two products 1671 us, 1.32 (1.43). The matrix cores are busy 55, 70 and 78% of the cycles
// (counters); loads alone take 88% of the time and products alone 63% (timed apart): what they share is LDS and the power.
// Rows past M or N and pieces past the row's end read as zero by the buffer's bounds.
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

// Eight float32 in three bfloat16 parts each: x = h + m + l with h = bf16(x), m = bf16(x - h), l = bf16(x - h - m), every
// difference exact: 24 bits (from 2^-110 on; below, the multiples of bfloat16's smallest step, 2^-133). Products whose parts' numbers add up to 2 or less are kept, smallest first; what is left out, m l
// twice and l l, is below 2^-24 of the product (it comes near for 1 + 2^-8 - 2^-17 squared).
struct Parts {
    bf16x8 p[3];
};
__device__ __forceinline__ Parts split(const Piece& a) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    u32x4 w[3];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float x = __uint_as_float(a.w[i / 2][i % 2 * 2]), y = __uint_as_float(a.w[i / 2][i % 2 * 2 + 1]);
#pragma unroll
        for (int n = 0; n < 3; ++n) {
            const f32x2 v = {x, y};
            const uint32_t b = __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
            w[n][i] = b;
            x -= __uint_as_float(b << 16);
            y -= __uint_as_float(b & 0xffff0000u);
        }
    }
    Parts o;
#pragma unroll
    for (int n = 0; n < 3; ++n) o.p[n] = __builtin_bit_cast(bf16x8, w[n]);
    return o;
}
__device__ __forceinline__ void mma(f32x16& acc, const Parts& a, const Parts& b) {
#pragma unroll
    for (int order = 2; order >= 0; --order)
#pragma unroll
        for (int i = order; i >= 0; --i) acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.p[order - i], b.p[i], acc, 0, 0, 0);
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
// every load in flight before each read of LDS; meet() below counts them. m0 is the compiler's own and cannot be named as
// overwritten: the build refuses code where anything else uses it (_code_check.py).
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
    int tm[2], tn[2], first;       // tiles of each, in all parts; workgroups of the first
};

// Tiles of T x T (as a pair: T rows and T / 2 columns of either product); a wavefront has NM blocks of 32 rows by NN of 32
// columns, of which a pair's first half is Bg's and the second Bu's. LDS is a ring of U places, each for A's or B's rows of one
// step, A and B in turn. HALVES: two wavefronts share a part of the tile, one for each half of every step, and add up at the end: small
// tiles are there for calls with few of them, whose steps are chains of a read, a split and products that nothing else hides.
template <int T, int NM, int NN, bool HALVES> constexpr int kWaves = (T / (32 * NM)) * (T / (32 * NN)) * (HALVES ? 2 : 1);
template <int ET, int T, int NM, int NN, int U, bool HALVES, bool PAIR>
__global__ __launch_bounds__((64 * kWaves<T, NM, NN, HALVES>), (T == 256 ? 1 : 2)) void ffn_product(const Both both) {
    constexpr int WM = 32 * NM, WN = 32 * NN, WAVES = kWaves<T, NM, NN, HALVES>, ACROSS = T / WN, OWNERS = HALVES ? WAVES / 2 : WAVES;
    constexpr int LOADS = T / (8 * WAVES), PLACE = T * kStep;   // a wavefront's loads of a place, of 8 rows each; its bytes
    __shared__ __attribute__((aligned(1024))) char lds[U][PLACE];
    const int second = static_cast<int>(blockIdx.x) >= both.first ? 1 : 0;
    const FfnProduct& p = both.p[second];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    __builtin_assume(w >= 0 && w < WAVES);
    const int wm = w % OWNERS / ACROSS, wn = w % ACROSS, mine_half = w / OWNERS;
    int ti, tj;
    tile_of(static_cast<int>(blockIdx.x) - (second ? both.first : 0), both.tm[second], both.tn[second], ti, tj);
    int part = 0;
    int64_t bytes = p.bytes, begin = 0;
    if constexpr (!PAIR) {
        const int down = both.tm[second] / p.parts;
        part = ti / down;
        ti -= part * down;
        begin = part * p.part;
        bytes = min(p.part, bytes - begin);
    }
    constexpr int BR = PAIR ? T / 2 : T;        // rows of a B that the tile takes
    const int64_t m0 = static_cast<int64_t>(ti) * T, n0 = static_cast<int64_t>(tj) * BR;
    auto rows_of = [&](const FfnOperand& o, int64_t first, int64_t all, int most) {
        const int64_t n = min(all - first, static_cast<int64_t>(most));
        return Buffer{o.p + first * o.ld + begin, static_cast<uint32_t>((n - 1) * o.ld + bytes)};
    };
    const Buffer ba = rows_of(p.A, m0, p.M, T), bb = rows_of(p.B, n0, p.N, BR), bc = PAIR ? rows_of(p.B2, n0, p.N, BR) : bb;

    // Load j of wavefront w fills rows (WAVES j + w) 8 .. + 7 of a place: a lane's row and piece, and their offsets in A and B.
    const int r8 = lane >> 3, piece = (lane & 7) ^ ((w & 1) << 2 | r8 >> 1);
    uint32_t off_a[LOADS], off_b[LOADS];
#pragma unroll
    for (int j = 0; j < LOADS; ++j) {
        const int r = (j * WAVES + w) * 8 + r8;
        off_a[j] = static_cast<uint32_t>(r * p.A.ld) + piece * 16;
        if constexpr (PAIR)
            off_b[j] = static_cast<uint32_t>((r / WN * (WN / 2) + r % (WN / 2)) * (r & WN / 2 ? p.B2.ld : p.B.ld)) + piece * 16;
        else
            off_b[j] = static_cast<uint32_t>(r * p.B.ld) + piece * 16;
    }
    const uint32_t base = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) char*)&lds[0][0]));
    const int steps = static_cast<int>((bytes + kStep - 1) / kStep);
    // The next step's buffers. Past the last step they are empty, since their bounds less what is behind would wrap around:
    // every load of such a step reads nothing.
    int at = 0;
    u32x4 ra, rb, rc;
    uint32_t none;
    auto next_step = [&]() {
        const int64_t from = static_cast<int64_t>(at) * kStep;
        const bool past = at >= steps;
        auto from_here = [&](const Buffer& b) { return resource(Buffer{b.p + (past ? 0 : from), past ? 0u : b.n - static_cast<uint32_t>(from)}); };
        ra = from_here(ba);
        rb = from_here(bb);
        rc = PAIR ? from_here(bc) : rb;
        none = from + piece * 16 >= bytes ? kNowhere : 0u;       // the row has ended
        ++at;
    };
    auto load_a = [&](int place, int j) { load_lds(ra, base + place * PLACE + (j * WAVES + w) * 1024, off_a[j] | none); };
    auto load_b = [&](int place, int j) {
        load_lds(PAIR && (j * WAVES + w) * 8 & WN / 2 ? rc : rb, base + place * PLACE + (j * WAVES + w) * 1024, off_b[j] | none);
    };
    f32x16 acc[NN][NM];                         // [columns][rows]
#pragma unroll
    for (int i = 0; i < NN; ++i)
#pragma unroll
        for (int j = 0; j < NM; ++j) acc[i][j] = (f32x16){0};
    Piece fa[2][NM], fb[2][NN];
    const int lr = lane & 31, lh = lane >> 5, sw = lr >> 1 & 7;
    constexpr int READS = 2 * (NM + NN), BLOCKS = NM * NN, AHEAD = BLOCKS > 4 ? BLOCKS * 3 / 4 : BLOCKS > 1 ? BLOCKS / 2 : 1;
    // Read n of a half step, in the order in which the products want them: B's first block, A's, B's others.
    auto read = [&](int pa, int pb, int to, int half, int n) {
        const int i = n / 2, k = n % 2, c = ((half * 4 + lh * 2 + k) ^ sw) * 16;
        if (i >= 1 && i <= NM)
            fa[to][i - 1].w[k] = *reinterpret_cast<const u32x4*>(&lds[pa][(wm * WM + (i - 1) * 32 + lr) * kStep + c]);
        else
            fb[to][i ? i - NM : 0].w[k] = *reinterpret_cast<const u32x4*>(&lds[pb][(wn * WN + (i ? i - NM : 0) * 32 + lr) * kStep + c]);
    };
    // Blocks of 64 clocks of products (float32: 192) of the pieces in `slot`, with the reads of the other slot's pieces behind the
    // first of them and loads spread over all, in the order written here (the compiler would gather the products behind the
    // barrier). Loads: `a` A's, `b` B's.
    auto blocks = [&](int slot, int pa, int pb, int half, bool a, bool b, int to_a, int to_b) {
        Parts sa[NM], sb[NN];       // of float32
#pragma unroll
        for (int n = 0; n < BLOCKS; ++n) {
            constexpr int kReads = READS / AHEAD;
#pragma unroll
            for (int k = 0; k < kReads; ++k)
                if (n * kReads + k < READS) read(pa, pb, 1 - slot, half, n * kReads + k);
#pragma unroll
            for (int k = n * LOADS / BLOCKS; k < (n + 1) * LOADS / BLOCKS; ++k) {
                if (a) load_a(to_a, k);
                if (b) load_b(to_b, k);
            }
            const int i = n / NM, j = n % NM;
            if constexpr (ET == kF32) {
                if (j == 0) sb[i] = split(fb[slot][i]);
                if (i == 0) sa[j] = split(fa[slot][j]);
                mma(acc[i][j], sb[i], sa[j]);
            } else {
                mma<ET>(acc[i][j], fb[slot][i], fa[slot][j]);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    // two steps, A's and B's rows in turn
#pragma unroll
    for (int s = 0; s < (HALVES ? U / 2 : 2); ++s) {
        next_step();
#pragma unroll
        for (int j = 0; j < LOADS; ++j) load_a(2 * s, j);
#pragma unroll
        for (int j = 0; j < LOADS; ++j) load_b(2 * s + 1, j);
    }
    meet<(HALVES ? U - 2 : 2) * LOADS>();
#pragma unroll
    for (int k = 0; k < READS; ++k) read(0, 1, 0, HALVES ? mine_half : 0, k);
    if constexpr (HALVES) {
        // Between two steps the wavefronts meet: the next one has landed and is read behind this one's products, and all reads of
        // this one are back, so its places take the loads of the step U / 2 later.
        auto step = [&](int slot, int t) {
            next_step();
            meet<(U - 4) * LOADS>();
            __builtin_amdgcn_sched_barrier(0);
            const int here = t % (U / 2) * 2, next = (t + 1) % (U / 2) * 2;
            blocks(slot, next, next + 1, mine_half, true, true, here, here + 1);
        };
        for (int t = 0; t < steps; t += 2) {
            step(0, t);
            if (t + 1 < steps) step(1, t + 1);
        }
    } else {
        // A step's second half is read while its first is multiplied, and the next step's first half while the second is. Between
        // the two the wavefronts meet: the next step has landed, and all reads of this one are back. Loads never pause: A's rows
        // of the step after the next go behind the first half, where the fifth place is free, and B's behind the second, to this
        // step's place for A (LDS is full: a burst of both behind the second half takes as long as a step, and the products wait).
        static_assert(U == 5, "A's and B's rows of two steps and a half");
        int at_a = 0;       // the place of this step's A; B's is the next one
        auto after = [](int place, int n) { return place + n < U ? place + n : place + n - U; };
        for (int t = 0; t < steps; ++t) {
            next_step();
            blocks(0, at_a, after(at_a, 1), 1, true, false, after(at_a, 4), 0);
            meet<LOADS>();
            __builtin_amdgcn_sched_barrier(0);
            blocks(1, after(at_a, 2), after(at_a, 3), 0, false, true, 0, at_a);
            at_a = after(at_a, 2);
        }
    }

    // Lane l holds columns 8 (i / 4) + 4 (l / 32) + i % 4 of row l % 32 of each block. 32 rows at a time go through the
    // wavefront's own part of LDS, so that its lanes store whole stretches of a row; rows there are 4 banks apart.
    meet<0>();
    constexpr int kRow = WN * 4 + 16, kLanes = (PAIR ? WN / 2 : WN) / 4, kRows = 64 / kLanes;
    static_assert(OWNERS * 32 * kRow + (HALVES ? OWNERS * 4096 : 0) <= static_cast<int>(sizeof(lds)), "the wavefronts' rows fit");
    if constexpr (HALVES) {
        static_assert(NM == 1 && NN == 1, "one block a wavefront");
        f32x4* other = reinterpret_cast<f32x4*>(&lds[0][0] + OWNERS * 32 * kRow + w % OWNERS * 4096) + lane;
        if (mine_half) {
#pragma unroll
            for (int q = 0; q < 4; ++q) other[q * 64] = f32x4{acc[0][0][q * 4], acc[0][0][q * 4 + 1], acc[0][0][q * 4 + 2], acc[0][0][q * 4 + 3]};
        }
        meet<0>();
        if (mine_half) return;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const f32x4 x = other[q * 64];
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[0][0][q * 4 + e] += x[e];
        }
    }
    char* mine = &lds[0][0] + w * 32 * kRow;
    const int col = lane % kLanes * 4;
    const int64_t n = n0 + wn * (PAIR ? WN / 2 : WN) + col, left = p.N - n;
    Scale sg[4], su[4];
    if constexpr (ET == kE4m3) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int64_t c = min(n + e, p.N - 1);
            sg[e] = scale_of(p.sn[c]);
            su[e] = scale_of(p.sn2[c]);
        }
    }
#pragma unroll
    for (int j = 0; j < NM; ++j) {
#pragma unroll
        for (int i = 0; i < NN; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                *reinterpret_cast<f32x4*>(mine + lr * kRow + (i * 32 + q * 8 + lh * 4) * 4) =
                    f32x4{acc[i][j][q * 4], acc[i][j][q * 4 + 1], acc[i][j][q * 4 + 2], acc[i][j][q * 4 + 3]};
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
        for (int r = lane / kLanes; r < 32; r += kRows) {
            const int64_t m = m0 + wm * WM + j * 32 + r;
            const f32x4* from = reinterpret_cast<const f32x4*>(mine + r * kRow + col * 4);
            if (m >= p.M || left <= 0) continue;
            const f32x4 x = from[0];
            float g[4] = {x[0], x[1], x[2], x[3]};
            if constexpr (!PAIR) {
                // parts: no second area
                char* c = m < p.split ? p.c : p.c2;
                store4(p.otype, c, (m < p.split ? (part * p.M + m) * p.ldc : (m - p.split) * p.ldc2) + n, left, g);
            } else {
                const f32x4 y = from[WN / 8];
                float u[4] = {y[0], y[1], y[2], y[3]}, h[4];
                if constexpr (ET == kE4m3) {
                    const Scale sm = scale_of(p.sm[m]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        g[e] = scaled(g[e], sm, sg[e]);
                        u[e] = scaled(u[e], sm, su[e]);
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

template <int ET, int T, int NM, int NN, int U, bool HALVES, bool PAIR>
hipError_t run(const FfnProduct* p, int n, hipStream_t s) {
    Both b{};
    int64_t total = 0;
    for (int i = 0; i < n; ++i) {
        b.p[i] = p[i];
        b.tm[i] = static_cast<int>((p[i].M + T - 1) / T) * (PAIR ? 1 : p[i].parts);
        b.tn[i] = static_cast<int>((p[i].N + (PAIR ? T / 2 : T) - 1) / (PAIR ? T / 2 : T));
        total += static_cast<int64_t>(b.tm[i]) * b.tn[i];
        if (i == 0) b.first = static_cast<int>(total);
    }
    ffn_product<ET, T, NM, NN, U, HALVES, PAIR><<<static_cast<unsigned>(total), 64 * kWaves<T, NM, NN, HALVES>, 0, s>>>(b);
    return hipGetLastError();
}
template <int ET, bool PAIR>
hipError_t tiled(const FfnProduct* p, int n, int tile, hipStream_t s) {
    if constexpr (ET != kF32)
        if (tile == 256) return run<ET, 256, 4, 2, 5, false, PAIR>(p, n, s);
    if (tile == 128) return run<ET, 128, 2, 2, 5, false, PAIR>(p, n, s);
    return run<ET, 64, 1, 1, 8, true, PAIR>(p, n, s);
}

}  // namespace

// 8-bit operands come as a pair only, float32 ones in tiles of 128 at the most (the host has no other call)
hipError_t launch_ffn_pair(const FfnProduct& p, int tile, hipStream_t s) {
    if (p.type == kE4m3) return tiled<kE4m3, true>(&p, 1, tile, s);
    if (p.type == kF32) return tiled<kF32, true>(&p, 1, tile, s);
    return p.type == kBf16 ? tiled<kBf16, true>(&p, 1, tile, s) : tiled<kF16, true>(&p, 1, tile, s);
}
hipError_t launch_ffn_products(const FfnProduct (&p)[2], int tile, hipStream_t s) {
    if (p[0].type == kF32) return tiled<kF32, false>(p, 2, tile, s);
    return p[0].type == kBf16 ? tiled<kBf16, false>(p, 2, tile, s) : tiled<kF16, false>(p, 2, tile, s);
}

}  // namespace sdm_delta
