// The gated linear recurrence (sdm_glr.h), forward, backward and recurrent form, for gfx950.
//
//     h_t = a_t h_{t-1} + x_t,  a_t = exp(g_t);   y_t = h_t act(z_t)
//
// What bounds it is memory: x, g and z are read and y written once. A stretch of tokens maps the state that enters it as
// h -> A h + H, and two stretches after one another as A = A2 A1, H = A2 H1 + H2 (A with its exponent apart: where gates grow and
// fall it may leave float32 though no state does). A workgroup owns 64 channels (a lane
// each) of one run and walks it in tiles of 128 tokens: each of 8 wavefronts holds 16 of them in registers, finds its (A,
// H), and after one barrier each composes the maps before it, in order, and runs its own tokens from the state that enters.
// The next tile's loads are in flight meanwhile. The gradient walks the tiles from the last to the first: the states come
// from the tile's mark and the same maps, and D's recurrence, e -> a_t (u_t + e) from right to left, has the same A.
//
// Where 64 channels of a run give too few workgroups, or one run is much longer than the others, the forward takes tiles from
// one queue instead (glr_chain below): still one pass. The gradient cuts runs into parts there: a first kernel finds each part's
// map, which reads dy, z and g once more. It walks its part away from the end at which the second kernel starts, so that what
// it read last is what is wanted first and may still be in the last-level cache.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

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

// The rows of a run, one token after the other; which token is the same for the whole wavefront.
template <class T>
struct Rows {
    T* p;
    int64_t step;
};
template <class T>
__device__ __forceinline__ Rows<T> rows_of(const sdm_seq_t& s, const Run& r) {
    return Rows<T>{static_cast<T*>(s.data) + r.row * s.batch + r.start * s.token, s.token};
}
// A stretch's A, m 2^x: a product of decays that grow and fall may leave float32 where no state does. m is in [1, 2), so
// that 2^x h stays below the product and rounds only where that does, or 0 with x 0.
struct Decay {
    float m;
    int x;
};
constexpr int kFar = 1 << 20;       // exponents past it mean the same
__device__ __forceinline__ Decay decay(float m, int x) {
    x = min(max(x + __builtin_amdgcn_frexp_expf(m) - 1, -kFar), kFar);
    return Decay{2.f * __builtin_amdgcn_frexp_mantf(m), m == 0.f ? 0 : x};
}
// A h + H; from no state nothing comes, also where A has left float32.
__device__ __forceinline__ float enter(const Decay& A, float H, float h) { return h == 0.f ? H : __builtin_fmaf(A.m, __builtin_amdgcn_ldexpf(h, A.x), H); }
// The product of a wavefront's decays, from their plain product and the largest. Where none is above 1 and the product is far
// from float32's smallest, no product on the way has lost anything; elsewhere it is made again, with its exponent apart.
__device__ __forceinline__ Decay product(const float (&e)[KT], float plain, float top) {
    int x = 0;
    if (__builtin_expect(!__all(top <= 1.f && plain >= 0x1p-100f), 0)) {
        plain = 1.f;
#pragma unroll
        for (int k = 0; k < KT; ++k) {
            plain *= e[k];
            x += __builtin_amdgcn_frexp_expf(plain);
            plain = __builtin_amdgcn_frexp_mantf(plain);
        }
    }
    return decay(plain, x);
}
// A map in LDS: m, H, x
__device__ __forceinline__ void keep(float (&ex)[3][64], int lane, const Decay& A, float H) {
    ex[0][lane] = A.m;
    ex[1][lane] = H;
    ex[2][lane] = __int_as_float(A.x);
}
__device__ __forceinline__ Decay kept(const float (&ex)[3][64], int lane) { return Decay{ex[0][lane], __float_as_int(ex[2][lane])}; }

// A lane's element of a row: the row's address is the wavefront's, the byte offset the lane's.
template <class T>
__device__ __forceinline__ T get(const T* row, uint32_t off) {
    return *reinterpret_cast<const T*>(reinterpret_cast<const char*>(row) + off);
}
template <class T>
__device__ __forceinline__ void put(T* row, uint32_t off, float v) {
    *reinterpret_cast<T*>(reinterpret_cast<char*>(row) + off) = static_cast<T>(v);
}

// A first token of which the compiler does not know that it is zero: else it makes the multiples of every stride before the
// loop, more than the scalar registers hold, and reads them back from lanes of vector registers (4 x 4096 tokens of 4096
// channels in 150 us instead of 127).
__device__ __forceinline__ int unknown(int t) {
    asm volatile("" : "+s"(t));
    return t;
}

// The wavefront's KT tokens from t: all of them in the run, or read from inside it whatever t is. (One form for both would
// have the compiler merge them and take an address register for each load.)
template <class T>
__device__ __forceinline__ void fetch(std::true_type, T (&o)[KT], const Rows<T>& s, int t, int, uint32_t c) {
    const T* p = s.p + t * s.step;
#pragma unroll
    for (int i = 0; i < KT; ++i, p += s.step) o[i] = get(p, c * static_cast<uint32_t>(sizeof(T)));
}
template <class T>
__device__ __forceinline__ void fetch(std::false_type, T (&o)[KT], const Rows<T>& s, int t, int len, uint32_t c) {
#pragma unroll
    for (int i = 0; i < KT; ++i) o[i] = get(s.p + min(t + i, len - 1) * s.step, c * static_cast<uint32_t>(sizeof(T)));
}

// The map of D's recurrence, from right to left, over each part of a run.
template <int DT, int GT, int ACT>
__global__ __launch_bounds__(kGlrThreads) void glr_parts(const sdm_glr_args_t a, const int cblocks, const int segs, float* __restrict__ part) {
    using T = elem_t<DT>;
    using G = elem_t<GT>;
    constexpr bool Z = ACT != SDM_ACT_NONE;
    __shared__ float ex[NW][3][64];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int cb = blockIdx.x % cblocks, rs = blockIdx.x / cblocks, seg = rs % segs, run = rs / segs;
    const Run r = run_of(a, run);
    const int D = static_cast<int>(a.D), c = cb * 64 + lane, cc = min(c, D - 1);
    const int seglen = ((r.len + segs - 1) / segs + TILE - 1) / TILE * TILE;
    const int64_t s0 = static_cast<int64_t>(seg) * seglen;
    if (s0 >= r.len) return;                                        // never asked for
    const int t0 = static_cast<int>(s0), t1 = min(r.len, t0 + seglen), each = seglen / NW;     // a multiple of KT
    const int lo = t0 + w * each, hi = min(t1, lo + each);
    Decay A{1.f, 0};
    float H = 0.f;
    T dy[KT], z[KT];
    G g[KT];
    const Rows<T> dys = rows_of<T>(a.dy, r), zs = rows_of<T>(a.z, r);
    const Rows<G> gs = rows_of<G>(a.g, r);
    const int n = hi > lo ? (hi - lo + KT - 1) / KT : 0;
    auto load = [&](auto whole, int t) __attribute__((always_inline)) {
        fetch(whole, dy, dys, t, r.len, cc);
        fetch(whole, g, gs, t, r.len, cc);
        if constexpr (Z) fetch(whole, z, zs, t, r.len, cc);
    };
    auto work = [&](auto whole, int t, int next) __attribute__((always_inline)) {
        float e[KT], u[KT];
#pragma unroll
        for (int k = 0; k < KT; ++k) {
            const bool in = whole.value || t + k < hi;
            e[k] = in ? exp_of(static_cast<float>(g[k])) : 1.f;
            u[k] = in ? static_cast<float>(dy[k]) : 0.f;
            if constexpr (Z) {
                float f, d;
                gate<DT != 0>(static_cast<float>(z[k]), ACT, f, d);
                u[k] = in ? u[k] * f : 0.f;
            }
        }
        if (next >= 0) load(std::true_type{}, next);
        float P = 1.f, top = 0.f, h = 0.f;
#pragma unroll
        for (int k = KT - 1; k >= 0; --k) {
            h = e[k] * (u[k] + h);
            P *= e[k];
            top = fmaxf(top, e[k]);
        }
        // the new stretch is to the right of those before it
        H = enter(A, H, h);
        const Decay right = product(e, P, top);
        A = decay(A.m * right.m, A.x + right.x);
    };
    // the wavefront's last block may not be whole
    const int whole = hi > lo ? (hi - lo) / KT : 0;
    if (whole > 0) load(std::true_type{}, lo);
    for (int i = 0; i < whole; ++i) work(std::true_type{}, lo + i * KT, i + 1 < whole ? lo + (i + 1) * KT : -1);
    if (n > whole) {
        load(std::false_type{}, lo + whole * KT);
        work(std::false_type{}, lo + whole * KT, -1);
    }
    keep(ex[w], lane, A, H);
    __syncthreads();
    if (w == 0 && c < D) {
        A = Decay{1.f, 0};
        H = 0.f;
#pragma unroll
        for (int i = 0; i < NW; ++i) {
            const Decay right = kept(ex[i], lane);
            H = enter(A, H, ex[i][1][lane]);
            A = decay(A.m * right.m, A.x + right.x);
        }
        float* p = part + (static_cast<int64_t>(run) * segs + seg) * 3 * a.D + c;
        p[0] = A.m;
        p[a.D] = H;
        p[2 * a.D] = __int_as_float(A.x);
    }
}

template <int DT, int GT, int ACT>
__global__ __launch_bounds__(kGlrThreads) void glr_forward(const sdm_glr_args_t a, const int cblocks, const uint64_t* __restrict__ words) {
    using T = elem_t<DT>;
    using G = elem_t<GT>;
    constexpr bool Z = ACT != SDM_ACT_NONE;
    __shared__ float ex[2][NW][3][64];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (words && words[1] == 0) return;        // the queue's
    const int cb = blockIdx.x % cblocks, run = blockIdx.x / cblocks;
    const Run r = run_of(a, run);
    const int D = static_cast<int>(a.D), c = cb * 64 + lane, cc = min(c, D - 1);
    float h0 = a.h0 ? a.h0[run * a.D + cc] : 0.f;
    T x[KT], z[KT];
    G g[KT];
    const Rows<T> xs = rows_of<T>(a.x, r), zs = rows_of<T>(a.z, r), ys = rows_of<T>(a.y, r);
    const Rows<G> gs = rows_of<G>(a.g, r);
    auto load = [&](auto whole, int t) __attribute__((always_inline)) {
        fetch(whole, x, xs, t, r.len, cc);
        fetch(whole, g, gs, t, r.len, cc);
        if constexpr (Z) fetch(whole, z, zs, t, r.len, cc);
    };
    const int end = r.len / TILE * TILE;       // of the whole tiles
    const int t0 = unknown(0);
    if (end > t0) load(std::true_type{}, t0 + w * KT);
    int buf = 0;
    auto work = [&](auto whole, int tile) __attribute__((always_inline)) {
        const int t = tile + w * KT;
        float e[KT], u[KT];
        T zz[KT];
        float A = 1.f, top = 0.f, H = 0.f;
#pragma unroll
        for (int k = 0; k < KT; ++k) {
            const bool in = whole.value || t + k < r.len;
            e[k] = in ? exp_of(static_cast<float>(g[k])) : 1.f;
            u[k] = in ? static_cast<float>(x[k]) : 0.f;
            H = __builtin_fmaf(e[k], H, u[k]);
            A *= e[k];
            top = fmaxf(top, e[k]);
            if constexpr (Z) zz[k] = z[k];
        }
        if (whole.value && tile + TILE < end) load(std::true_type{}, t + TILE);
        keep(ex[buf][w], lane, product(e, A, top), H);
        lds_barrier();      // the other buffer is written again only after the next one
        float h = h0, next = h0;
#pragma unroll
        for (int i = 0; i < NW; ++i) {
            h = i == w ? next : h;
            next = enter(kept(ex[buf][i], lane), ex[buf][i][1][lane], next);
        }
        if (w == 0 && a.marks && c < D) a.marks[(r.mark + tile / TILE) * a.D + c] = h0;
        h0 = next;
        if (c >= D) return;
        T* yp = ys.p + t * ys.step;
#pragma unroll
        for (int k = 0; k < KT; ++k, yp += ys.step) {
            h = __builtin_fmaf(e[k], h, u[k]);
            float y = h;
            if constexpr (Z) {
                float f, d;
                gate<DT != 0>(static_cast<float>(zz[k]), ACT, f, d);
                y *= f;
            }
            if (whole.value || t + k < r.len) put(yp, c * sizeof(T), y);
        }
    };
    for (int tile = t0; tile < end; tile += TILE, buf ^= 1) work(std::true_type{}, tile);
    if (end < r.len) {
        load(std::false_type{}, end + w * KT);
        work(std::false_type{}, end);
    }
    if (w == 0 && c < D && a.h_final) a.h_final[run * a.D + c] = h0;
}

// Tiles from a queue. Workgroups take tickets in order: which tile is which ticket's follows from the sizes and bounds alone, so
// who takes it does not change a bit of the result. Beside the eight wavefronts that hold the tile, a ninth takes the tickets and
// joins the tile to those before it in its run. When the eight have found the tile's map it publishes it, waits for the state
// after the last tile of the group before and for the maps of the tiles of its own group before it, composes them in
// order, publishes the state after its tile and hands the eight the one that enters. They load the next tile and find this
// one's gates meanwhile. A run's states thus pass from group to group, and maps within one. Groups are of 4 tiles, or of 8 where
// few runs and channels leave a tile little but waiting (bfloat16, groups of 2, 4 and 8: 16384 tokens of 4096 channels 150, 154
// and 162 us; 2 x 4096 of 4096 79, 81 and 85; one run of 6784 and 22 of 64, 2048 channels, 70, 70 and 71; 3 packed of 3000, 1024
// channels, 45, 42 and 43; 32768 tokens of 512 91, 65 and 59). Two workgroups a CU without loads ahead took 184 for the first.
//
// What is published goes as words of 8 bytes, a map or a state, with a bit that says that it is there, by relaxed atomics of
// device scope: a word is there or not, and needs no order with others. All words are cleared by a kernel before. No wait goes
// unended: a ticket waits for lower ones only, which running workgroups hold, each of which publishes whatever its tile is;
// after some seconds of waiting, which nothing but a fault explains, a tile goes on with NaN.
//
// One run of 16384 tokens and 4096 channels, bfloat16 with float32 g and z: 156 us, 4.3 TB/s (walking it in four parts, whose
// maps a kernel before has to find: 215). A tile takes its workgroup 4.7 us, of which the exponentials and the last walk are
// half and the join the rest; the loads are hidden.
constexpr int kGroup = 8;       // at the most
constexpr int kPolls = 1 << 22;

struct Ticket {
    int64_t row, start, mark;       // b, the run's first token, the tile's row of marks
    int run, tile, len, cb;         // the run and its length, the tile's number in it, the block of channels
    int state;                      // 0: no more; 1: a row of marks that has no tile; 2: a tile
};

// A map's word: a bit that says that it is there, 31 for A and 32 for H. Of A in [2^-126, 2) or zero, which is any product of
// decays but the smallest, they are its own bits, the first of which is clear. Where it is set, 10 of the others are an exponent
// and 20 a fraction rounded to 2^-21: what a state brings through a tile that all but forgets it, or multiplies it. Below 2^-511
// no float32 leaves anything, from 2^511 on every one becomes infinite; where A itself is not finite, H is not either.
__device__ __forceinline__ uint64_t map_word(const Decay& A, float H) {
    const bool there = A.m < 2.f;
    const int x = there ? min(A.x, 511) : 511;
    uint32_t c = __float_as_uint(__builtin_amdgcn_ldexpf(A.m, A.x));
    if (x > 0 || x < -126)
        c = x < -511 ? 0u : 0x40000000u + (static_cast<uint32_t>(x + 512) << 20) + min(((__float_as_uint(there ? A.m : 1.f) + 4u) >> 3) - (0x3f800000u >> 3), x == 511 ? 0u : 0x100000u);
    return static_cast<uint64_t>(c | 0x80000000u) << 32 | __float_as_uint(H);
}
__device__ __forceinline__ float enter(uint64_t word, float h) {
    const uint32_t c = static_cast<uint32_t>(word >> 32);
    const bool far = c >> 30 & 1;
    const Decay A{__uint_as_float(far ? 0x3f800000u | (c & 0xfffffu) << 3 : c & 0x7fffffffu), far ? static_cast<int>(c >> 20 & 0x3ff) - 512 : 0};
    return enter(A, __uint_as_float(static_cast<uint32_t>(word)), h);
}
__device__ __forceinline__ uint64_t state_word(float h) { return uint64_t(1) << 63 | __float_as_uint(h); }
__device__ __forceinline__ void publish(uint64_t* p, uint64_t v) { __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }
__device__ __forceinline__ uint64_t look(const uint64_t* p) { return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }

// The ticket's tile, found by one wavefront.
__device__ __forceinline__ Ticket ticket_of(const sdm_glr_args_t& a, int64_t id, int64_t rows, int cblocks) {
    Ticket t{};
    if (id >= rows * cblocks) return t;
    const int64_t r = id / cblocks;
    t.cb = static_cast<int>(id % cblocks);
    t.state = 2;
    if (a.cu_seqlens == nullptr) {
        // all rows' first tiles, then all second ones
        t.run = static_cast<int>(r % a.nseq);
        t.tile = static_cast<int>(r / a.nseq);
        const Run run = run_of(a, t.run);
        t.row = run.row;
        t.len = run.len;
        t.mark = run.mark + t.tile;
        return t;
    }
    // the last run whose first row of marks is not past r: 64 of them at a time
    const int T = static_cast<int>(a.T), lane = threadIdx.x & 63;
    int lo = 0, n = static_cast<int>(a.nseq);
    while (n > 1) {
        const int step = (n + 63) / 64, i = lo + min(lane * step, n - 1);
        const bool in = lane * step < n && min(max(a.cu_seqlens[i], 0), T) / TILE + i <= r;
        const int k = max(static_cast<int>(__popcll(__ballot(in))) - 1, 0), at = min(k * step, n - 1);
        n = min(step, n - at);
        lo += at;
    }
    const Run run = run_of(a, lo);
    const int64_t tile = r - run.mark;
    t.run = lo;
    t.start = run.start;
    t.len = run.len;
    t.mark = r;
    t.tile = static_cast<int>(max(tile, int64_t(0)));
    if (tile < 0 || tile * TILE >= run.len) t.state = 1;
    return t;
}

template <int DT, int GT, int ACT>
__global__ __launch_bounds__(kGlrChainThreads) void glr_chain(const sdm_glr_args_t a, const int cblocks, const int64_t rows, const int groups, uint64_t* __restrict__ words) {
    using T = elem_t<DT>;
    using G = elem_t<GT>;
    constexpr bool Z = ACT != SDM_ACT_NONE;
    __shared__ float ex[NW][3][64], entering[64];
    __shared__ int tickets[2][sizeof(Ticket) / 4];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), D = static_cast<int>(a.D);
    // the first words: the queue's counter, whether runs are walked; then, of each tile, 64 maps and 64 states
    if (words[1] != 0) return;
    unsigned long long* counter = reinterpret_cast<unsigned long long*>(words);
    auto words_of = [&](int64_t mark, int cb) { return words + 64 + (mark * cblocks + cb) * 128 + lane; };
    auto take = [&](int slot) {
        unsigned long long id = 0;
        if (lane == 0) id = __hip_atomic_fetch_add(counter, 1ull, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        id = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(id)) | static_cast<uint64_t>(__builtin_amdgcn_readfirstlane(static_cast<uint32_t>(id >> 32))) << 32;
        const Ticket t = ticket_of(a, static_cast<int64_t>(id), rows, cblocks);
        if (lane == 0) __builtin_memcpy(tickets[slot], &t, sizeof(t));
    };
    // a ticket from LDS, the same for the whole wavefront
    auto ticket = [&](int slot) {
        int of[sizeof(Ticket) / 4];
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(Ticket) / 4); ++i) of[i] = __builtin_amdgcn_readfirstlane(tickets[slot][i]);
        Ticket t;
        __builtin_memcpy(&t, of, sizeof(t));
        return t;
    };
    // runs without tokens have no tile
    for (int64_t i = blockIdx.x; i < a.nseq && a.cu_seqlens && a.h_final; i += gridDim.x)
        if (run_of(a, static_cast<int>(i)).len == 0)
            for (int c = threadIdx.x; c < D; c += kGlrChainThreads) a.h_final[i * D + c] = a.h0 ? a.h0[i * D + c] : 0.f;

    if (w == NW) {
        take(0);
        lds_barrier();                                          // the first ticket
        for (int slot = 0;; slot ^= 1) {
            const Ticket t = ticket(slot);
            if (t.state == 0) break;
            const int c = t.cb * 64 + lane, cc = min(c, D - 1);
            const int64_t at = static_cast<int64_t>(t.run) * D + cc;
            const int group = t.tile & -groups;
            float h = group == 0 && a.h0 && t.state == 2 ? a.h0[at] : 0.f;
            take(slot ^ 1);
            lds_barrier();                                      // the tile's maps, the next ticket
            Decay A{1.f, 0};
            float H = 0.f;
            if (t.state == 2) {
                // eight factors below 2
#pragma unroll
                for (int i = 0; i < NW; ++i) {
                    const Decay next = kept(ex[i], lane);
                    H = enter(next, ex[i][1][lane], H);
                    A.m *= next.m;
                    A.x += next.x;
                }
                A = decay(A.m, A.x);
            }
            uint64_t* own = words_of(t.mark, t.cb);
            publish(own, map_word(A, H));
            if (t.state == 2) {
                const int before = t.tile - group;              // tiles of the group before this one
                uint64_t m[kGroup - 1], s = state_word(h);
                // what is still missing, a bit each: the maps and, in the last one, the state; what is there is not read again
                uint32_t missing = ((1u << before) - 1) | (group ? 1u << (kGroup - 1) : 0u);
                for (int polls = 0; missing && polls < kPolls; ++polls) {
                    if (polls) __builtin_amdgcn_s_sleep(1);
                    if (missing >> (kGroup - 1)) s = look(words_of(t.mark - before - 1, t.cb) + 64);
#pragma unroll
                    for (int i = 0; i < kGroup - 1; ++i)
                        if (missing >> i & 1) m[i] = look(words_of(t.mark - before + i, t.cb));
                    if (missing >> (kGroup - 1) && __all(s >> 63)) missing &= (1u << (kGroup - 1)) - 1;
#pragma unroll
                    for (int i = 0; i < kGroup - 1; ++i)
                        if (missing >> i & 1 && __all(m[i] >> 63)) missing &= ~(1u << i);
                }
                h = __uint_as_float(static_cast<uint32_t>(s));
#pragma unroll
                for (int i = 0; i < kGroup - 1; ++i)
                    if (i < before) h = enter(m[i], h);
                if (missing) h = __uint_as_float(0x7fc00000u);
            }
            const float after = enter(A, H, h);
            publish(own + 64, state_word(after));
            entering[lane] = h;
            lds_barrier();                                      // the state that enters
            lds_barrier();                                      // it and the maps have been read
            if (t.state == 2 && c < D) {
                if (a.marks) a.marks[t.mark * D + c] = h;
                if (a.h_final && (t.tile + 1) * static_cast<int64_t>(TILE) >= t.len) a.h_final[at] = after;
            }
        }
        return;
    }

    T x[KT], z[KT];
    G g[KT];
    auto whole_tile = [](const Ticket& t) { return t.state == 2 && (t.tile + 1) * static_cast<int64_t>(TILE) <= t.len; };
    auto load = [&](auto whole, const Ticket& t) __attribute__((always_inline)) {
        Run r;
        r.row = t.row;
        r.start = t.start;
        const uint32_t cc = min(t.cb * 64 + lane, D - 1);
        const int first = t.tile * TILE + w * KT;
        fetch(whole, x, rows_of<T>(a.x, r), first, t.len, cc);
        fetch(whole, g, rows_of<G>(a.g, r), first, t.len, cc);
        if constexpr (Z) fetch(whole, z, rows_of<T>(a.z, r), first, t.len, cc);
    };
    auto work = [&](auto whole, const Ticket& t, int slot) __attribute__((always_inline)) {
        const int first = t.tile * TILE + w * KT, c = t.cb * 64 + lane;
        float e[KT], u[KT], f[KT], A = 1.f, top = 0.f, H = 0.f;
        T zz[KT];
#pragma unroll
        for (int k = 0; k < KT; ++k) {
            const bool in = whole.value || first + k < t.len;
            e[k] = in ? exp_of(static_cast<float>(g[k])) : 1.f;
            u[k] = in ? static_cast<float>(x[k]) : 0.f;
            H = __builtin_fmaf(e[k], H, u[k]);
            A *= e[k];
            top = fmaxf(top, e[k]);
            if constexpr (Z) zz[k] = z[k];
        }
        keep(ex[w], lane, product(e, A, top), H);
        lds_barrier();
        const Ticket next = ticket(slot ^ 1);
        if (whole_tile(next)) load(std::true_type{}, next);
        // the gates, while the ninth waits; not to be moved behind the barrier
        if constexpr (Z) {
#pragma unroll
            for (int k = 0; k < KT; ++k) {
                float d;
                gate<DT != 0>(static_cast<float>(zz[k]), ACT, f[k], d);
                asm volatile("" : "+v"(f[k]));
            }
        }
        lds_barrier();
        float h = entering[lane];
#pragma unroll
        for (int i = 0; i < NW - 1; ++i)
            if (i < w) h = enter(kept(ex[i], lane), ex[i][1][lane], h);
        lds_barrier();      // before the next tile's maps
        if (c >= D) return;
        Run r;
        r.row = t.row;
        r.start = t.start;
        const Rows<T> ys = rows_of<T>(a.y, r);
        T* yp = ys.p + first * ys.step;
#pragma unroll
        for (int k = 0; k < KT; ++k, yp += ys.step) {
            h = __builtin_fmaf(e[k], h, u[k]);
            if (whole.value || first + k < t.len) put(yp, c * sizeof(T), Z ? h * f[k] : h);
        }
    };
    lds_barrier();                                              // the first ticket
    {
        const Ticket t = ticket(0);
        if (whole_tile(t)) load(std::true_type{}, t);
    }
    for (int slot = 0;; slot ^= 1) {
        const Ticket t = ticket(slot);
        if (t.state == 0) break;
        if (t.state == 1) {
            lds_barrier();
            const Ticket next = ticket(slot ^ 1);
            if (whole_tile(next)) load(std::true_type{}, next);
            lds_barrier();
            lds_barrier();
        } else if (whole_tile(t)) {
            work(std::true_type{}, t, slot);
        } else {
            load(std::false_type{}, t);
            work(std::false_type{}, t, slot);
        }
    }
}

// Clears the words, 16 bytes a thread, and for packed runs decides between the queue and walking (glr_walks), since only here
// their lengths are known.
__global__ __launch_bounds__(256) void glr_clear(const sdm_glr_args_t a, const int cblocks, const int64_t rows, u32x4* __restrict__ p, const int64_t n) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    uint32_t walk = 0;
    if (blockIdx.x == 0 && a.cu_seqlens) {
        __shared__ int longest;
        if (threadIdx.x == 0) longest = 0;
        __syncthreads();
        int l = 0;
#pragma unroll 8
        for (int64_t r = threadIdx.x; r < a.nseq; r += 256) l = max(l, run_of(a, static_cast<int>(r)).len);
        atomicMax(&longest, l);
        __syncthreads();
        walk = glr_walks((longest + TILE - 1) / TILE, rows * cblocks);
    }
    if (i < n) p[i] = u32x4{0u, 0u, i == 0 ? walk : 0u, 0u};
}

template <int DT, int GT, int ACT>
__global__ __launch_bounds__(kGlrThreads) void glr_backward(const sdm_glr_args_t a, const int cblocks, const int segs, const float* __restrict__ part) {
    using T = elem_t<DT>;
    using G = elem_t<GT>;
    constexpr bool Z = ACT != SDM_ACT_NONE;
    __shared__ float ex[2][NW][3][64], ends[2][NW][64];
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
    const Rows<T> xs = rows_of<T>(a.x, r), zs = rows_of<T>(a.z, r), dys = rows_of<T>(a.dy, r), dxs = rows_of<T>(a.dx, r), dzs = rows_of<T>(a.dz, r);
    const Rows<G> gs = rows_of<G>(a.g, r), dgs = rows_of<G>(a.dg, r);
    auto load = [&](auto whole, int tile) __attribute__((always_inline)) {
        const int t = tile + w * KT;
        fetch(whole, x, xs, t, r.len, cc);
        fetch(whole, g, gs, t, r.len, cc);
        fetch(whole, dy, dys, t, r.len, cc);
        if constexpr (Z) fetch(whole, z, zs, t, r.len, cc);
        m = a.marks[(r.mark + tile / TILE) * a.D + cc];
    };
    const int end = t0 + (t1 - t0) / TILE * TILE;       // of the whole tiles
    if (end < t1)
        load(std::false_type{}, end);
    else
        load(std::true_type{}, end - TILE);
    const int used = (r.len - 1) / seglen;      // the last part that has tokens
    for (int s = used; s > seg; --s) {
        const float* p = part + (static_cast<int64_t>(run) * segs + s) * 3 * a.D + cc;
        e0 = enter(Decay{p[0], __float_as_int(p[2 * a.D])}, p[a.D], e0);
    }
    int buf = 0;
    auto work = [&](auto whole, int tile) __attribute__((always_inline)) {
        const int t = tile + w * KT;
        float e[KT], u[KT], f[KT], v[KT], df[KT];     // a, x, dy act(z), and dy act'(z)
        float A = 1.f, top = 0.f, H = 0.f, E = 0.f;
#pragma unroll
        for (int k = 0; k < KT; ++k) {
            const bool in = whole.value || t + k < t1;
            e[k] = in ? exp_of(static_cast<float>(g[k])) : 1.f;
            u[k] = in ? static_cast<float>(x[k]) : 0.f;
            v[k] = in ? static_cast<float>(dy[k]) : 0.f;
            f[k] = v[k];
            if constexpr (Z) {
                float q, d;
                gate<DT != 0>(static_cast<float>(z[k]), ACT, q, d);
                f[k] = in ? v[k] * q : 0.f;
                df[k] = v[k] * d;
            }
            H = __builtin_fmaf(e[k], H, u[k]);
            A *= e[k];
            top = fmaxf(top, e[k]);
        }
#pragma unroll
        for (int k = KT - 1; k >= 0; --k) E = e[k] * (f[k] + E);
        float h = m;
        if (tile > t0) load(std::true_type{}, tile - TILE);
        keep(ex[buf][w], lane, product(e, A, top), H);
        ends[buf][w][lane] = E;
        lds_barrier();      // the other buffer is written again only after the next one
#pragma unroll
        for (int i = 0; i < NW - 1; ++i)
            if (i < w) h = enter(kept(ex[buf][i], lane), ex[buf][i][1][lane], h);
        float q = e0, next = e0;
#pragma unroll
        for (int i = NW - 1; i >= 0; --i) {
            q = i == w ? next : q;
            next = enter(kept(ex[buf][i], lane), ends[buf][i][lane], next);
        }
        e0 = next;
        if (c >= D) return;
        float met[KT];
#pragma unroll
        for (int k = 0; k < KT; ++k) {
            met[k] = h;
            h = __builtin_fmaf(e[k], h, u[k]);
        }
        T *dxp = dxs.p + (t + KT - 1) * dxs.step, *dzp = dzs.p + (t + KT - 1) * dzs.step;
        G* dgp = dgs.p + (t + KT - 1) * dgs.step;
#pragma unroll
        for (int k = KT - 1; k >= 0; --k, dxp -= dxs.step, dgp -= dgs.step, dzp -= dzs.step) {
            const float d = f[k] + q;
            q = e[k] * d;
            if (whole.value || t + k < t1) {
                put(dxp, c * sizeof(T), d);
                put(dgp, c * sizeof(G), q * met[k]);
                if constexpr (Z) put(dzp, c * sizeof(T), df[k] * __builtin_fmaf(e[k], met[k], u[k]));
            }
        }
    };
    if (end < t1) {
        work(std::false_type{}, end);
        buf ^= 1;
    }
    for (int tile = end - TILE; tile >= t0; tile -= TILE, buf ^= 1) work(std::true_type{}, tile);
    if (seg == 0 && w == 0 && c < D && a.dh0) a.dh0[run * a.D + c] = e0;
}

// A thread has one channel of one stream.
template <int DT, int GT, int ACT>
__global__ __launch_bounds__(kGlrStepThreads) void glr_step(const sdm_glr_step_args_t a, const int cblocks) {
    using T = elem_t<DT>;
    using G = elem_t<GT>;
    constexpr bool Z = ACT != SDM_ACT_NONE;
    const int64_t b = blockIdx.x / cblocks;
    const int c = blockIdx.x % cblocks * kGlrStepThreads + threadIdx.x;
    if (c >= a.D) return;
    const int64_t slot = a.slots ? a.slots[b] : b;
    const T *x = static_cast<const T*>(a.x.data) + b * a.x.batch + c, *z = Z ? static_cast<const T*>(a.z.data) + b * a.z.batch + c : nullptr;
    const G* g = static_cast<const G*>(a.g.data) + b * a.g.batch + c;
    T* y = static_cast<T*>(a.y.data) + b * a.y.batch + c;
    if (slot < 0 || slot >= a.pool) {
        for (int64_t t = 0; t < a.T; ++t) y[t * a.y.token] = static_cast<T>(0.f);
        return;
    }
    float h = a.state[slot * a.D + c];
    for (int64_t t = 0; t < a.T; ++t) {
        h = __builtin_fmaf(exp_of(static_cast<float>(g[t * a.g.token])), h, static_cast<float>(x[t * a.x.token]));
        float f = 1.f, d;
        if constexpr (Z) gate<DT != 0>(static_cast<float>(z[t * a.z.token]), ACT, f, d);
        y[t * a.y.token] = static_cast<T>(h * f);
    }
    a.state[slot * a.D + c] = h;
}

template <int DT, int GT, int ACT>
hipError_t forward_of(const sdm_glr_args_t& a, const GlrPlan& p, void* ws, hipStream_t s) {
    if (p.rows) {
        const int64_t n = glr_chain_words(p) / 2;
        glr_clear<<<static_cast<unsigned>((n + 255) / 256), 256, 0, s>>>(a, p.cblocks, p.rows, static_cast<u32x4*>(ws), n);
        const int64_t tickets = p.rows * p.cblocks;
        glr_chain<DT, GT, ACT><<<static_cast<unsigned>(tickets < kGlrChainGroups ? tickets : kGlrChainGroups), kGlrChainThreads, 0, s>>>(
            a, p.cblocks, p.rows, a.nseq * p.cblocks <= 8 ? 8 : 4, static_cast<uint64_t*>(ws));
    }
    if (!p.rows || a.cu_seqlens)
        glr_forward<DT, GT, ACT><<<static_cast<unsigned>(a.nseq * p.cblocks), kGlrThreads, 0, s>>>(
            a, p.cblocks, p.rows ? static_cast<const uint64_t*>(ws) : nullptr);
    return hipGetLastError();
}
template <int DT, int GT, int ACT>
hipError_t backward_of(const sdm_glr_args_t& a, const GlrPlan& p, void* ws, hipStream_t s) {
    const unsigned grid = static_cast<unsigned>(a.nseq * p.segs * p.cblocks);
    float* part = static_cast<float*>(ws);
    if (p.segs > 1) glr_parts<DT, GT, ACT><<<grid, kGlrThreads, 0, s>>>(a, p.cblocks, p.segs, part);
    glr_backward<DT, GT, ACT><<<grid, kGlrThreads, 0, s>>>(a, p.cblocks, p.segs, part);
    return hipGetLastError();
}
template <int DT, int GT, int ACT>
hipError_t step_of(const sdm_glr_step_args_t& a, hipStream_t s) {
    const int cblocks = static_cast<int>((a.D + kGlrStepThreads - 1) / kGlrStepThreads);
    glr_step<DT, GT, ACT><<<static_cast<unsigned>(a.B * cblocks), kGlrStepThreads, 0, s>>>(a, cblocks);
    return hipGetLastError();
}

// gtype is dtype or float32 (the host checks)
#define SDM_GLR_ACTS(F, DT, GT, ...)                                                                            \
    return a.act == SDM_ACT_NONE      ? F<DT, GT, SDM_ACT_NONE>(__VA_ARGS__)                                    \
           : a.act == SDM_ACT_SIGMOID ? F<DT, GT, SDM_ACT_SIGMOID>(__VA_ARGS__)                                 \
                                      : F<DT, GT, SDM_ACT_SILU>(__VA_ARGS__);
#define SDM_GLR_TYPES(F, ...)                                                                                   \
    if (a.dtype == SDM_F32) SDM_GLR_ACTS(F, 0, 0, __VA_ARGS__)                                                  \
    if (a.dtype == SDM_BF16 && a.gtype == SDM_F32) SDM_GLR_ACTS(F, 1, 0, __VA_ARGS__)                           \
    if (a.dtype == SDM_BF16) SDM_GLR_ACTS(F, 1, 1, __VA_ARGS__)                                                 \
    if (a.gtype == SDM_F32) SDM_GLR_ACTS(F, 2, 0, __VA_ARGS__)                                                  \
    SDM_GLR_ACTS(F, 2, 2, __VA_ARGS__)

}  // namespace

hipError_t launch_glr_forward(const sdm_glr_args_t& a, const GlrPlan& p, void* ws, hipStream_t s) { SDM_GLR_TYPES(forward_of, a, p, ws, s) }
hipError_t launch_glr_backward(const sdm_glr_args_t& a, const GlrPlan& p, void* ws, hipStream_t s) { SDM_GLR_TYPES(backward_of, a, p, ws, s) }
hipError_t launch_glr_step(const sdm_glr_step_args_t& a, hipStream_t s) { SDM_GLR_TYPES(step_of, a, s) }

}  // namespace sdm_delta
