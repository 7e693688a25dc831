// Device pieces of the gated-delta-rule kernels: split operands, matrix-core steps, chunk geometry.
//
// Split operands. The bfloat16 matrix cores run 16 times the float32 ones' rate. A float32 x is h + m + l with
// h = bf16(x), m = bf16(x - h), l = bf16(x - h - m), each difference exact: 24 bits. A product of two such sums keeps
// the part products whose parts' numbers add up to 2 or less; what is left out is below 2^-25 of the product, so a
// product costs 6 matrix-core steps and is as exact as float32's own (a quarter of the time of a float32 matrix-core
// product). Elements that are bfloat16 to begin with are one part (3 steps against a float32 operand), float16 ones
// two. Results of 16 bits need them all too: Q S and P U can each be thousands of times their sum, the output, where a
// key overwrites what the state holds.
//
// Fragments. One matrix-core operand of v_mfma_f32_16x16x32_bf16: lane l holds row l % 16, elements
// 8 (l / 16) .. + 7 of a 32-wide block of the summed axis. Both operands have this layout, each with its summed axis
// contiguous. Results: lane l holds rows 4 (l / 16) .. + 3 of column l % 16.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "delta_types.h"
#include "gdr.h"

namespace sdm_delta {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));

template <int DT> constexpr int kParts = DT == 0 ? 3 : DT == 1 ? 1 : 2;

template <int N>
struct Frag {
    bf16x8 p[N];
};

// f as N bfloat16 parts, largest first. Two elements at a time: one conversion makes both halves of a register, a shift
// and a mask take them out again.
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
template <int N>
__device__ __forceinline__ void split2(uint32_t (&o)[N], float a, float b) {
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const f32x2 v = {a, b};
        const uint32_t w = __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
        o[n] = w;
        if (n + 1 < N) {
            a -= __uint_as_float(w << 16);
            b -= __uint_as_float(w & 0xffff0000u);
        }
    }
}
template <int N>
__device__ __forceinline__ void split8(Frag<N>& o, const float (&f)[8]) {
    u32x4 w[N];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t x[N];
        split2<N>(x, f[2 * i], f[2 * i + 1]);
#pragma unroll
        for (int n = 0; n < N; ++n) w[n][i] = x[n];
    }
#pragma unroll
    for (int n = 0; n < N; ++n) o.p[n] = __builtin_bit_cast(bf16x8, w[n]);
}
template <int N>
__device__ __forceinline__ void split4(bf16x4 (&o)[N], const f32x4& f) {
    uint32_t x[N], y[N];
    split2<N>(x, f[0], f[1]);
    split2<N>(y, f[2], f[3]);
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const u32x2 w = {x[n], y[n]};
        o[n] = __builtin_bit_cast(bf16x4, w);
    }
}

// acc += a b, the part products of order below 3, smallest first
template <int NA, int NB>
__device__ __forceinline__ void mma(f32x4& acc, const Frag<NA>& a, const Frag<NB>& b) {
#pragma unroll
    for (int s = 2; s >= 0; --s)
#pragma unroll
        for (int i = 0; i < NA; ++i)
            if (s - i >= 0 && s - i < NB) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.p[i], b.p[s - i], acc, 0, 0, 0);
}

// Always from a place inside the row (`row` itself has to be readable), zero where c is past `lim` or !ok: no branch
// around a load, so that loads stay in flight together. VEC: lim is a multiple of 8.
template <int DT, bool VEC>
__device__ __forceinline__ void load_raw(Raw<DT>& o, const elem_t<DT>* __restrict__ row, int c, int lim, bool ok) {
    const u32x4 zero = {0, 0, 0, 0};
    if constexpr (VEC) {
        ok = ok && c < lim;
        const u32x4u* p = reinterpret_cast<const u32x4u*>(row + (ok ? c : 0));
        const u32x4 x = p[0];
        o.w[0] = ok ? x : zero;
        if constexpr (DT == 0) {
            const u32x4 y = p[1];
            o.w[1] = ok ? y : zero;
        }
    } else if constexpr (DT == 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const bool in = ok && c + i < lim;
            const uint32_t x = __float_as_uint(row[in ? c + i : 0]);
            o.w[i / 4][i % 4] = in ? x : 0u;
        }
    } else {
        const uint16_t* r = reinterpret_cast<const uint16_t*>(row);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bool il = ok && c + 2 * i < lim, ih = ok && c + 2 * i + 1 < lim;
            const uint32_t lo = r[il ? c + 2 * i : 0], hi = r[ih ? c + 2 * i + 1 : 0];
            o.w[0][i] = (il ? lo : 0u) | (ih ? hi << 16 : 0u);
        }
    }
}
template <int DT>
__device__ __forceinline__ void raw_frag(Frag<kParts<DT>>& o, const Raw<DT>& r) {
    if constexpr (DT == 1) {
        o.p[0] = __builtin_bit_cast(bf16x8, r.w[0]);
    } else {
        float f[8];
        raw_floats<DT>(f, r);
        split8(o, f);
    }
}

// A fragment stored as [part][64 lanes][8]: tile t, k block kb of a matrix of `kbs` k blocks.
template <int N>
__device__ __forceinline__ uint16_t* frag_at(uint16_t* base, int t, int kb, int kbs) {
    return base + static_cast<int64_t>(t * kbs + kb) * N * 512;
}
template <int N>
__device__ __forceinline__ void load_frag(Frag<N>& o, const uint16_t* __restrict__ at) {
#pragma unroll
    for (int n = 0; n < N; ++n)
        o.p[n] = *reinterpret_cast<const bf16x8*>(at + n * 512 + (threadIdx.x & 63) * 8);
}
template <int N>
__device__ __forceinline__ void store_frag(uint16_t* at, const Frag<N>& f) {
#pragma unroll
    for (int n = 0; n < N; ++n) *reinterpret_cast<bf16x8*>(at + n * 512 + (threadIdx.x & 63) * 8) = f.p[n];
}

// A split matrix in LDS, as fragments: [part][32-wide k block][16-row tile][64 lanes][8]. A fragment's read is 1 KB in
// lane order and a transposed result tile's write 512 bytes without a gap, so neither meets a bank conflict (rows
// padded to 8 more than a multiple of 32 elements had one on every second read).
template <int N, int ROWS, int KS>
struct Tile {
    alignas(16) __bf16 v[N][KS / 32][ROWS / 16][64][8];
    // where element (row, k) lies; k a multiple of 4 (8) for 8-byte (16-byte) access
    __device__ __forceinline__ __bf16* at(int part, int row, int k) {
        return &v[part][k >> 5][row >> 4][(row & 15) + 16 * (k >> 3 & 3)][k & 7];
    }
    // the first M parts of a fragment
    template <int M>
    __device__ __forceinline__ void frag(Frag<M>& o, int row0, int k0) const {
#pragma unroll
        for (int n = 0; n < M; ++n) o.p[n] = *reinterpret_cast<const bf16x8*>(v[n][k0 >> 5][row0 >> 4][threadIdx.x & 63]);
    }
    // a result tile, transposed: its column is the row here
    __device__ __forceinline__ void put(int row0, int k0, const f32x4& d) {
        const int l = threadIdx.x & 63;
        bf16x4 s[N];
        split4<N>(s, d);
#pragma unroll
        for (int n = 0; n < N; ++n) *reinterpret_cast<bf16x4*>(at(n, row0 + (l & 15), k0 + 4 * (l >> 4))) = s[n];
    }
};

// Whether the k blocks of the triangular 64 x 64 matrices that are all zero are left out, unwritten and unread, by loops
// of their own for the wavefronts concerned: the registers of wide and float32 heads do not bear the second copy.
template <int DT, int DKP> constexpr bool kSkipZero = DKP == 64 || (DT != 0 && DKP == 128);

// All loads so far have landed. Before a loop whose loads cross its back edge: the compiler otherwise waits at the
// loop's head for the order in which the loads before the loop happen to stand, every time round.
__device__ __forceinline__ void loads_landed() { __builtin_amdgcn_s_waitcnt(0x0f70); }

// e^x in 1 ulp or two: the hardware's 2^t with t = x log2(e) as a float, times 1 + ln(2) (what t's rounding left out).
// (The library's expf is a quarter of the time of a chunk's 64 x 64 decays longer.) Below -103 it is 0, as e^x in
// float32 nearly is.
__device__ __forceinline__ float exp_of(float x) {
    const float t = x * 1.44269502f;
    const float rest = fmaf(x, 1.44269502f, -t) + x * 1.92596299e-8f;
    const float y = __builtin_amdgcn_exp2f(t);
    return fmaf(y, rest * 0.693147181f, y);
}

// One sequence: its first token, length and first chunk slot.
struct Seq {
    int32_t b, start, len, slot;
};
__device__ __forceinline__ Seq sequence(const sdm_gdr_args_t& a, int i) {
    Seq s;
    if (a.cu_seqlens) {
        const int T = static_cast<int>(a.T);
        const int lo = min(max(a.cu_seqlens[i], 0), T), hi = min(max(a.cu_seqlens[i + 1], lo), T);
        s.b = 0;
        s.start = lo;
        s.len = hi - lo;
        s.slot = lo / kChunk + i;
    } else {
        s.b = i;
        s.start = 0;
        s.len = static_cast<int>(a.T);
        s.slot = i * ((s.len + kChunk - 1) / kChunk);
    }
    return s;
}
// The sequence that owns a chunk slot and the chunk's number in it; false for a slot that none uses.
__device__ __forceinline__ bool owner(const sdm_gdr_args_t& a, int slot, int& seq, int& chunk, Seq& s) {
    if (a.cu_seqlens) {
        int lo = 0, hi = static_cast<int>(a.nseq) - 1;      // the last run whose first slot is not past this one
        const int T = static_cast<int>(a.T);
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (min(max(a.cu_seqlens[mid], 0), T) / kChunk + mid <= slot)
                lo = mid;
            else
                hi = mid - 1;
        }
        seq = lo;
    } else {
        seq = slot / ((static_cast<int>(a.T) + kChunk - 1) / kChunk);
    }
    s = sequence(a, seq);
    chunk = slot - s.slot;
    return chunk >= 0 && static_cast<int64_t>(chunk) * kChunk < s.len;
}

// The first element of a sequence's row of one head; tokens follow at r.token.
template <class T>
__device__ __forceinline__ T* rows_at(const sdm_rows_t& r, const Seq& s, int head) {
    return static_cast<T*>(r.data) + s.b * r.batch + s.start * r.token + head * r.head;
}

// Consecutive logical workgroups on one XCD (hardware deals workgroup ids round the 8 XCDs): those that share a head's
// chunks then share an L2. n logical workgroups run on a grid of 8 * ceil(n / 8); false past the last.
__device__ __forceinline__ bool on_one_xcd(int n, int& id) {
    id = static_cast<int>((blockIdx.x & 7) * (gridDim.x >> 3) + (blockIdx.x >> 3));
    return id < n;
}

}  // namespace sdm_delta
