// What the feed-forward's products read beside the inputs where they lie (sdm_ffn.h): operands laid out anew (odd
// alignments, float32 in three bfloat16 parts, and turned for the gradient's sums over rows), and dg and du, for gfx950.
//
// Bounded by memory: each value is read once and written once a part. Tiles of 64 x 64 are turned through LDS, so that both
// sides move whole lines.
//
// Parts. A float32 x is h + m + l with h = bf16(x), m = bf16(x - h), l = bf16(x - h - m), each difference exact: 24 bits. A
// value that is not finite, or rounds to infinity, is its first part alone.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "block_device.h"
#include "ffn.h"

namespace sdm_delta {
namespace {

template <int DT> struct Bits { using type = uint16_t; };
template <> struct Bits<SDM_E4M3> { using type = uint8_t; };
template <int DT> constexpr int kParts = DT == SDM_F32 ? 3 : 1;

__device__ __forceinline__ uint16_t bits(__bf16 x) { return __builtin_bit_cast(uint16_t, x); }
__device__ __forceinline__ void split(uint16_t (&o)[3], float x) {
    const __bf16 h = static_cast<__bf16>(x);
    o[0] = bits(h);
    const float m = x - static_cast<float>(h);
    const bool fine = fabsf(static_cast<float>(h)) < __uint_as_float(0x7f800000u);
    const __bf16 b = static_cast<__bf16>(m);
    o[1] = fine ? bits(b) : 0;
    o[2] = fine ? bits(static_cast<__bf16>(m - static_cast<float>(b))) : 0;
}
// A source element as the bits of its parts.
template <int DT>
__device__ __forceinline__ void parts_of(typename Bits<DT>::type (&o)[kParts<DT>], const void* src, int64_t at) {
    if constexpr (DT == SDM_F32)
        split(o, static_cast<const float*>(src)[at]);
    else
        o[0] = static_cast<const typename Bits<DT>::type*>(src)[at];
}

// Up to three operands in one launch: workgroup b belongs to the one whose stretch it lies in.
struct Three {
    FfnLay l[3];
    unsigned upto[3];
};
__device__ __forceinline__ int which(const Three& t, unsigned& b) {
    const int i = b < t.upto[0] ? 0 : b < t.upto[1] ? 1 : 2;
    b -= i ? t.upto[i - 1] : 0;
    return i;
}

// A thread has 8 columns of one row.
template <int DT>
__global__ __launch_bounds__(256) void lay_rows(const Three three) {
    using B = typename Bits<DT>::type;
    constexpr int P = kParts<DT>;
    unsigned b = blockIdx.x;
    const FfnLay& l = three.l[which(three, b)];
    const int64_t groups = l.pad / 8, id = static_cast<int64_t>(b) * 256 + threadIdx.x;
    if (id >= l.R * groups) return;
    const int64_t r = id / groups, c = id % groups * 8;
    B o[P][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        B x[P];
        parts_of<DT>(x, l.src, r * l.ld + min(c + i, l.C - 1));
#pragma unroll
        for (int p = 0; p < P; ++p) o[p][i] = c + i < l.C ? x[p] : 0;
    }
#pragma unroll
    for (int p = 0; p < P; ++p) {
        char* to = l.dst + p * l.plane + r * l.ldd + c * static_cast<int64_t>(sizeof(B));
        if constexpr (sizeof(B) == 2)
            *reinterpret_cast<u32x4*>(to) = __builtin_bit_cast(u32x4, o[p]);
        else
            *reinterpret_cast<u32x2*>(to) = __builtin_bit_cast(u32x2, o[p]);
    }
}

// 16 bytes of a turned tile's row: tile[k][c] for k = from .. from + 7
__device__ __forceinline__ u32x4 column(const uint16_t (*tile)[66], int from, int c) {
    u32x4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = tile[from + 2 * i][c] | static_cast<uint32_t>(tile[from + 2 * i + 1][c]) << 16;
    return o;
}

// Four columns of a row from c: all there, or read from inside the row and zero past its end (or for a row that is none).
template <int DT>
__device__ __forceinline__ void four(typename Bits<DT>::type (&o)[4][kParts<DT>], const void* src, int64_t row, int64_t c, int64_t n, bool in) {
    using B = typename Bits<DT>::type;
    if (c + 4 <= n) {
        if constexpr (DT == SDM_F32) {
            typedef uint32_t u32x4a __attribute__((ext_vector_type(4), aligned(4)));
            const u32x4 x = *reinterpret_cast<const u32x4a*>(static_cast<const float*>(src) + row + c);
#pragma unroll
            for (int i = 0; i < 4; ++i) split(o[i], __uint_as_float(x[i]));
        } else {
            typedef uint32_t u32x2u __attribute__((ext_vector_type(2), aligned(2)));
            const u32x2 x = *reinterpret_cast<const u32x2u*>(static_cast<const B*>(src) + row + c);
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i][0] = static_cast<B>(x[i / 2] >> (16 * (i % 2)));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int p = 0; p < kParts<DT>; ++p) o[i][p] = in ? o[i][p] : 0;
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        parts_of<DT>(o[i], src, row + min(c + i, n - 1));
#pragma unroll
        for (int p = 0; p < kParts<DT>; ++p) o[i][p] = in && c + i < n ? o[i][p] : 0;
    }
}

// dst[part][c][r]: a tile of 64 rows and 64 columns. 16-bit parts.
template <int DT>
__global__ __launch_bounds__(256) void lay_turned(const Three three) {
    constexpr int P = kParts<DT>;
    __shared__ uint16_t tile[P][64][66];
    unsigned b = blockIdx.x;
    const FfnLay& l = three.l[which(three, b)];
    const unsigned across = static_cast<unsigned>((l.C + 63) / 64);
    const int64_t r0 = static_cast<int64_t>(b / across) * 64, c0 = static_cast<int64_t>(b % across) * 64;
    uint16_t x[4][4][P];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = i * 16 + threadIdx.x / 16, c = threadIdx.x % 16 * 4;
        four<DT>(x[i], l.src, min(r0 + r, l.R - 1) * l.ld, c0 + c, l.C, r0 + r < l.R);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
            for (int k = 0; k < 4; k += 2)
                *reinterpret_cast<uint32_t*>(&tile[p][i * 16 + threadIdx.x / 16][threadIdx.x % 16 * 4 + k]) = x[i][k][p] | static_cast<uint32_t>(x[i][k + 1][p]) << 16;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int c = i * 32 + threadIdx.x / 8, r = threadIdx.x % 8 * 8;
        if (c0 + c >= l.C || r0 + r >= l.pad) continue;
#pragma unroll
        for (int p = 0; p < P; ++p)
            *reinterpret_cast<u32x4*>(l.dst + p * l.plane + (c0 + c) * l.ldd + (r0 + r) * 2) = column(tile[p], r, c);
    }
}

template <int DT>
__global__ __launch_bounds__(256) void ffn_grad(const FfnGrad a, const int across) {
    using T = elem_t<DT>;
    constexpr int P = kParts<DT>;
    __shared__ uint16_t tile[2][P][64][66];
    const int64_t m0 = static_cast<int64_t>(blockIdx.x / across) * 64, f0 = static_cast<int64_t>(blockIdx.x % across) * 64;
    const int r16 = threadIdx.x / 16, c = threadIdx.x % 16 * 4;
    float dh[4][4], g[4][4], u[4][4];
    const bool whole = f0 + c + 4 <= a.F;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t m = min(m0 + i * 16 + r16, a.M - 1);
        const T* d = static_cast<const T*>(a.dh) + m * a.ld_dh;
        const float *gr = a.gate + m * a.ld_gate, *ur = a.up + m * a.ld_up;
        if (whole) {
            typedef uint32_t u32x4a __attribute__((ext_vector_type(4), aligned(4)));
            const u32x4 x = *reinterpret_cast<const u32x4a*>(gr + f0 + c), y = *reinterpret_cast<const u32x4a*>(ur + f0 + c);
            if constexpr (DT == SDM_F32) {
                const u32x4 z = *reinterpret_cast<const u32x4a*>(d + f0 + c);
#pragma unroll
                for (int k = 0; k < 4; ++k) dh[i][k] = __uint_as_float(z[k]);
            } else {
                typedef uint32_t u32x2u __attribute__((ext_vector_type(2), aligned(2)));
                typedef T t4 __attribute__((ext_vector_type(4)));
                const u32x2 w = *reinterpret_cast<const u32x2u*>(d + f0 + c);
                const t4 z = __builtin_bit_cast(t4, w);
#pragma unroll
                for (int k = 0; k < 4; ++k) dh[i][k] = static_cast<float>(z[k]);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                g[i][k] = __uint_as_float(x[k]);
                u[i][k] = __uint_as_float(y[k]);
            }
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int64_t f = min(f0 + c + k, a.F - 1);
                dh[i][k] = static_cast<float>(d[f]);
                g[i][k] = gr[f];
                u[i][k] = ur[f];
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = i * 16 + r16;
        uint16_t x[2][4][P];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float act, d;
            gate<DT != SDM_F32>(g[i][k], a.act, act, d);
            const bool in = m0 + r < a.M && f0 + c + k < a.F;
            const float v[2] = {in ? dh[i][k] * u[i][k] * d : 0.f, in ? dh[i][k] * act : 0.f};
#pragma unroll
            for (int s = 0; s < 2; ++s)
                if constexpr (DT == SDM_F32)
                    split(x[s][k], v[s]);
                else
                    x[s][k][0] = __builtin_bit_cast(uint16_t, static_cast<T>(v[s]));
        }
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int p = 0; p < P; ++p) {
                const u32x2 o = {x[s][0][p] | static_cast<uint32_t>(x[s][1][p]) << 16, x[s][2][p] | static_cast<uint32_t>(x[s][3][p]) << 16};
                *reinterpret_cast<uint32_t*>(&tile[s][p][r][c]) = o[0];
                *reinterpret_cast<uint32_t*>(&tile[s][p][r][c + 2]) = o[1];
                // 8 values of padding at the most: a row's end is a multiple of 8 and c of 4
                if (m0 + r < a.M && f0 + c < a.Fp)
                    *reinterpret_cast<u32x2*>(a.rows + p * a.rows_plane + ((m0 + r) * 2 * a.Fp + s * a.Fp + f0 + c) * 2) = o;
            }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int f = i * 32 + threadIdx.x / 8, m = threadIdx.x % 8 * 8;
        if (f0 + f >= a.F || m0 + m >= a.Mp) continue;
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int p = 0; p < P; ++p)
                *reinterpret_cast<u32x4*>(a.cols + p * a.cols_plane + ((s * a.F + f0 + f) * a.Mp + m0 + m) * 2) = column(tile[s][p], m, f);
    }
}

int64_t tiles(int64_t n) { return (n + 63) / 64; }

template <int DT>
hipError_t lay(const FfnLay (&l)[3], bool turned, hipStream_t s) {
    Three t{};
    unsigned n = 0;
    for (int i = 0; i < 3; ++i) {
        t.l[i] = l[i];
        if (l[i].R) n += static_cast<unsigned>(turned ? tiles(l[i].pad) * tiles(l[i].C) : (l[i].R * (l[i].pad / 8) + 255) / 256);
        t.upto[i] = n;
    }
    if (!n) return hipSuccess;
    if (!turned)
        lay_rows<DT><<<n, 256, 0, s>>>(t);
    else if constexpr (DT != SDM_E4M3)
        lay_turned<DT><<<n, 256, 0, s>>>(t);
    return hipGetLastError();
}

}  // namespace

// All three of one type; 8-bit ones are never turned (they have no gradient).
hipError_t launch_ffn_lay(const FfnLay (&l)[3], bool turned, hipStream_t s) {
    const int dtype = l[0].R ? l[0].dtype : l[1].R ? l[1].dtype : l[2].dtype;
    if (dtype == SDM_F32) return lay<SDM_F32>(l, turned, s);
    return dtype == SDM_E4M3 ? lay<SDM_E4M3>(l, turned, s) : lay<SDM_BF16>(l, turned, s);
}

hipError_t launch_ffn_grad(const FfnGrad& g, hipStream_t s) {
    const unsigned grid = static_cast<unsigned>(tiles(g.Mp) * tiles(g.Fp));
    const int across = static_cast<int>(tiles(g.Fp));
    if (g.dtype == SDM_F32)
        ffn_grad<SDM_F32><<<grid, 256, 0, s>>>(g, across);
    else if (g.dtype == SDM_BF16)
        ffn_grad<SDM_BF16><<<grid, 256, 0, s>>>(g, across);
    else
        ffn_grad<SDM_F16><<<grid, 256, 0, s>>>(g, across);
    return hipGetLastError();
}

}  // namespace sdm_delta
