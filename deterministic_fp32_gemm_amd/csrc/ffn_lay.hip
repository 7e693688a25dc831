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

// A thread has 8 columns of one row.
template <int DT>
__global__ __launch_bounds__(256) void lay_rows(const FfnLay l, const int64_t groups) {
    using B = typename Bits<DT>::type;
    constexpr int P = kParts<DT>;
    const int64_t id = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
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

// dst[part][c][r]: a tile of 64 rows and 64 columns. 16-bit parts.
template <int DT>
__global__ __launch_bounds__(256) void lay_turned(const FfnLay l, const int across) {
    constexpr int P = kParts<DT>;
    __shared__ uint16_t tile[P][64][66];
    const int64_t r0 = static_cast<int64_t>(blockIdx.x / across) * 64, c0 = static_cast<int64_t>(blockIdx.x % across) * 64;
    for (int i = threadIdx.x; i < 64 * 64; i += 256) {
        const int r = i >> 6, c = i & 63;
        uint16_t x[P];
        parts_of<DT>(x, l.src, min(r0 + r, l.R - 1) * l.ld + min(c0 + c, l.C - 1));
        const bool in = r0 + r < l.R;
#pragma unroll
        for (int p = 0; p < P; ++p) tile[p][r][c] = in ? x[p] : 0;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 64 * 8; i += 256) {
        const int c = i >> 3, r = (i & 7) * 8;
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
    for (int i = threadIdx.x; i < 64 * 64; i += 256) {
        const int r = i >> 6, c = i & 63;
        const int64_t m = min(m0 + r, a.M - 1), f = min(f0 + c, a.F - 1);
        const float dh = static_cast<float>(static_cast<const T*>(a.dh)[m * a.ld_dh + f]);
        const float g = a.gate[m * a.ld_gate + f], u = a.up[m * a.ld_up + f];
        float act, d;
        gate<DT != SDM_F32>(g, a.act, act, d);
        const bool in = m0 + r < a.M && f0 + c < a.F;
        const float v[2] = {dh * u * d, dh * act};
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            uint16_t x[P];
            if constexpr (DT == SDM_F32)
                split(x, v[k]);
            else
                x[0] = __builtin_bit_cast(uint16_t, static_cast<T>(v[k]));
#pragma unroll
            for (int p = 0; p < P; ++p) tile[k][p][r][c] = in ? x[p] : 0;
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 64 * 8; i += 256) {
        const int r = i >> 3, c = (i & 7) * 8;
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int p = 0; p < P; ++p) {
                if (m0 + r < a.M && f0 + c < a.Fp) {
                    u32x4 o;
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[e] = tile[k][p][r][c + 2 * e] | static_cast<uint32_t>(tile[k][p][r][c + 2 * e + 1]) << 16;
                    *reinterpret_cast<u32x4*>(a.rows + p * a.rows_plane + ((m0 + r) * 2 * a.Fp + k * a.Fp + f0 + c) * 2) = o;
                }
                if (f0 + r < a.F && m0 + c < a.Mp)
                    *reinterpret_cast<u32x4*>(a.cols + p * a.cols_plane + ((k * a.F + f0 + r) * a.Mp + m0 + c) * 2) = column(tile[k][p], c, r);
            }
    }
}

int64_t tiles(int64_t n) { return (n + 63) / 64; }

template <int DT>
hipError_t lay(const FfnLay& l, bool turned, hipStream_t s) {
    if (turned) {
        if constexpr (DT == SDM_E4M3)
            return hipErrorInvalidValue;
        else
            lay_turned<DT><<<static_cast<unsigned>(tiles(l.pad) * tiles(l.C)), 256, 0, s>>>(l, static_cast<int>(tiles(l.C)));
    } else {
        const int64_t groups = l.pad / 8;
        lay_rows<DT><<<static_cast<unsigned>((l.R * groups + 255) / 256), 256, 0, s>>>(l, groups);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_ffn_lay(const FfnLay& l, bool turned, hipStream_t s) {
    if (l.dtype == SDM_F32) return lay<SDM_F32>(l, turned, s);
    return l.dtype == SDM_E4M3 ? lay<SDM_E4M3>(l, turned, s) : lay<SDM_BF16>(l, turned, s);
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
