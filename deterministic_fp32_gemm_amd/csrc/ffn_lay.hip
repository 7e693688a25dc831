// What the feed-forward's products read beside the inputs where they lie (sdm_ffn.h): operands laid out anew (odd
// alignments, and turned for the gradient's sums over rows), and dg and du, for gfx950.
//
// Bounded by memory: each value is read once and written once (dg and du twice, by rows and by columns). Tiles of 64 x 64 are
// turned through LDS, so that both sides move whole lines.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "block_device.h"
#include "ffn.h"

namespace sdm_delta {
namespace {

template <int N> struct Bits;       // an element of N bytes
template <> struct Bits<1> { using type = uint8_t; };
template <> struct Bits<2> { using type = uint16_t; };
template <> struct Bits<4> { using type = uint32_t; };
template <int N> using bits_t = typename Bits<N>::type;

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

// A thread has 16 bytes of one row.
template <int N>
__global__ __launch_bounds__(256) void lay_rows(const Three three) {
    using B = bits_t<N>;
    constexpr int E = 16 / N;
    unsigned b = blockIdx.x;
    const FfnLay& l = three.l[which(three, b)];
    const int64_t groups = l.pad / E, id = static_cast<int64_t>(b) * 256 + threadIdx.x;
    if (id >= l.R * groups) return;
    const int64_t r = id / groups, c = id % groups * E;
    const B* src = static_cast<const B*>(l.src) + r * l.ld;
    struct Sixteen {
        B v[E];
    } o;
#pragma unroll
    for (int i = 0; i < E; ++i) {
        const B x = src[min(c + i, l.C - 1)];
        o.v[i] = c + i < l.C ? x : 0;
    }
    *reinterpret_cast<u32x4*>(l.dst + r * l.ldd + c * N) = __builtin_bit_cast(u32x4, o);
}

// A tile of 64 x 64 on its way to being turned; rows are an odd number of banks apart.
template <int N> constexpr int kAcross = N == 4 ? 65 : 66;
// 16 bytes of a column: tile[k][c] from k = from
__device__ __forceinline__ u32x4 column(const uint16_t (*tile)[66], int from, int c) {
    u32x4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = tile[from + 2 * i][c] | static_cast<uint32_t>(tile[from + 2 * i + 1][c]) << 16;
    return o;
}
__device__ __forceinline__ u32x4 column(const uint32_t (*tile)[65], int from, int c) {
    return u32x4{tile[from][c], tile[from + 1][c], tile[from + 2][c], tile[from + 3][c]};
}
// Four neighbours of a row, to LDS and to memory.
__device__ __forceinline__ void put4(uint16_t* p, const uint16_t (&v)[4]) {
    reinterpret_cast<uint32_t*>(p)[0] = v[0] | static_cast<uint32_t>(v[1]) << 16;
    reinterpret_cast<uint32_t*>(p)[1] = v[2] | static_cast<uint32_t>(v[3]) << 16;
}
__device__ __forceinline__ void put4(uint32_t* p, const uint32_t (&v)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = v[i];
}
__device__ __forceinline__ void store4(char* p, const uint16_t (&v)[4]) {
    *reinterpret_cast<u32x2*>(p) = u32x2{v[0] | static_cast<uint32_t>(v[1]) << 16, v[2] | static_cast<uint32_t>(v[3]) << 16};
}
__device__ __forceinline__ void store4(char* p, const uint32_t (&v)[4]) { *reinterpret_cast<u32x4*>(p) = u32x4{v[0], v[1], v[2], v[3]}; }

// Four columns of a row from c as their bits: all there, or read from inside the row and zero past its end.
__device__ __forceinline__ void four(uint32_t (&o)[4], const uint32_t* row, int64_t c, int64_t n) {
    typedef uint32_t u32x4a __attribute__((ext_vector_type(4), aligned(4)));
    if (c + 4 <= n) {
        const u32x4 x = *reinterpret_cast<const u32x4a*>(row + c);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = x[i];
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t x = row[min(c + i, n - 1)];
        o[i] = c + i < n ? x : 0;
    }
}
__device__ __forceinline__ void four(uint16_t (&o)[4], const uint16_t* row, int64_t c, int64_t n) {
    typedef uint32_t u32x2u __attribute__((ext_vector_type(2), aligned(2)));
    if (c + 4 <= n) {
        const u32x2 x = *reinterpret_cast<const u32x2u*>(row + c);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = static_cast<uint16_t>(x[i / 2] >> (16 * (i % 2)));
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint16_t x = row[min(c + i, n - 1)];
        o[i] = c + i < n ? x : 0;
    }
}

// dst[c][r]: a tile of 64 rows and 64 columns.
template <int N>
__device__ __forceinline__ void lay_turned(const Three& three, unsigned b, bits_t<N> (&tile)[64][kAcross<N>]) {
    using B = bits_t<N>;
    const FfnLay& l = three.l[which(three, b)];
    const unsigned across = static_cast<unsigned>((l.C + 63) / 64);
    const int64_t r0 = static_cast<int64_t>(b / across) * 64, c0 = static_cast<int64_t>(b % across) * 64;
    const int r16 = threadIdx.x / 16, c4 = threadIdx.x % 16 * 4;
    B x[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) four(x[i], static_cast<const B*>(l.src) + min(r0 + i * 16 + r16, l.R - 1) * l.ld, c0 + c4, l.C);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int k = 0; k < 4; ++k) x[i][k] = r0 + i * 16 + r16 < l.R ? x[i][k] : 0;
        put4(&tile[i * 16 + r16][c4], x[i]);
    }
    __syncthreads();
    constexpr int E = 16 / N, L = 64 / E;
#pragma unroll
    for (int i = 0; i < L / 4; ++i) {
        const int c = i * (256 / L) + threadIdx.x / L, r = threadIdx.x % L * E;
        if (c0 + c >= l.C || r0 + r >= l.pad) continue;
        char* p = l.dst + (c0 + c) * l.ldd + (r0 + r) * N;
        *reinterpret_cast<u32x4*>(p) = column(tile, r, c);
        if (l.again) *reinterpret_cast<u32x4*>(p + l.again) = column(tile, r, c);
    }
}

__device__ __forceinline__ float value(uint32_t b, float) { return __uint_as_float(b); }
__device__ __forceinline__ float value(uint16_t b, __bf16) { return static_cast<float>(__builtin_bit_cast(__bf16, b)); }
__device__ __forceinline__ float value(uint16_t b, _Float16) { return static_cast<float>(__builtin_bit_cast(_Float16, b)); }

// dg and du, and, in the workgroups from `first` on, the operands to be turned: one launch for all that the gradient's products
// read. 16-bit types: dg and du are rounded to dtype, as their products take them, in PARTS parts.
template <int DT, int PARTS>
__global__ __launch_bounds__(256) void ffn_grad(const FfnGrad a, const int across, const Three three, const unsigned first) {
    using T = elem_t<DT>;
    constexpr int N = sizeof(T);
    using B = bits_t<N>;
    __shared__ B tile[2][64][kAcross<N>];
    if (blockIdx.x >= first) {
        lay_turned<N>(three, blockIdx.x - first, tile[0]);
        return;
    }
    const int64_t m0 = static_cast<int64_t>(blockIdx.x / across) * 64, f0 = static_cast<int64_t>(blockIdx.x % across) * 64;
    const int r16 = threadIdx.x / 16, c = threadIdx.x % 16 * 4;
    B dh[4][4], lost[PARTS == 2 ? 4 : 1][2][4];
    uint32_t g[4][4], u[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t m = min(m0 + i * 16 + r16, a.M - 1);
        four(dh[i], static_cast<const B*>(a.dh) + m * a.ld_dh, f0 + c, a.F);
        four(g[i], reinterpret_cast<const uint32_t*>(a.gate) + m * a.ld_gate, f0 + c, a.F);
        four(u[i], reinterpret_cast<const uint32_t*>(a.up) + m * a.ld_up, f0 + c, a.F);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = i * 16 + r16;
        B x[2][4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float act, d;
            gate<DT != SDM_F32>(__uint_as_float(g[i][k]), a.act, act, d);
            const bool in = m0 + r < a.M && f0 + c + k < a.F;
            const float h = value(dh[i][k], T{});
            const float v[2] = {in ? h * __uint_as_float(u[i][k]) * d : 0.f, in ? h * act : 0.f};
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const T first_part = static_cast<T>(v[s]);
                x[s][k] = __builtin_bit_cast(B, first_part);
                // nothing is lost of what is not finite
                if constexpr (PARTS == 2)
                    lost[i][s][k] = __builtin_bit_cast(B, static_cast<T>(__builtin_isfinite(static_cast<float>(first_part)) ? v[s] - static_cast<float>(first_part) : 0.f));
            }
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            put4(&tile[s][r][c], x[s]);
            // c and a row's padded length are multiples of 4
            if (m0 + r < a.M && f0 + c < a.Fp) {
                char* p = a.rows + ((m0 + r) * 2 * PARTS * a.Fp + s * a.Fp + f0 + c) * N;
                store4(p, x[s]);
                if constexpr (PARTS == 2) store4(p + 2 * a.Fp * N, lost[i][s]);
            }
        }
    }
    constexpr int E = 16 / N, L = 64 / E;
#pragma unroll
    for (int part = 0; part < PARTS; ++part) {
        __syncthreads();
        if (part) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int s = 0; s < 2; ++s) put4(&tile[s][i * 16 + r16][c], lost[i][s]);
            __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < L / 4; ++i) {
            const int f = i * (256 / L) + threadIdx.x / L, m = threadIdx.x % L * E;
            if (f0 + f >= a.F || m0 + m >= a.Mp) continue;
#pragma unroll
            for (int s = 0; s < 2; ++s)
                *reinterpret_cast<u32x4*>(a.cols + ((s * a.F + f0 + f) * PARTS * a.Mp + part * a.Mp + m0 + m) * N) = column(tile[s], m, f);
        }
    }
}

struct Joins {
    FfnJoin j[2];
    int64_t first;      // threads of the first
};
// A thread has four columns of a row.
__global__ __launch_bounds__(256) void ffn_join(const Joins joins, const int64_t all) {
    int64_t id = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (id >= all) return;
    const FfnJoin& j = joins.j[id >= joins.first];
    id -= id >= joins.first ? joins.first : 0;
    const int64_t m = id / (j.ld / 4), n = id % (j.ld / 4) * 4;
    f32x4 sum = {0.f, 0.f, 0.f, 0.f};
    for (int i = 0; i < j.parts; ++i) sum += *reinterpret_cast<const f32x4*>(j.from + (i * j.M + m) * j.ld + n);
    char* c = m < j.split ? j.c : j.c2;
    const int64_t at = (m < j.split ? m * j.ldc : (m - j.split) * j.ldc2) + n;
    for (int e = 0; e < 4 && n + e < j.N; ++e) {
        if (j.otype == SDM_F32)
            reinterpret_cast<float*>(c)[at + e] = sum[e];
        else if (j.otype == SDM_BF16)
            reinterpret_cast<__bf16*>(c)[at + e] = static_cast<__bf16>(sum[e]);
        else
            reinterpret_cast<_Float16*>(c)[at + e] = static_cast<_Float16>(sum[e]);
    }
}

int64_t tiles(int64_t n) { return (n + 63) / 64; }

template <int N>
hipError_t lay(const FfnLay (&l)[3], hipStream_t s) {
    Three t{};
    unsigned n = 0;
    for (int i = 0; i < 3; ++i) {
        t.l[i] = l[i];
        n += static_cast<unsigned>((l[i].R * (l[i].pad * N / 16) + 255) / 256);
        t.upto[i] = n;
    }
    if (n) lay_rows<N><<<n, 256, 0, s>>>(t);
    return hipGetLastError();
}

template <int DT>
hipError_t grad(const FfnGrad& g, const FfnLay (&l)[3], hipStream_t s) {
    const unsigned first = static_cast<unsigned>(tiles(g.Mp) * tiles(g.Fp));
    Three t{};
    unsigned n = 0;
    for (int i = 0; i < 3; ++i) {
        t.l[i] = l[i];
        n += static_cast<unsigned>(tiles(l[i].pad) * tiles(l[i].C));
        t.upto[i] = n;
    }
    if (g.parts == 1)
        ffn_grad<DT, 1><<<first + n, 256, 0, s>>>(g, static_cast<int>(tiles(g.Fp)), t, first);
    else if constexpr (DT != SDM_F32)
        ffn_grad<DT, 2><<<first + n, 256, 0, s>>>(g, static_cast<int>(tiles(g.Fp)), t, first);
    return hipGetLastError();
}

}  // namespace

// All three of one type; without rows: none
hipError_t launch_ffn_lay(const FfnLay (&l)[3], hipStream_t s) {
    const int dtype = l[0].R ? l[0].dtype : l[1].R ? l[1].dtype : l[2].dtype;
    return dtype == SDM_F32 ? lay<4>(l, s) : dtype == SDM_E4M3 ? lay<1>(l, s) : lay<2>(l, s);
}

hipError_t launch_ffn_join(const FfnJoin (&j)[2], hipStream_t s) {
    Joins joins{{j[0], j[1]}, j[0].parts > 1 ? j[0].M * (j[0].ld / 4) : 0};
    const int64_t all = joins.first + (j[1].parts > 1 ? j[1].M * (j[1].ld / 4) : 0);
    if (all) ffn_join<<<static_cast<unsigned>((all + 255) / 256), 256, 0, s>>>(joins, all);
    return hipGetLastError();
}

hipError_t launch_ffn_grad(const FfnGrad& g, const FfnLay (&l)[3], hipStream_t s) {
    if (g.dtype == SDM_F32) return grad<SDM_F32>(g, l, s);
    return g.dtype == SDM_BF16 ? grad<SDM_BF16>(g, l, s) : grad<SDM_F16>(g, l, s);
}

}  // namespace sdm_delta
