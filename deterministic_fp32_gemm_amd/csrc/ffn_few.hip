// The gated feed-forward product of few rows (sdm_ffn.h): one token, or a batch of streams' next ones, for gfx950.
//
// Bounded by the weights' bytes, each read once. A workgroup owns 16 rows of either weight: its eight wavefronts take
// blocks of 256 bytes of them in turn, straight from memory into the matrix cores' operands (lane l: 16 bytes of row l % 16
// for each 64 bytes), against the same bytes of x's rows, which stay in the caches. The next block's loads are in
// flight while a block is multiplied. The wavefronts' sums meet in
// LDS and are added in order. Which element meets which place of an instruction's summed axis does not matter as long as
// both operands agree. One row of 2048 to 8192 in bfloat16: 12.2 us, 5.5 TB/s. float32 takes float32 matrix instructions: their rate is enough for what memory brings.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "block_device.h"
#include "ffn.h"

namespace sdm_delta {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef long i64x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4b __attribute__((ext_vector_type(4), aligned(1)));

constexpr int kWaves = 8, kDepth = 4;       // wavefronts that share the rows, 64-byte steps of a block

// DT: sdm_dtype or SDM_E4M3; a 16-byte piece of a weight's 16 rows against that of 16 rows of x
template <int DT>
__device__ __forceinline__ void mma(f32x4& acc, const u32x4& w, const u32x4& x) {
    if constexpr (DT == SDM_F32) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(w[i]), __uint_as_float(x[i]), acc, 0, 0, 0);
    } else if constexpr (DT == SDM_BF16) {
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w), __builtin_bit_cast(bf16x8, x), acc, 0, 0, 0);
    } else if constexpr (DT == SDM_F16) {
        acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, w), __builtin_bit_cast(f16x8, x), acc, 0, 0, 0);
    } else {
        const i64x2 a = __builtin_bit_cast(i64x2, w), b = __builtin_bit_cast(i64x2, x);
#pragma unroll
        for (int i = 0; i < 2; ++i) acc = __builtin_amdgcn_mfma_f32_16x16x32_fp8_fp8(a[i], b[i], acc, 0, 0, 0);
    }
}

// 16 bytes from byte c of a row of n bytes, zero past its end. An element never lies across the end.
template <int ES>
__device__ __forceinline__ u32x4 piece(const char* row, int64_t c, int64_t n) {
    if (c + 16 <= n) return *reinterpret_cast<const u32x4b*>(row + c);
    u32x4 o = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 16 / ES; ++i) {
        if (c + i * ES >= n) continue;
        const char* p = row + c + i * ES;
        uint32_t v;
        if constexpr (ES == 4)
            v = *reinterpret_cast<const uint32_t*>(p);
        else if constexpr (ES == 2)
            v = *reinterpret_cast<const uint16_t*>(p);
        else
            v = *reinterpret_cast<const uint8_t*>(p);
        o[i * ES / 4] |= v << (i * ES % 4 * 8);
    }
    return o;
}

template <class T>
__device__ __forceinline__ void put(void* base, int64_t at, float v) {
    static_cast<T*>(base)[at] = static_cast<T>(v);
}
__device__ __forceinline__ void put(int otype, void* base, int64_t at, float v) {
    if (otype == SDM_F32)
        put<float>(base, at, v);
    else if (otype == SDM_BF16)
        put<__bf16>(base, at, v);
    else
        put<_Float16>(base, at, v);
}

template <int DT, int MT>
__global__ __launch_bounds__(kWaves * 64) void ffn_few(const sdm_ffn_args_t a) {
    constexpr int ES = DT == SDM_F32 ? 4 : DT == SDM_E4M3 ? 1 : 2;
    __shared__ float sums[kWaves][2][MT * 16][17];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r = lane & 15, part = lane >> 4;
    const int64_t f0 = static_cast<int64_t>(blockIdx.x) * 16, n = a.K * ES, f = min(f0 + r, a.F - 1);
    const char* g = static_cast<const char*>(a.wg) + f * a.ld_wg * ES;
    const char* u = static_cast<const char*>(a.wu) + f * a.ld_wu * ES;
    const char* x[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) x[i] = static_cast<const char*>(a.x) + min(static_cast<int64_t>(i * 16 + r), a.M - 1) * a.ld_x * ES;
    f32x4 ag[MT], au[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) ag[i] = au[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    constexpr int kBlock = kDepth * 64;
    const int64_t whole = n / kBlock * kBlock;
    u32x4 pg[kDepth], pu[kDepth];
    auto fetch = [&](int64_t c) {
#pragma unroll
        for (int k = 0; k < kDepth; ++k) {
            pg[k] = *reinterpret_cast<const u32x4b*>(g + c + k * 64 + part * 16);
            pu[k] = *reinterpret_cast<const u32x4b*>(u + c + k * 64 + part * 16);
        }
    };
    if (w * kBlock < whole) fetch(w * kBlock);
    for (int64_t c = w * kBlock; c < whole; c += kWaves * kBlock) {
        u32x4 qg[kDepth], qu[kDepth], px[kDepth][MT];
#pragma unroll
        for (int k = 0; k < kDepth; ++k) {
            qg[k] = pg[k];
            qu[k] = pu[k];
#pragma unroll
            for (int i = 0; i < MT; ++i) px[k][i] = *reinterpret_cast<const u32x4b*>(x[i] + c + k * 64 + part * 16);
        }
        if (c + kWaves * kBlock < whole) fetch(c + kWaves * kBlock);
#pragma unroll
        for (int k = 0; k < kDepth; ++k)
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                mma<DT>(ag[i], qg[k], px[k][i]);
                mma<DT>(au[i], qu[k], px[k][i]);
            }
    }
    // what is left of the rows, a step a wavefront
    for (int64_t c = whole + w * 64; c < n; c += kWaves * 64) {
        const u32x4 pg = piece<ES>(g, c + part * 16, n), pu = piece<ES>(u, c + part * 16, n);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const u32x4 px = piece<ES>(x[i], c + part * 16, n);
            mma<DT>(ag[i], pg, px);
            mma<DT>(au[i], pu, px);
        }
    }
    // lane l holds rows 4 (l / 16) .. + 3 of the weights for row l % 16 of x
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            sums[w][0][i * 16 + r][part * 4 + e] = ag[i][e];
            sums[w][1][i * 16 + r][part * 4 + e] = au[i][e];
        }
    __syncthreads();
    for (int i = threadIdx.x; i < MT * 256; i += kWaves * 64) {
        const int m = i >> 4, c = i & 15;
        const int64_t col = f0 + c;
        if (m >= a.M || col >= a.F) continue;
        float x0 = sums[0][0][m][c], x1 = sums[0][1][m][c];
#pragma unroll
        for (int k = 1; k < kWaves; ++k) {
            x0 += sums[k][0][m][c];
            x1 += sums[k][1][m][c];
        }
        if constexpr (DT == SDM_E4M3) {
            const Scale sm = scale_of(a.sx[m]);
            x0 = scaled(x0, sm, scale_of(a.sg[col]));
            x1 = scaled(x1, sm, scale_of(a.su[col]));
        }
        float h, d;
        gate<DT != SDM_F32>(x0, a.act, h, d);
        put(a.otype, a.h, m * a.ld_h + col, h * x1);
        if (a.gate) {
            a.gate[m * a.ld_gate + col] = x0;
            a.up[m * a.ld_up + col] = x1;
        }
    }
}

template <int DT>
hipError_t run(const sdm_ffn_args_t& a, hipStream_t s) {
    const unsigned grid = static_cast<unsigned>((a.F + 15) / 16);
    if constexpr (DT == SDM_F32) {
        if (a.M > 16)
            ffn_few<DT, 2><<<grid, kWaves * 64, 0, s>>>(a);
    }
    if (a.M <= 16) ffn_few<DT, 1><<<grid, kWaves * 64, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_ffn_few(const sdm_ffn_args_t& a, hipStream_t s) {
    if (a.dtype == SDM_F32) return run<SDM_F32>(a, s);
    if (a.dtype == SDM_BF16) return run<SDM_BF16>(a, s);
    return a.dtype == SDM_F16 ? run<SDM_F16>(a, s) : run<SDM_E4M3>(a, s);
}

}  // namespace sdm_delta
