// Rows brought to 8 bits (sdm_qnt.h), with the residual's addition and the norm before it or alone, for gfx950.
//
//     x' = x + r;  y = x' w r1,  r1 = 1 / sqrt(mean x'^2 + eps);  s = max |y| / 448;  q = e4m3(y / s)
//
// What bounds it is memory: x and r are read, x' and q written, each once. A row lives in the registers of one workgroup
// from its load to its store. Since r1 is one positive number a row and rounding is monotonic, max |x' w r1| is the rounded
// max |x' w| r1: the sum and the maximum of a row go through the workgroup together, one barrier a row. The maximum is taken
// of the bits of |x' w|, whose order as integers is that of the values with infinities and then NaN on top: one comparison
// finds a row that cannot be scaled. 16384 rows of 4096 in bfloat16 with a residual: 80 us, 5.9 TB/s; 5000 of 2050 in float32,
// whose rows begin on 8 bytes: 15.5 us, 3.3 TB/s.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "delta_types.h"
#include "qnt.h"

namespace sdm_delta {
namespace {

constexpr uint32_t kInf = 0x7f800000u;

template <int DT, int WT, int NT, int NV>
__global__ __launch_bounds__(NT) void qnt_rows(const sdm_qnt_args_t a) {
    using T = elem_t<DT>;
    constexpr bool kAhead = NT < 1024 || NV == 1;       // the longest rows leave no registers for the next one
    __shared__ float sums[2][16];
    __shared__ uint32_t tops[2][16];
    const int D = static_cast<int>(a.D), id = static_cast<int>(threadIdx.x), nt = static_cast<int>(blockDim.x), waves = nt >> 6;
    const float inv = 1.f / static_cast<float>(D);
    const bool has_r = a.r != nullptr, has_w = a.w != nullptr;
    struct {
        Raw<DT> x[NV], r[NV];
    } in;
    auto fetch = [&](int64_t row) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * nt + id) * 8;
            load_row<DT, true>(in.x[v], static_cast<const T*>(a.x) + row * a.ld_x, c, D);
            if (has_r) load_row<DT, true>(in.r[v], static_cast<const T*>(a.r) + row * a.ld_r, c, D);
        }
    };
    if constexpr (kAhead) fetch(blockIdx.x);
    float w[NV][8];
    if (has_w) {
#pragma unroll
        for (int v = 0; v < NV; ++v) load8<WT>(w[v], static_cast<const elem_t<WT>*>(a.w), (v * nt + id) * 8, D);
    }
    int buf = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, buf ^= 1) {
        float x[NV][8];
        float ss = 0.f;
        uint32_t top = 0u;
        if constexpr (!kAhead) fetch(row);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * nt + id) * 8, past = c + 8 - D;
            raw_floats<DT>(x[v], in.x[v]);
            if (__builtin_expect(past > 0 && D >= 8, 0)) move_down(x[v], past);
            if (has_r) {
                float r[8];
                raw_floats<DT>(r, in.r[v]);
                if (__builtin_expect(past > 0 && D >= 8, 0)) move_down(r, past);
#pragma unroll
                for (int i = 0; i < 8; ++i) x[v][i] = static_cast<float>(static_cast<T>(x[v][i] + r[i]));
            }
        }
        if (kAhead && row + gridDim.x < a.rows) fetch(row + gridDim.x);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * nt + id) * 8;
            if (has_r) store8(static_cast<T*>(a.x_new) + row * a.ld_xn, c, D, x[v]);
            if (has_w) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    ss = __builtin_fmaf(x[v][i], x[v][i], ss);
                    x[v][i] *= w[v][i];
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(x[v][i]) & 0x7fffffffu);
        }
        // in an order set by the lane and wavefront numbers alone
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) {
            if (has_w) ss += __shfl_xor(ss, m, 64);
            top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), m, 64)));
        }
        if constexpr (NT > 64) {
            if ((id & 63) == 0) {
                sums[buf][id >> 6] = ss;
                tops[buf][id >> 6] = top;
            }
            lds_barrier();      // the other row of either array is written again only after the next one
            ss = 0.f;
            top = 0u;
#pragma unroll
            for (int i = 0; i < NT / 64; ++i)
                if (i < waves) {
                    ss += sums[buf][i];
                    top = max(top, tops[buf][i]);
                }
        }
        const float r1 = has_w ? 1.f / sqrtf(ss * inv + a.eps) : 1.f;
        float peak = __uint_as_float(top) * r1;
        // infinite or NaN: a value, or the mean of a row of huge ones (r1 is zero)
        const bool bad = top >= kInf || !(ss < __uint_as_float(kInf)) || !(peak < __uint_as_float(kInf));
        const float scale = bad ? __uint_as_float(0x7fc00000u) : fmaxf(peak / 448.f, 1.17549435e-38f);
        const float k = 1.f / scale;
        if (id == 0) a.scale[row] = scale;
        uint8_t* q = static_cast<uint8_t*>(a.q) + row * a.ld_q;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * nt + id) * 8;
            u32x2 o = {0u, 0u};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                // peak / scale may round to just above 448, which rounds to 448
                const float p = x[v][2 * i] * r1 * k, n = x[v][2 * i + 1] * r1 * k;
                int word = __builtin_amdgcn_cvt_pk_fp8_f32(p, n, 0, false) & 0xffff;
                if (bad) word = 0x7f7f;
                o[i / 2] |= static_cast<uint32_t>(word) << (16 * (i % 2));
            }
            if (c + 8 <= D) {
                typedef uint32_t u32x2u __attribute__((ext_vector_type(2), aligned(1)));
                *reinterpret_cast<u32x2u*>(q + c) = o;
            } else {
#pragma unroll
                for (int i = 0; i < 7; ++i)
                    if (c + i < D) q[c + i] = static_cast<uint8_t>(o[i / 4] >> (8 * (i % 4)));
            }
        }
    }
}

template <int DT, int WT, int NT, int NV>
hipError_t run(const sdm_qnt_args_t& a, const QntPlan& p, hipStream_t s) {
    qnt_rows<DT, WT, NT, NV><<<p.groups, p.threads, 0, s>>>(a);
    return hipGetLastError();
}
template <int DT, int WT>
hipError_t of(const sdm_qnt_args_t& a, const QntPlan& p, hipStream_t s) {
    if (p.most == 64) return run<DT, WT, 64, 1>(a, p, s);
    if (p.most == 256) return p.vecs == 1 ? run<DT, WT, 256, 1>(a, p, s) : run<DT, WT, 256, 2>(a, p, s);
    return p.vecs == 1 ? run<DT, WT, 1024, 1>(a, p, s) : run<DT, WT, 1024, 2>(a, p, s);
}

}  // namespace

// wtype is dtype or float32 (the host checks)
hipError_t launch_qnt(const sdm_qnt_args_t& a, const QntPlan& p, hipStream_t s) {
    if (a.dtype == SDM_F32) return of<0, 0>(a, p, s);
    if (a.dtype == SDM_BF16) return a.wtype == SDM_F32 ? of<1, 0>(a, p, s) : of<1, 1>(a, p, s);
    return a.wtype == SDM_F32 ? of<2, 0>(a, p, s) : of<2, 2>(a, p, s);
}

}  // namespace sdm_delta
