// Element types of the delta kernels and their loads and stores: float32, bfloat16 and float16 rows of any alignment.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace sdm_delta {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

template <int DT> struct Elem;
template <> struct Elem<0> { using type = float; };
template <> struct Elem<1> { using type = __bf16; };
template <> struct Elem<2> { using type = _Float16; };
template <int DT> using elem_t = typename Elem<DT>::type;

// 16 bytes on the boundary of an element: global memory takes them at any.
typedef uint32_t u32x4u __attribute__((ext_vector_type(4), aligned(2)));

// Eight elements of a row as they lie in memory, kept until they are needed: a prefetch costs no more registers than
// its bytes.
template <int DT>
struct Raw {
    u32x4 w[DT == 0 ? 2 : 1];
};
// Eight values of a row of `lim`, from column c; only columns < lim are read. A thread whose columns end past the row
// takes the row's last eight, which move_down puts right when they are used: no branch, so nothing waits for the load
// here. STREAM: the caches need not keep what is read.
template <int DT, bool STREAM = false>
__device__ __forceinline__ void load_row(Raw<DT>& o, const elem_t<DT>* __restrict__ row, int c, int lim) {
    if (lim >= 8) {
        const u32x4u* p = reinterpret_cast<const u32x4u*>(row + min(c, lim - 8));
        o.w[0] = STREAM ? __builtin_nontemporal_load(p) : p[0];
        if constexpr (DT == 0) o.w[1] = STREAM ? __builtin_nontemporal_load(p + 1) : p[1];
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int k = min(c + i, lim - 1);
        if constexpr (DT == 0) {
            const uint32_t x = __float_as_uint(row[k]);
            o.w[i / 4][i % 4] = c + i < lim ? x : 0u;
        } else {
            const uint32_t x = reinterpret_cast<const uint16_t*>(row)[k], y = c + i < lim ? x : 0u;
            o.w[0][i / 2] = i % 2 ? o.w[0][i / 2] | y << 16 : y;
        }
    }
}
template <int DT>
__device__ __forceinline__ void raw_floats(float (&f)[8], const Raw<DT>& r) {
    if constexpr (DT == 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(r.w[i / 4][i % 4]);
    } else {
        typedef elem_t<DT> t8 __attribute__((ext_vector_type(8)));
        const t8 a = __builtin_bit_cast(t8, r.w[0]);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = static_cast<float>(a[i]);
    }
}
// The values of a thread whose columns end past the row, moved to their columns; zero past the row. For a row of 8 or
// more and past = c + 8 - lim > 0.
__device__ __forceinline__ void move_down(float (&f)[8], int past) {
#pragma unroll
    for (int k = 4; k > 0; k >>= 1)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float x = i + k < 8 ? f[i + k < 8 ? i + k : i] : 0.f;
            f[i] = past & k ? x : f[i];
        }
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = past >= 8 ? 0.f : f[i];
}
// load_row and its floats in their columns
template <int DT>
__device__ __forceinline__ void load8(float (&f)[8], const elem_t<DT>* __restrict__ row, int c, int lim) {
    Raw<DT> r;
    load_row<DT>(r, row, c, lim);
    raw_floats<DT>(f, r);
    if (lim >= 8 && c + 8 > lim) move_down(f, c + 8 - lim);
}

template <class T>
__device__ __forceinline__ void store8(T* __restrict__ row, int c, int lim, const float (&f)[8]) {
    if (c + 8 <= lim) {
        u32x4u* p = reinterpret_cast<u32x4u*>(row + c);
        if constexpr (sizeof(T) == 4) {
            p[0] = u32x4{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])};
            p[1] = u32x4{__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7])};
        } else {
            typedef T t8 __attribute__((ext_vector_type(8)));
            t8 a;
#pragma unroll
            for (int i = 0; i < 8; ++i) a[i] = static_cast<T>(f[i]);
            p[0] = __builtin_bit_cast(u32x4, a);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 7; ++i)
        if (c + i < lim) row[c + i] = static_cast<T>(f[i]);
}

// LDS written by this workgroup becomes visible to it. The fences name LDS alone: unlike __syncthreads, the barrier
// does not wait for global loads in flight.
__device__ __forceinline__ void lds_barrier() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

}  // namespace sdm_delta
