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

// Eight elements of a row from column c as float, zero from column `lim` on; only columns < lim are read. `vec`: the
// row starts on a 16-byte boundary and c is a multiple of 8, so eight elements are one or two 16-byte loads.
template <class T>
__device__ __forceinline__ void load8(float (&f)[8], const T* __restrict__ row, int c, int lim, bool vec) {
    if (vec && c + 8 <= lim) {
        if constexpr (sizeof(T) == 4) {
            const f32x4 a = *reinterpret_cast<const f32x4*>(row + c), b = *reinterpret_cast<const f32x4*>(row + c + 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = a[i], f[4 + i] = b[i];
        } else {
            typedef T t8 __attribute__((ext_vector_type(8)));
            const t8 a = *reinterpret_cast<const t8*>(row + c);
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = static_cast<float>(a[i]);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = c + i < lim ? static_cast<float>(row[c + i]) : 0.f;
}

template <class T>
__device__ __forceinline__ void store8(T* __restrict__ row, int c, int lim, bool vec, const float (&f)[8]) {
    if (vec && c + 8 <= lim) {
        if constexpr (sizeof(T) == 4) {
            *reinterpret_cast<f32x4*>(row + c) = f32x4{f[0], f[1], f[2], f[3]};
            *reinterpret_cast<f32x4*>(row + c + 4) = f32x4{f[4], f[5], f[6], f[7]};
        } else {
            typedef T t8 __attribute__((ext_vector_type(8)));
            t8 a;
#pragma unroll
            for (int i = 0; i < 8; ++i) a[i] = static_cast<T>(f[i]);
            *reinterpret_cast<t8*>(row + c) = a;
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
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
