// Device pieces shared by the kernels of libsdm_block.
#pragma once

#include "delta_types.h"
#include "../../include/sdm_ffn.h"

namespace sdm_delta {

// e^x within 2^-23 of it in 7 instructions: the hardware's 2^t for t = x log2(e), whose rounding (and log2(e)'s own) goes back
// in as a factor 1 + r. Below -150 it is zero, as float32 has it without its last denormals.
__device__ __forceinline__ float exp_of(float x) {
    x = x < -150.f ? -150.f : x;
    const float t = x * 1.44269504f, e = __builtin_amdgcn_exp2f(t);
    // log2(e) - 1.44269504f = 1.9259630e-8; times ln 2
    const float r = 0.69314718f * __builtin_fmaf(x, 1.44269504f, -t) + 1.3349759e-8f * x;
    return __builtin_fmaf(e, r, e);
}

// p = 1 / (1 + e^-z) and q = 1 - p. With e = e^-|z| they are 1 / (1 + e) and e / (1 + e), in the order of z's sign: as a
// difference q would keep nothing of itself from z = 17 on, and neither is ever 0 times infinity. FAST: the hardware's
// exponential and reciprocal (their errors, and 2^-24 |z| of the exponent's argument, are far below a rounding to 16 bits), else
// one more step of Newton's for the reciprocal. What is below 2^-126 may be zero.
template <bool FAST>
__device__ __forceinline__ void sigmoid(float z, float& p, float& q) {
    const float e = FAST ? __builtin_amdgcn_exp2f(-1.44269504f * fabsf(z)) : exp_of(-fabsf(z)), d = 1.f + e;
    float large = __builtin_amdgcn_rcpf(d);
    if constexpr (!FAST) large = __builtin_fmaf(__builtin_fmaf(-d, large, 1.f), large, large);
    const float small = e * large;
    p = z < 0.f ? small : large;
    q = z < 0.f ? large : small;
}

// act(z) and act'(z). Far below zero z p and its derivative are zero, since p is; at z = -inf they are NaN, -inf times 0.
template <bool FAST>
__device__ __forceinline__ void gate(float z, int act, float& a, float& d) {
    if (act == SDM_ACT_NONE) {
        a = z;
        d = 1.f;
        return;
    }
    if (act == SDM_ACT_GELU) {
        // z Phi(z): erfc keeps Phi's last bits where z is far below zero
        const float p = 0.5f * erfcf(-0.70710678f * z);
        const float e = FAST ? __builtin_amdgcn_exp2f(-0.72134752f * z * z) : expf(-0.5f * z * z);
        a = z * p;
        d = __builtin_fmaf(0.39894228f * e, z, p);
        return;
    }
    float p, q;
    sigmoid<FAST>(z, p, q);
    if (act == SDM_ACT_SIGMOID) {
        a = p;
        d = p * q;
    } else {
        a = z * p;
        d = p * __builtin_fmaf(z, q, 1.f);
    }
}

// An 8-bit product times its rows' scales, whose own product may leave float32 where the result does not: their exponents go
// apart (8192 rows of 4096 to 8192: 489 us where plain products take 485; in 64 bits 502 where they take 495).
struct Scale {
    float m;
    int x;
};
__device__ __forceinline__ Scale scale_of(float s) { return Scale{__builtin_amdgcn_frexp_mantf(s), __builtin_amdgcn_frexp_expf(s)}; }
__device__ __forceinline__ float scaled(float v, const Scale& s, const Scale& t) { return __builtin_amdgcn_ldexpf(v * (s.m * t.m), s.x + t.x); }

}  // namespace sdm_delta
