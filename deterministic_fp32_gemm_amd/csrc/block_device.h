// Device pieces shared by the kernels of libsdm_block.
#pragma once

#include "delta_types.h"
#include "../../include/sdm_ffn.h"

namespace sdm_delta {

// act(z) and act'(z). With e = exp(-|z|) the sigmoid p and 1 - p are 1 / (1 + e) and e / (1 + e), in the order of z's sign:
// 1 - p taken as a difference would keep nothing of act' from z = 17 on. FAST: the hardware's exponential and reciprocal (1
// ulp of float32), for results of 16 bits. At z = -inf z p is NaN as the formula has it.
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
    float e, large;
    if constexpr (FAST) {
        e = __builtin_amdgcn_exp2f(-1.44269504f * fabsf(z));
        large = __builtin_amdgcn_rcpf(1.f + e);
    } else {
        e = expf(-fabsf(z));
        large = 1.f / (1.f + e);
    }
    const float small = e * large, p = z < 0.f ? small : large, q = z < 0.f ? large : small;
    if (act == SDM_ACT_SIGMOID) {
        a = p;
        d = p * q;
    } else {
        a = z * p;
        d = p * (1.f + z * q);
    }
}

}  // namespace sdm_delta
