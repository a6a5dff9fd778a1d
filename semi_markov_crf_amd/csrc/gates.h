// Sigmoid gates on the hardware's exponential and reciprocal (each within 1 ulp).
#pragma once

#include "common.h"

namespace semicrf {

constexpr float LOG2EF = 1.44269504088896f;

__device__ __forceinline__ float rcp(float x) { return __builtin_amdgcn_rcpf(x); }
__device__ __forceinline__ float sigmoid(float z) { return rcp(1.0f + fast_exp2(z * -LOG2EF)); }

// sig(z) and 1 - sig(z), both with a small relative error: the exponential is kept finite, so that
// neither is lost where the gate is far open or far closed.  The comparison lets a NaN pass.
__device__ __forceinline__ void sigmoids(float z, float& p, float& q) {
    const float t = z * -LOG2EF, e = fast_exp2(t > 126.0f ? 126.0f : t);
    p = rcp(1.0f + e);
    q = e * p;
}

}  // namespace semicrf
