// The work behind a fused product: bias, activation, gate, residual (gfx950 only).
#pragma once

#include "device_common.h"

namespace fp8g {

// v / (1 + exp(-p(v))), p(v) = v (c1 + c3 v^2): SILU has c1 = 1, c3 = 0, and
// the tanh form of GELU, v (1 + tanh u) / 2 = v / (1 + exp(-2 u)), has
// c1 = 2 sqrt(2 / pi), c3 = 0.044715 c1.  Held times -log2(e), so that the
// exponential is one instruction.
struct Act {
    float c1, c3;
    int32_t on;
};

inline Act act_of(int act) {
    constexpr double LOG2E = 1.4426950408889634, GELU = 1.5957691216057308;
    if (act == 1) return Act{(float)-LOG2E, 0.0f, 1};
    if (act == 2) return Act{(float)(-LOG2E * GELU), (float)(-LOG2E * GELU * 0.044715), 1};
    return Act{0.0f, 0.0f, 0};
}

__device__ __forceinline__ float activate(float v, float c1, float c3) {
    const float t = v * __builtin_fmaf(c3 * v, v, c1);
    return v * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(t));
}

}  // namespace fp8g
