// Division of a row by its scale amax / MAX, and the casts behind it: what the
// quantizers with a row or tensor scale share (gfx950 only).  The quotient is
// the correctly rounded one by Markstein's correction; see quantize.hip.
#pragma once

#include <type_traits>

#include "device_common.h"

namespace fp8g {

constexpr float FLT_MIN_NORMAL = 1.17549435e-38f;

// ---- output formats: the largest finite magnitude (the divisor of amax) and
// the saturating round-to-nearest-even cast of four values into one dword
struct OutE4M3 {
    static constexpr float MAX = 448.0f;
    __device__ __forceinline__ static uint32_t pack4(float a, float b, float c, float d) {
        return e4m3_pack4(a, b, c, d);
    }
};

struct OutE5M2 {
    static constexpr float MAX = 57344.0f;
    __device__ __forceinline__ static uint32_t pack4(float a, float b, float c, float d) {
        return e5m2_pack4(a, b, c, d);
    }
};

// Per-row (per-tensor) divisor: the scale, its correctly rounded reciprocal, the path.
struct RowDiv {
    float s, y;
    bool zero;    // s == 0: signed zeros
    bool ieee;    // s below the smallest normal: plain IEEE division
};

// amax is the same in every lane; readfirstlane makes that visible to the
// compiler, so the path is chosen once with a scalar branch.
template <class O>
__device__ __forceinline__ RowDiv row_div(float amax) {
    amax = __builtin_bit_cast(float, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, amax)));
    RowDiv d;
    d.s = amax / O::MAX;
    d.y = 1.0f / d.s;
    d.zero = (d.s == 0.0f);
    d.ieee = (d.s < FLT_MIN_NORMAL);
    return d;
}

// PATH 0: Markstein quotient; 1: IEEE division; 2: signed zero (s == 0)
template <int PATH>
__device__ __forceinline__ float quot(float x, const RowDiv& d) {
    if constexpr (PATH == 2) {
        return x * 0.0f;
    } else if constexpr (PATH == 1) {
        return x / d.s;
    } else {
        const float q0 = x * d.y;
        const float e = __builtin_fmaf(-q0, d.s, x);
        // x = -0 gives e = +0 and q0 + e y = +0; the quotient has x's sign (s > 0)
        return __builtin_copysignf(__builtin_fmaf(e, d.y, q0), x);
    }
}

// f(path_tag) with the path as a compile-time constant
template <typename F>
__device__ __forceinline__ void by_path(const RowDiv& d, F&& f) {
    if (d.zero) f(std::integral_constant<int, 2>{});
    else if (d.ieee) f(std::integral_constant<int, 1>{});
    else f(std::integral_constant<int, 0>{});
}

__device__ __forceinline__ float amax2(float a, float b) { return __builtin_fmaxf(__builtin_fabsf(a), __builtin_fabsf(b)); }

}  // namespace fp8g
