// What the fused products' kernels share: the activations of their epilogues, block
// scales and vectors that start anywhere (gfx950 only).
#pragma once

#include "device_common.h"

namespace fp8g {

// v / (1 + exp(-p(v))), p(v) = v (c1 + c3 v^2): SILU has c1 = 1, and the tanh form
// of GELU, v (1 + tanh u) / 2 = v / (1 + exp(-2 u)), has c1 = 2 sqrt(2 / pi), c3 =
// 0.044715 c1.  Held times -log2(e), so that the exponential is one instruction.
// Of +inf both are +inf, of -inf and NaN they are NaN, as the formulas are.
//
// SILU's c3 is not 0, which times +inf would be NaN, but 2^-100: below |v| = 2^37
// it rounds away against c1 (c3 v^2 < 2^-26), and from there on exp(-p) is 0 or
// infinite either way.  (The largest finite v in place of +inf, by one v_min, moved
// the 256x256 experts' kernel's registers: 65536 rows of 128 experts 604 -> 680 us.)
struct Act {
    float c1, c3;
    int32_t on;
};

inline Act act_of(int act) {
    constexpr double LOG2E = 1.4426950408889634, GELU = 1.5957691216057308;
    if (act == 1) return Act{(float)-LOG2E, -0x1p-100f, 1};
    if (act == 2) return Act{(float)(-LOG2E * GELU), (float)(-LOG2E * GELU * 0.044715), 1};
    return Act{0.0f, 0.0f, 0};
}

__device__ __forceinline__ float activate(float v, float c1, float c3) {
    const float t = v * __builtin_fmaf(c3 * v, v, c1);
    return v * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(t));
}

// Dword c of a row of nblk scale bytes that starts at any byte, by the aligned
// dwords that hold it; bytes behind the row are unspecified.
__device__ __forceinline__ uint32_t scale_word(const uint8_t* row, int c, int nblk) {
    const uint32_t by = (uint32_t)(reinterpret_cast<uintptr_t>(row) & 3);
    const uint32_t* w = reinterpret_cast<const uint32_t*>(row - by) + c;
    const int last = (int)((by + (uint32_t)nblk - 1) / 4);      // the row's last aligned dword
    const uint32_t lo = c <= last ? w[0] : 0u;
    if (by == 0) return lo;
    const uint32_t hi = c + 1 <= last ? w[1] : 0u;
    return (lo >> (8 * by)) | (hi << (32 - 8 * by));
}

typedef unsigned int v4u __attribute__((ext_vector_type(4)));
// 16 bytes of elements from any element on, the first `many` of them (0 or fewer:
// none; the others are 0, or left alone).  Vector loads and stores need only an
// element's alignment here.
template <class E>
struct __attribute__((packed, aligned(sizeof(E)))) AnyUnit {
    v4u v;
};
template <class E>
__device__ __forceinline__ v4u load_some(const E* p, int many) {
    constexpr int PER = 16 / sizeof(E), BITS = 8 * sizeof(E);
    if (many >= PER) return reinterpret_cast<const AnyUnit<E>*>(p)->v;
    v4u d = {};
#pragma unroll
    for (int i = 0; i < PER - 1; ++i)
        if (i < many) d[i * BITS / 32] |= (uint32_t)p[i] << (i * BITS % 32);
    return d;
}
template <class E>
__device__ __forceinline__ void store_some(E* p, int many, v4u d) {
    constexpr int PER = 16 / sizeof(E), BITS = 8 * sizeof(E);
    if (many >= PER) {
        reinterpret_cast<AnyUnit<E>*>(p)->v = d;
        return;
    }
#pragma unroll
    for (int i = 0; i < PER - 1; ++i)
        if (i < many) p[i] = (E)(d[i * BITS / 32] >> (i * BITS % 32));
}

}  // namespace fp8g
