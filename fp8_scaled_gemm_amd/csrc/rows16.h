// Rows of bf16 or fp32 elements in vectors of 16 bytes (gfx950 only).
#pragma once

#include "device_common.h"

namespace fp8g {

typedef unsigned int v4u __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));

template <bool F32>
struct Row16 {
    static constexpr int VEC = F32 ? 4 : 8;   // elements of 16 bytes
    static __device__ __forceinline__ void unpack(v4u r, float* f) {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            if constexpr (F32) {
                // the vector as a whole: a bit cast of one element of it reads element 0
                f[i] = __builtin_bit_cast(v4f, r)[i];
            } else {
                f[2 * i] = __builtin_bit_cast(float, r[i] << 16);
                f[2 * i + 1] = __builtin_bit_cast(float, r[i] & 0xFFFF0000u);
            }
        }
    }
    static __device__ __forceinline__ v4u pack(const float* f) {
        v4u r;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            if constexpr (F32)
                r[i] = __builtin_bit_cast(uint32_t, f[i]);
            else
                r[i] = bf16x2_bits(f[2 * i], f[2 * i + 1]);
        }
        return r;
    }
};

}  // namespace fp8g
