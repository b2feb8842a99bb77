// Sums and maxima over a wave of 64 lanes by data-parallel moves, without LDS
// (gfx950 only).
#pragma once

#include "device_common.h"

namespace fp8g {

// A value that comes from lanes to the left, or `none` where there are none.
template <int CTRL, bool ZERO>
__device__ __forceinline__ float dpp_from(float v, float none) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(__builtin_bit_cast(int, none), __builtin_bit_cast(int, v), CTRL,
                                                                 0xF, 0xF, ZERO));
}
template <int CTRL, bool ZERO>
__device__ __forceinline__ double dpp_from(double v, double none) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v), o = __builtin_bit_cast(uint64_t, none);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp((int)(uint32_t)o, (int)(uint32_t)b, CTRL, 0xF, 0xF, ZERO);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp((int)(uint32_t)(o >> 32), (int)(uint32_t)(b >> 32), CTRL, 0xF, 0xF, ZERO);
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
// a uniform lane's value, as a scalar
__device__ __forceinline__ float from_lane(float v, int lane) {
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}
__device__ __forceinline__ double from_lane(double v, int lane) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, lane);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), lane);
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
__device__ __forceinline__ float larger(float u, float v) { return __builtin_fmaxf(u, v); }
__device__ __forceinline__ double larger(double u, double v) { return __builtin_fmax(u, v); }
// Over the wave: over rows of 16 lanes, then over the four rows; the last lane has
// it all.  A lane without a lane to its left takes itself (largest) or 0 (sum),
// so that each step is one instruction.
// (fp32: the six steps written out, as the compiler takes four instructions for
// one of them; a lane written by the instruction before is read two waits later)
__device__ __forceinline__ float wave_most(float v) {
    asm volatile(
        "s_nop 1\n\tv_max_f32_dpp %0, %0, %0 row_shr:1 row_mask:0xf bank_mask:0xf\n\t"
        "s_nop 1\n\tv_max_f32_dpp %0, %0, %0 row_shr:2 row_mask:0xf bank_mask:0xf\n\t"
        "s_nop 1\n\tv_max_f32_dpp %0, %0, %0 row_shr:4 row_mask:0xf bank_mask:0xf\n\t"
        "s_nop 1\n\tv_max_f32_dpp %0, %0, %0 row_shr:8 row_mask:0xf bank_mask:0xf\n\t"
        "s_nop 1\n\tv_max_f32_dpp %0, %0, %0 row_bcast:15 row_mask:0xf bank_mask:0xf\n\t"
        "s_nop 1\n\tv_max_f32_dpp %0, %0, %0 row_bcast:31 row_mask:0xf bank_mask:0xf\n\t"
        "s_nop 1"
        : "+v"(v));
    return from_lane(v, 63);
}
__device__ __forceinline__ double wave_most(double v) {
    v = larger(v, dpp_from<0x111, false>(v, v));      // row_shr:1, 2, 4, 8
    v = larger(v, dpp_from<0x112, false>(v, v));
    v = larger(v, dpp_from<0x114, false>(v, v));
    v = larger(v, dpp_from<0x118, false>(v, v));
    v = larger(v, dpp_from<0x142, false>(v, v));      // row_bcast:15, 31
    v = larger(v, dpp_from<0x143, false>(v, v));
    return from_lane(v, 63);
}
template <class R>
__device__ __forceinline__ R wave_total(R v) {
    v += dpp_from<0x111, true>(v, (R)0);
    v += dpp_from<0x112, true>(v, (R)0);
    v += dpp_from<0x114, true>(v, (R)0);
    v += dpp_from<0x118, true>(v, (R)0);
    v += dpp_from<0x142, true>(v, (R)0);
    v += dpp_from<0x143, true>(v, (R)0);
    return from_lane(v, 63);
}

}  // namespace fp8g
