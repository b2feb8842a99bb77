// kv4_append and kv4_gather: rows of keys and values to and from a paged MXFP4
// cache (E2M1 codes, one UE8M0 scale for 32 elements of a row).
//
//   e = smallest integer with amax <= 6 * 2^e;  code = E2M1_RNE(x * 2^-e)
//
// With amax = 1.f * 2^(E - 127) (E its exponent field) and 6 = 1.5 * 2^2, e =
// E - 129, one more where the fraction f is above one half: the scale code e +
// 127 = E - 2 + (f > 1/2) comes from the bits of amax, clamped at 0 from below
// (amax < 2^128 keeps it under 254).  The convert instructions take the scale
// as a float whose exponent field is the code and divide (encode) or multiply
// (decode) by 2^(code - 127) exactly, code 0 included; the encode rounds to
// nearest, ties to the even code, and no element is above 6 * 2^e, so it never
// saturates.  Both were checked on every code and at every rounding boundary.
//
// HBM-bound: a lane holds 8 elements (16 bytes of bf16, 4 bytes of codes), a
// block of 32 lies in 4 neighbouring lanes.  Keys and values go in one launch.

#include "device_common.h"
#include "launch_block.h"

namespace fp8g {

typedef unsigned int v4u __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

constexpr int KV_THREADS = 256;

// max over the 4 lanes of a quad, in all of them
__device__ __forceinline__ float quad_max(float v) {
    const int a = __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0xB1, 0xF, 0xF, true);   // lanes 1 0 3 2
    v = __builtin_fmaxf(v, __builtin_bit_cast(float, a));
    const int b = __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x4E, 0xF, 0xF, true);   // lanes 2 3 0 1
    return __builtin_fmaxf(v, __builtin_bit_cast(float, b));
}

// Where chunk `c` (8 elements) of a token's rows lies: keys first, then values.
struct Chunk {
    int side, head, chunk, dim;
    uint8_t *codes, *scales;
    const void* in;
    void* out;
    int64_t stride;
};
__device__ __forceinline__ Chunk chunk_of(const Kv4RowsArgs& a, int c) {
    Chunk r;
    const int per_k = a.side[0].dim >> 3, k_all = per_k * a.heads;
    r.side = c >= k_all;
    const int per = r.side ? a.side[1].dim >> 3 : per_k;
    c -= r.side ? k_all : 0;
    r.head = c / per;
    r.chunk = c - r.head * per;
    // selects of arguments that are in registers, not an indexed load
    r.dim = r.side ? a.side[1].dim : a.side[0].dim;
    r.codes = r.side ? a.side[1].codes : a.side[0].codes;
    r.scales = r.side ? a.side[1].scales : a.side[0].scales;
    r.in = r.side ? a.in[1] : a.in[0];
    r.out = r.side ? a.out[1] : a.out[0];
    r.stride = r.side ? a.stride[1] : a.stride[0];
    return r;
}

template <bool BF16>
__global__ __launch_bounds__(KV_THREADS) void kv4_append_kernel(Kv4RowsArgs a, int per_token, int tokens_per_wg) {
    const int64_t t0 = (int64_t)blockIdx.x * tokens_per_wg;
    const int all = per_token * tokens_per_wg;
    for (int i = threadIdx.x; i < all; i += KV_THREADS) {
        const int sub = i / per_token;
        const int64_t t = t0 + sub;
        if (t >= a.tokens) break;
        const int64_t slot = a.slots[t];
        const Chunk c = chunk_of(a, i - sub * per_token);
        const int64_t at = t * c.stride + (int64_t)c.head * c.dim + c.chunk * 8;
        float x[8];
        if constexpr (BF16) {
            const v4u r = *reinterpret_cast<const v4u*>(static_cast<const uint16_t*>(c.in) + at);
#pragma unroll
            for (int j = 0; j < 4; j++) {
                x[2 * j] = __builtin_bit_cast(float, r[j] << 16);
                x[2 * j + 1] = __builtin_bit_cast(float, r[j] & 0xFFFF0000u);
            }
        } else {
            const v4f* p = reinterpret_cast<const v4f*>(static_cast<const float*>(c.in) + at);
            const v4f lo = p[0], hi = p[1];
#pragma unroll
            for (int j = 0; j < 4; j++) x[j] = lo[j], x[4 + j] = hi[j];
        }
        float m = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; j++) m = __builtin_fmaxf(m, __builtin_fabsf(x[j]));
        const uint32_t bits = __builtin_bit_cast(uint32_t, quad_max(m));
        int code = (int)(bits >> 23) - 2 + ((bits & 0x7FFFFFu) > 0x400000u);
        code = code < 0 ? 0 : code;
        const float scale = __builtin_bit_cast(float, (uint32_t)code << 23);
        uint32_t q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, x[0], x[1], scale, 0);
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, x[2], x[3], scale, 1);
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, x[4], x[5], scale, 2);
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, x[6], x[7], scale, 3);
        if (slot < 0 || slot >= a.slot_end) continue;
        const int64_t page = slot / a.page_size;
        const int row = (int)(slot - page * a.page_size);
        const int64_t ph = page * a.heads + c.head;
        *reinterpret_cast<uint32_t*>(c.codes + (ph * a.page_size + row) * (c.dim >> 1) + c.chunk * 4) = q;
        if ((c.chunk & 3) == 0)
            c.scales[(ph * (c.dim >> 5) + (c.chunk >> 2)) * a.page_size + row] = (uint8_t)code;
    }
}

template <bool F32>
__global__ __launch_bounds__(KV_THREADS) void kv4_gather_kernel(Kv4RowsArgs a, int per_token, int tokens_per_wg) {
    const int64_t t0 = (int64_t)blockIdx.x * tokens_per_wg;
    const int all = per_token * tokens_per_wg;
    for (int i = threadIdx.x; i < all; i += KV_THREADS) {
        const int sub = i / per_token;
        const int64_t t = t0 + sub;
        if (t >= a.tokens) break;
        const int64_t slot = a.slots[t];
        const Chunk c = chunk_of(a, i - sub * per_token);
        uint32_t q = 0, code = 0;
        if (slot >= 0 && slot < a.slot_end) {
            const int64_t page = slot / a.page_size;
            const int row = (int)(slot - page * a.page_size);
            const int64_t ph = page * a.heads + c.head;
            q = *reinterpret_cast<const uint32_t*>(c.codes + (ph * a.page_size + row) * (c.dim >> 1) + c.chunk * 4);
            code = c.scales[(ph * (c.dim >> 5) + (c.chunk >> 2)) * a.page_size + row];
        }
        const float scale = __builtin_bit_cast(float, code << 23);
        v4u r;
        r[0] = __builtin_bit_cast(uint32_t, (bf16x2_t)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 0));
        r[1] = __builtin_bit_cast(uint32_t, (bf16x2_t)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 1));
        r[2] = __builtin_bit_cast(uint32_t, (bf16x2_t)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 2));
        r[3] = __builtin_bit_cast(uint32_t, (bf16x2_t)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 3));
        const int64_t at = (t * a.heads + c.head) * c.dim + c.chunk * 8;
        if constexpr (F32) {
            v4f lo, hi;
#pragma unroll
            for (int j = 0; j < 2; j++) {
                lo[2 * j] = __builtin_bit_cast(float, r[j] << 16);
                lo[2 * j + 1] = __builtin_bit_cast(float, r[j] & 0xFFFF0000u);
                hi[2 * j] = __builtin_bit_cast(float, r[2 + j] << 16);
                hi[2 * j + 1] = __builtin_bit_cast(float, r[2 + j] & 0xFFFF0000u);
            }
            v4f* p = reinterpret_cast<v4f*>(static_cast<float*>(c.out) + at);
            p[0] = lo;
            p[1] = hi;
        } else {
            *reinterpret_cast<v4u*>(static_cast<uint16_t*>(c.out) + at) = r;
        }
    }
}

struct RowsGrid {
    int per_token, tokens_per_wg;
    unsigned blocks;
};
// Enough tokens to give every thread of a workgroup 2 chunks where there are
// many of them, and one token a workgroup where there are few.
static RowsGrid rows_grid(const Kv4RowsArgs& a) {
    RowsGrid g;
    g.per_token = a.heads * ((a.side[0].dim + a.side[1].dim) >> 3);
    g.tokens_per_wg = 1;
    while (g.per_token * g.tokens_per_wg < 2 * KV_THREADS && a.tokens / (g.tokens_per_wg * 2) >= 512)
        g.tokens_per_wg *= 2;
    g.blocks = (unsigned)(((int64_t)a.tokens + g.tokens_per_wg - 1) / g.tokens_per_wg);
    return g;
}

hipError_t launch_kv4_append(const Kv4RowsArgs& a, int bf16, hipStream_t stream) {
    const RowsGrid g = rows_grid(a);
    if (bf16)
        kv4_append_kernel<true><<<dim3(g.blocks), dim3(KV_THREADS), 0, stream>>>(a, g.per_token, g.tokens_per_wg);
    else
        kv4_append_kernel<false><<<dim3(g.blocks), dim3(KV_THREADS), 0, stream>>>(a, g.per_token, g.tokens_per_wg);
    return hipGetLastError();
}

hipError_t launch_kv4_gather(const Kv4RowsArgs& a, int f32, hipStream_t stream) {
    const RowsGrid g = rows_grid(a);
    if (f32)
        kv4_gather_kernel<true><<<dim3(g.blocks), dim3(KV_THREADS), 0, stream>>>(a, g.per_token, g.tokens_per_wg);
    else
        kv4_gather_kernel<false><<<dim3(g.blocks), dim3(KV_THREADS), 0, stream>>>(a, g.per_token, g.tokens_per_wg);
    return hipGetLastError();
}

}  // namespace fp8g
