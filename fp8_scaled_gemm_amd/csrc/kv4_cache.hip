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
// block of 32 lies in 4 neighbouring lanes, and a thread has 4 of them in flight.
// Keys and values go in one launch.
//
// Measured: 16384 tokens x 16 heads x (192 + 128) bf16, append 47 us, gather 47 us,
// 4.5 TB/s (copies on this part reach 5.8); 57 and 49 before 16 tokens lay side by side,
// four chunks were in flight and divisions were multiplies.

#include "device_common.h"
#include "launch_block.h"
#include "segments.h"

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

constexpr int KV_AHEAD = 4;       // chunks of a thread in flight

// A workgroup's part of a tile: 2^tokens_log2 tokens, for each side and head its
// tokens' chunks one after the other.  A head's rows of neighbouring tokens are
// neighbours in a page, so a tile writes runs of the cache's codes and scales
// that are long and nobody else's.
struct RowsPlan {
    int tokens_log2, k_all, all;              // chunks of a tile: of its keys, and all
    int parts, part;                          // workgroups of a tile, and their chunks
    FastDiv k_chunks, v_chunks, page;
    int wide;                                 // slots of 2^31 and more: divided in 64 bits
};

// Where chunk i (8 elements) of a workgroup's tokens lies: keys first, then
// values.  row < 0: nowhere in the cache.
struct Chunk {
    int64_t t, cell;          // token; page * heads + head
    int row, chunk, dim, head;
    uint8_t *codes, *scales;
    const void* in;
    void* out;
    int64_t stride;
};
__device__ __forceinline__ Chunk chunk_of(const Kv4RowsArgs& a, const RowsPlan& p, int64_t t0, int i) {
    Chunk r;
    const bool v = i >= p.k_all;
    i -= v ? p.k_all : 0;
    // selects of arguments that are in registers, not an indexed load
    r.dim = v ? a.side[1].dim : a.side[0].dim;
    r.codes = v ? a.side[1].codes : a.side[0].codes;
    r.scales = v ? a.side[1].scales : a.side[0].scales;
    r.in = v ? a.in[1] : a.in[0];
    r.out = v ? a.out[1] : a.out[0];
    r.stride = v ? a.stride[1] : a.stride[0];
    const int row = (int)(v ? divide(i, p.v_chunks) : divide(i, p.k_chunks));
    r.chunk = i - row * (r.dim >> 3);
    r.head = row >> p.tokens_log2;
    r.t = t0 + (row & ((1 << p.tokens_log2) - 1));
    return r;
}
__device__ __forceinline__ void place(const Kv4RowsArgs& a, const RowsPlan& p, int64_t slot, Chunk& r) {
    int64_t page;
    if (p.wide) {
        page = slot / a.page_size;
        r.row = (int)(slot - page * a.page_size);
    } else {
        const uint32_t q = divide((uint32_t)slot, p.page);
        page = q;
        r.row = (int)((uint32_t)slot - q * (uint32_t)a.page_size);
    }
    r.cell = page * a.heads + r.head;
    if (slot < 0 || slot >= a.slot_end) r.row = -1;
}

template <bool BF16>
__global__ __launch_bounds__(KV_THREADS) void kv4_append_kernel(Kv4RowsArgs a, RowsPlan p) {
    const int tile = blockIdx.x / p.parts, from = (blockIdx.x - tile * p.parts) * p.part;
    const int64_t t0 = (int64_t)tile << p.tokens_log2;
    const int all = min(p.all, from + p.part);
    for (int i0 = from + threadIdx.x; i0 < all; i0 += KV_AHEAD * KV_THREADS) {
        Chunk c[KV_AHEAD];
        v4u raw[KV_AHEAD][BF16 ? 1 : 2];
        int64_t slot[KV_AHEAD];
#pragma unroll
        for (int u = 0; u < KV_AHEAD; u++) {
            // past the end: the last chunk or token again, not written
            c[u] = chunk_of(a, p, t0, min(i0 + u * KV_THREADS, all - 1));
            const int64_t t = min(c[u].t, (int64_t)a.tokens - 1);
            slot[u] = a.slots[t];
            const int64_t at = t * c[u].stride + (int64_t)c[u].head * c[u].dim + c[u].chunk * 8;
            const v4u* src = reinterpret_cast<const v4u*>(static_cast<const char*>(c[u].in) + at * (BF16 ? 2 : 4));
            raw[u][0] = __builtin_nontemporal_load(src);
            if constexpr (!BF16) raw[u][1] = __builtin_nontemporal_load(src + 1);
        }
#pragma unroll
        for (int u = 0; u < KV_AHEAD; u++) {
            // the four lanes of a block are inside or outside together
            if (i0 + u * KV_THREADS >= all || c[u].t >= a.tokens) continue;
            place(a, p, slot[u], c[u]);
            float x[8];
#pragma unroll
            for (int j = 0; j < 4; j++) {
                if constexpr (BF16) {
                    x[2 * j] = __builtin_bit_cast(float, raw[u][0][j] << 16);
                    x[2 * j + 1] = __builtin_bit_cast(float, raw[u][0][j] & 0xFFFF0000u);
                } else {
                    x[j] = __builtin_bit_cast(v4f, raw[u][0])[j];
                    x[4 + j] = __builtin_bit_cast(v4f, raw[u][BF16 ? 0 : 1])[j];
                }
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
            if (c[u].row < 0) continue;
            *reinterpret_cast<uint32_t*>(c[u].codes + (c[u].cell * a.page_size + c[u].row) * (c[u].dim >> 1) + c[u].chunk * 4) = q;
            if ((c[u].chunk & 3) == 0)
                c[u].scales[(c[u].cell * (c[u].dim >> 5) + (c[u].chunk >> 2)) * a.page_size + c[u].row] = (uint8_t)code;
        }
    }
}

template <bool F32>
__global__ __launch_bounds__(KV_THREADS) void kv4_gather_kernel(Kv4RowsArgs a, RowsPlan p) {
    const int tile = blockIdx.x / p.parts, from = (blockIdx.x - tile * p.parts) * p.part;
    const int64_t t0 = (int64_t)tile << p.tokens_log2;
    const int all = min(p.all, from + p.part);
    for (int i0 = from + threadIdx.x; i0 < all; i0 += KV_AHEAD * KV_THREADS) {
        Chunk c[KV_AHEAD];
        int64_t slot[KV_AHEAD];
        uint32_t q[KV_AHEAD], code[KV_AHEAD];
#pragma unroll
        for (int u = 0; u < KV_AHEAD; u++) {
            c[u] = chunk_of(a, p, t0, min(i0 + u * KV_THREADS, all - 1));
            slot[u] = a.slots[min(c[u].t, (int64_t)a.tokens - 1)];
        }
#pragma unroll
        for (int u = 0; u < KV_AHEAD; u++) {
            place(a, p, slot[u], c[u]);
            q[u] = 0, code[u] = 0;
            if (c[u].row >= 0) {
                q[u] = *reinterpret_cast<const uint32_t*>(c[u].codes + (c[u].cell * a.page_size + c[u].row) * (c[u].dim >> 1) + c[u].chunk * 4);
                code[u] = c[u].scales[(c[u].cell * (c[u].dim >> 5) + (c[u].chunk >> 2)) * a.page_size + c[u].row];
            }
        }
#pragma unroll
        for (int u = 0; u < KV_AHEAD; u++) {
            if (i0 + u * KV_THREADS >= all || c[u].t >= a.tokens) continue;
            const float scale = __builtin_bit_cast(float, code[u] << 23);
            v4u r;
            r[0] = __builtin_bit_cast(uint32_t, (bf16x2_t)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q[u], scale, 0));
            r[1] = __builtin_bit_cast(uint32_t, (bf16x2_t)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q[u], scale, 1));
            r[2] = __builtin_bit_cast(uint32_t, (bf16x2_t)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q[u], scale, 2));
            r[3] = __builtin_bit_cast(uint32_t, (bf16x2_t)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q[u], scale, 3));
            const int64_t at = (c[u].t * a.heads + c[u].head) * c[u].dim + c[u].chunk * 8;
            if constexpr (F32) {
                v4f lo, hi;
#pragma unroll
                for (int j = 0; j < 2; j++) {
                    lo[2 * j] = __builtin_bit_cast(float, r[j] << 16);
                    lo[2 * j + 1] = __builtin_bit_cast(float, r[j] & 0xFFFF0000u);
                    hi[2 * j] = __builtin_bit_cast(float, r[2 + j] << 16);
                    hi[2 * j + 1] = __builtin_bit_cast(float, r[2 + j] & 0xFFFF0000u);
                }
                v4f* dst = reinterpret_cast<v4f*>(static_cast<float*>(c[u].out) + at);
                dst[0] = lo;
                dst[1] = hi;
            } else {
                *reinterpret_cast<v4u*>(static_cast<uint16_t*>(c[u].out) + at) = r;
            }
        }
    }
}

// Few tokens: one a tile.  Many: 16, cut into parts of two full batches of every
// thread or so.
static RowsPlan rows_plan(const Kv4RowsArgs& a, int64_t* blocks) {
    RowsPlan p;
    p.tokens_log2 = a.tokens >= 1024 ? 4 : 0;
    p.k_all = (a.heads * (a.side[0].dim >> 3)) << p.tokens_log2;
    p.all = p.k_all + ((a.heads * (a.side[1].dim >> 3)) << p.tokens_log2);
    const int batch = KV_AHEAD * KV_THREADS;
    p.parts = p.all > 2 * batch ? (p.all + 2 * batch - 1) / (2 * batch) : 1;
    if (p.tokens_log2 == 0) p.parts = (p.all + KV_THREADS - 1) / KV_THREADS;
    p.part = ((p.all + p.parts - 1) / p.parts + KV_THREADS - 1) / KV_THREADS * KV_THREADS;
    p.parts = (p.all + p.part - 1) / p.part;
    p.k_chunks = fast_div(a.side[0].dim >> 3);
    p.v_chunks = fast_div(a.side[1].dim >> 3);
    p.page = fast_div(a.page_size);
    p.wide = a.slot_end > ((int64_t)1 << 31);
    *blocks = ((((int64_t)a.tokens - 1) >> p.tokens_log2) + 1) * p.parts;
    return p;
}

bool kv4_rows_fit(const Kv4RowsArgs& a) {
    int64_t blocks;
    rows_plan(a, &blocks);
    return blocks <= most_blocks(KV_THREADS);
}

hipError_t launch_kv4_append(const Kv4RowsArgs& a, int bf16, hipStream_t stream) {
    int64_t blocks;
    const RowsPlan p = rows_plan(a, &blocks);
    if (bf16)
        kv4_append_kernel<true><<<dim3((unsigned)blocks), dim3(KV_THREADS), 0, stream>>>(a, p);
    else
        kv4_append_kernel<false><<<dim3((unsigned)blocks), dim3(KV_THREADS), 0, stream>>>(a, p);
    return hipGetLastError();
}

hipError_t launch_kv4_gather(const Kv4RowsArgs& a, int f32, hipStream_t stream) {
    int64_t blocks;
    const RowsPlan p = rows_plan(a, &blocks);
    if (f32)
        kv4_gather_kernel<true><<<dim3((unsigned)blocks), dim3(KV_THREADS), 0, stream>>>(a, p);
    else
        kv4_gather_kernel<false><<<dim3((unsigned)blocks), dim3(KV_THREADS), 0, stream>>>(a, p);
    return hipGetLastError();
}

}  // namespace fp8g
