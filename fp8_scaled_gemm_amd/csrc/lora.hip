// lora_add: out[t] = base[t] + scale[a] * B[a] (A[a] x[t]), the adapter a by the
// token's segment.
//
// Two launches, both on the bf16 matrix cores (v_mfma_f32_16x16x32_bf16):
//   shrink  h[t, :] = A[a] x[t], the k axis split over workgroups so that a few
//           tokens still read their adapters with the whole chip; fp32 partial
//           sums in the workspace, one slice a split
//   expand  sums the slices in order (the same result every time), multiplies
//           by scale, and adds B[a] h to base
//
// A block is 16 tokens of one segment (segments.h), the matrix core's N; the
// adapter's rows are its M.  In decode, where every token has its own adapter,
// both kernels are bound by reading A and B once; in prefill by x, base and out.
//
// h goes into the second product as bf16 pieces that add up to it: two (16
// significant bits) for a bf16 result, three (24 bits, all of fp32) for a
// float32 one.  The pieces lie side by side along the product's K, against the
// same columns of B, so nothing but the matrix core pays for them; one piece
// would put an error of 2^-9 of the whole low-rank term into the result.

#include "device_common.h"
#include "launch_block.h"
#include "segments.h"

namespace fp8g {

typedef unsigned int v4u __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int LORA_THREADS = 256;
constexpr int LORA_BLOCK_LOG2 = 4, LORA_BLOCK = 1 << LORA_BLOCK_LOG2;   // tokens a block
constexpr int LORA_MAX_SPLITS = 16;

// The block's tokens [t0, t1) and its adapter (-1: none).  Tokens in front of
// the first segment and behind the last are segments without an adapter.
struct LoraBlock {
    int t0, t1, adapter;
};
__device__ __forceinline__ LoraBlock lora_block(const LoraArgs& a, int id) {
    const int S = a.segments;
    auto start = [&](int v) {   // starts of the S + 2 segments, and the end
        if (v <= 0) return 0;
        if (v > S + 1) return a.tokens;
        return min(max(a.seg_start[v - 1], 0), a.tokens);
    };
    const int v = find_block(start, S + 2, 1, LORA_BLOCK_LOG2, id) - 1;
    const int begin = __builtin_amdgcn_readfirstlane(start(v)), end = __builtin_amdgcn_readfirstlane(start(v + 1));
    LoraBlock b;
    b.t0 = begin + (id - ((begin >> LORA_BLOCK_LOG2) + v)) * LORA_BLOCK;
    b.t1 = min(end, b.t0 + LORA_BLOCK);
    b.adapter = v >= 1 && v <= S ? __builtin_amdgcn_readfirstlane(a.seg_adapter[v - 1]) : -1;
    if (b.adapter >= a.adapters) b.adapter = -1;
    return b;
}

__device__ __forceinline__ bf16x8 load8(const uint16_t* p, bool live) {
    const v4u zero = {0, 0, 0, 0};
    return __builtin_bit_cast(bf16x8, live ? *reinterpret_cast<const v4u*>(p) : zero);
}

template <int RT>   // 16-row tiles of the rank
__global__ __launch_bounds__(LORA_THREADS) void lora_shrink_kernel(LoraArgs a, int splits, int k_split) {
    __shared__ float part[4][RT][16 * 16];
    const int id = blockIdx.x / splits, split = blockIdx.x - id * splits;
    const LoraBlock b = lora_block(a, id);
    if (b.t0 >= b.t1 || b.adapter < 0) return;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, m = lane & 15, g = lane >> 4;
    const int k0 = split * k_split, k1 = min(a.k, k0 + k_split);
    const uint16_t* x = static_cast<const uint16_t*>(a.x) + (int64_t)min(b.t0 + m, b.t1 - 1) * a.k;
    const uint16_t* A = static_cast<const uint16_t*>(a.A) + (int64_t)b.adapter * a.rank * a.k;
    const uint16_t* rows[RT];
    v4f acc[RT];
#pragma unroll
    for (int r = 0; r < RT; r++) {
        rows[r] = A + (int64_t)min(16 * r + m, a.rank - 1) * a.k;
        acc[r] = v4f{0, 0, 0, 0};
    }
#pragma unroll 4
    for (int k = k0 + 32 * wave; k < k1; k += 128) {
        const int at = k + 8 * g;
        const bool live = at < k1;
        const bf16x8 xf = load8(x + at, live);
#pragma unroll
        for (int r = 0; r < RT; r++)
            acc[r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(load8(rows[r] + at, live), xf, acc[r], 0, 0, 0);
    }
    // lane: token m, ranks 16 r + 4 g + i; the four waves' sums meet in LDS
#pragma unroll
    for (int r = 0; r < RT; r++) *reinterpret_cast<v4f*>(&part[wave][r][m * 16 + 4 * g]) = acc[r];
    __syncthreads();
    for (int i = threadIdx.x; i < RT * 256; i += LORA_THREADS) {
        const int r = i >> 8, tok = (i >> 4) & 15, rank = 16 * r + (i & 15);
        const float sum = (part[0][r][i & 255] + part[1][r][i & 255]) + (part[2][r][i & 255] + part[3][r][i & 255]);
        if (rank < a.rank && b.t0 + tok < b.t1)
            a.workspace[((int64_t)split * a.tokens + b.t0 + tok) * a.rank + rank] = sum;
    }
}

template <bool F32>
struct LoraOut {
    // 4 consecutive elements, aligned to their own size only: a row of odd
    // length starts anywhere
    typedef float f4 __attribute__((ext_vector_type(4), aligned(4)));
    typedef uint32_t u2 __attribute__((ext_vector_type(2), aligned(2)));
    static __device__ __forceinline__ v4f load(const char* p) {
        if constexpr (F32) {
            const f4 v = *reinterpret_cast<const f4*>(p);
            return v4f{v[0], v[1], v[2], v[3]};
        } else {
            const u2 v = *reinterpret_cast<const u2*>(p);
            return v4f{__builtin_bit_cast(float, v[0] << 16), __builtin_bit_cast(float, v[0] & 0xFFFF0000u),
                       __builtin_bit_cast(float, v[1] << 16), __builtin_bit_cast(float, v[1] & 0xFFFF0000u)};
        }
    }
    static __device__ __forceinline__ void store(char* p, v4f v) {
        if constexpr (F32)
            *reinterpret_cast<f4*>(p) = f4{v[0], v[1], v[2], v[3]};
        else
            *reinterpret_cast<u2*>(p) = u2{bf16x2_bits(v[0], v[1]), bf16x2_bits(v[2], v[3])};
    }
    static __device__ __forceinline__ float load1(const char* p) {
        if constexpr (F32)
            return *reinterpret_cast<const float*>(p);
        else
            return __builtin_bit_cast(float, (uint32_t)*reinterpret_cast<const uint16_t*>(p) << 16);
    }
    static __device__ __forceinline__ void store1(char* p, float v) {
        if constexpr (F32)
            *reinterpret_cast<float*>(p) = v;
        else
            *reinterpret_cast<uint16_t*>(p) = (uint16_t)(bf16x2_bits(v, 0.0f) & 0xFFFFu);
    }
};

template <bool F32>
__global__ __launch_bounds__(LORA_THREADS) void lora_expand_kernel(LoraArgs a, int splits, int col_blocks, int cols) {
    constexpr int PIECES = F32 ? 3 : 2, ESZ = F32 ? 4 : 2;
    using Out = LoraOut<F32>;
    extern __shared__ uint16_t pieces[];   // [16 tokens][kk], kk = PIECES * rank up to a multiple of 32, + 8
    const int id = blockIdx.x / col_blocks, part = blockIdx.x - id * col_blocks;
    const LoraBlock b = lora_block(a, id);
    if (b.t0 >= b.t1) return;
    const int n0 = part * cols, n1 = min(a.n, n0 + cols);
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, m = lane & 15, g = lane >> 4;
    const int t = b.t0 + m;
    const char* base = static_cast<const char*>(a.base) + (int64_t)t * a.n * ESZ;
    char* out = static_cast<char*>(a.out) + (int64_t)t * a.n * ESZ;
    if (b.adapter < 0) {
        if (a.out == a.base || t >= b.t1) return;
        for (int n = n0 + 64 * wave + 16 * g; n < n1; n += 256)
            for (int q = 0; q < 16 && n + q < n1; q += 4) {
                if (n + q + 4 <= n1)
                    Out::store(out + (int64_t)(n + q) * ESZ, Out::load(base + (int64_t)(n + q) * ESZ));
                else
                    for (int i = n + q; i < n1; i++) Out::store1(out + (int64_t)i * ESZ, Out::load1(base + (int64_t)i * ESZ));
            }
        return;
    }
    const int steps = (PIECES * a.rank + 31) >> 5, row = steps * 32 + 8;
    const float scale = a.scale[b.adapter];
    for (int i = threadIdx.x; i < LORA_BLOCK * a.rank; i += LORA_THREADS) {
        const int tok = i / a.rank, r = i - tok * a.rank;
        float h = 0.0f;
        if (b.t0 + tok < b.t1)
            for (int s = 0; s < splits; s++) h += a.workspace[((int64_t)s * a.tokens + b.t0 + tok) * a.rank + r];
        h *= scale;
#pragma unroll
        for (int p = 0; p < PIECES; p++) {
            const uint32_t bits = bf16x2_bits(h, 0.0f) & 0xFFFFu;
            pieces[tok * row + p * a.rank + r] = (uint16_t)bits;
            h -= __builtin_bit_cast(float, bits << 16);
        }
    }
    const int tail = steps * 32 - PIECES * a.rank;
    for (int i = threadIdx.x; i < LORA_BLOCK * tail; i += LORA_THREADS)
        pieces[(i / tail) * row + PIECES * a.rank + i % tail] = 0;
    __syncthreads();
    const uint16_t* B = static_cast<const uint16_t*>(a.B) + (int64_t)b.adapter * a.n * a.rank;
    for (int n = n0 + 64 * wave; n < n1; n += 256) {
        // tile q, row m of the product: column n + 16 (m / 4) + 4 q + m % 4, so
        // that a lane ends up with 16 consecutive columns of its token
        v4f acc[4];
#pragma unroll
        for (int q = 0; q < 4; q++) acc[q] = v4f{0, 0, 0, 0};
        const int col = n + 16 * (m >> 2) + (m & 3);
        for (int f = 0; f < steps; f++) {
            const int at = 32 * f + 8 * g;
            const bool live = at < PIECES * a.rank;
            int r = at;
            while (r >= a.rank && live) r -= a.rank;
            const bf16x8 h = *reinterpret_cast<const bf16x8*>(&pieces[m * row + at]);
#pragma unroll
            for (int q = 0; q < 4; q++) {
                const bf16x8 w = load8(B + (int64_t)min(col + 4 * q, a.n - 1) * a.rank + r, live);
                acc[q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, h, acc[q], 0, 0, 0);
            }
        }
        if (t < b.t1) {
#pragma unroll
            for (int q = 0; q < 4; q++) {
                const int c = n + 16 * g + 4 * q;
                const int64_t off = (int64_t)c * ESZ;
                if (c + 4 <= n1) {
                    Out::store(out + off, Out::load(base + off) + acc[q]);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; i++)
                        if (c + i < n1) Out::store1(out + off + i * ESZ, Out::load1(base + off + i * ESZ) + acc[q][i]);
                }
            }
        }
    }
}

struct LoraPlan {
    int ids, splits, k_split, col_blocks, cols;
};
static LoraPlan lora_plan(const LoraArgs& a) {
    LoraPlan p;
    p.ids = a.tokens / LORA_BLOCK + a.segments + 2;
    // blocks that certainly have tokens
    const int full = (a.tokens + LORA_BLOCK - 1) / LORA_BLOCK;
    const int blocks = full > a.segments ? full : (a.segments < a.tokens ? a.segments : a.tokens);
    // about two workgroups a CU, of at least 256 of k each
    int splits = (512 + blocks - 1) / blocks;
    const int most = (a.k + 255) / 256;
    splits = splits > most ? most : splits;
    splits = splits > LORA_MAX_SPLITS ? LORA_MAX_SPLITS : splits < 1 ? 1 : splits;
    p.k_split = ((a.k + splits - 1) / splits + 127) / 128 * 128;
    p.splits = a.k > 0 ? (a.k + p.k_split - 1) / p.k_split : 0;
    int col_blocks = (1024 + blocks - 1) / blocks;
    const int most_cols = (a.n + 255) / 256;
    col_blocks = col_blocks > most_cols ? most_cols : col_blocks;
    p.cols = ((a.n + col_blocks - 1) / col_blocks + 255) / 256 * 256;
    p.col_blocks = (a.n + p.cols - 1) / p.cols;
    return p;
}

int64_t lora_add_bytes(const LoraArgs& a) {
    if (a.tokens == 0 || a.n == 0 || a.k == 0 || a.rank == 0) return 0;
    return (int64_t)lora_plan(a).splits * a.tokens * a.rank * 4;
}

template <int RT>
static hipError_t shrink(const LoraArgs& a, const LoraPlan& p, hipStream_t stream) {
    lora_shrink_kernel<RT><<<dim3((unsigned)(p.ids * p.splits)), dim3(LORA_THREADS), 0, stream>>>(a, p.splits, p.k_split);
    return hipGetLastError();
}

hipError_t launch_lora_add(const LoraArgs& in, int f32, hipStream_t stream) {
    LoraArgs a = in;
    if (a.k == 0 || a.rank == 0) a.adapters = 0;   // no low-rank term: every block copies its rows
    const LoraPlan p = lora_plan(a);
    if (a.adapters > 0 && a.segments > 0) {
        hipError_t e;
        if (a.rank <= 16) e = shrink<1>(a, p, stream);
        else if (a.rank <= 32) e = shrink<2>(a, p, stream);
        else if (a.rank <= 64) e = shrink<4>(a, p, stream);
        else if (a.rank <= 128) e = shrink<8>(a, p, stream);
        else e = shrink<16>(a, p, stream);
        if (e != hipSuccess) return e;
    } else if (a.out == a.base) {
        return hipSuccess;
    }
    const int steps = ((f32 ? 3 : 2) * a.rank + 31) / 32;
    const unsigned lds = LORA_BLOCK * (steps * 32 + 8) * 2;
    const dim3 grid((unsigned)(p.ids * p.col_blocks)), block(LORA_THREADS);
    if (f32)
        lora_expand_kernel<true><<<grid, block, lds, stream>>>(a, p.splits, p.col_blocks, p.cols);
    else
        lora_expand_kernel<false><<<grid, block, lds, stream>>>(a, p.splits, p.col_blocks, p.cols);
    return hipGetLastError();
}

}  // namespace fp8g
