// lora_add: out[t] = base[t] + scale[a] * B[a] (A[a] x[t]), the adapter a by the
// token's segment.
//
// Two launches, both on the bf16 matrix cores (v_mfma_f32_16x16x32_bf16):
//   shrink  h[t, :] = scale[a] * A[a] x[t].  A workgroup takes a block of tokens
//           of one segment (segments.h), up to 64 or 128 rows of the adapter
//           and a part of k; its waves take turns over k and meet in LDS.  The
//           parts of k leave fp32 sums in the workspace, one slice each.
//   expand  out = base + B[a] h, with h the sum of the slices in order (the same
//           result every time).
// Decode, where every token has its own adapter, reads A and B once; prefill is
// bound by x, base and out.
//
// h enters the second product as bf16 pieces that add up to it: two (16
// significant bits) for a bf16 result, three (24 bits, all of fp32) for a
// float32 one; one piece would put an error of 2^-9 of the low-rank term into
// the result.
//
// A matrix-core operand wants 16 bytes of 16 different rows in neighbouring
// lanes.  Loaded like that from memory, every lane is a cache access of its own
// and a CU gets 16 bytes a clock (measured, from L1 and L2 alike), against 28
// for 64-byte and 45 for whole runs.  So shrink, and expand for long segments,
// load whole 128-byte lines and turn them around in LDS.
//
// Measured: 8192 tokens, 7 segments, k 8192, n 2048, rank 64, bf16: shrink 34 us (x
// read once: 3.9 TB/s), expand 26 us; 64 adapters of rank 16 for 64 tokens, k = n =
// 4096: 5.0 and 6.5 us, of which reading A and B takes 2.7 at a large copy's rate.

#include "device_common.h"
#include "launch_block.h"
#include "segments.h"

namespace fp8g {

typedef unsigned int v4u __attribute__((ext_vector_type(4)));
typedef unsigned int v2u __attribute__((ext_vector_type(2)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int LORA_THREADS = 256;

// The block's tokens [t0, t1), at most 64 or 16, and its adapter (-1: none).
// Tokens in front of the first segment and behind the last are segments
// without an adapter.
struct LoraBlock {
    int t0, t1, adapter;
};
template <bool WIDE>
__device__ __forceinline__ LoraBlock lora_block(const LoraArgs& a, int id) {
    constexpr int LOG2 = WIDE ? 6 : 4;
    const int S = a.segments;
    auto start = [&](int v) {   // starts of the S + 2 segments, and the end
        if (v <= 0) return 0;
        if (v > S + 1) return a.tokens;
        return min(max(a.seg_start[v - 1], 0), a.tokens);
    };
    const Sequence q = find_sequence(
        start, [&](int v) { return v >= 1 && v <= S ? a.seg_adapter[v - 1] : -1; }, S + 2, 1, LOG2, id);
    LoraBlock b;
    b.t0 = q.start + (id - ((q.start >> LOG2) + q.index)) * (1 << LOG2);
    b.t1 = min(q.end, b.t0 + (1 << LOG2));
    b.adapter = q.word;
    if (b.adapter >= a.adapters) b.adapter = -1;
    return b;
}

// Chunk c (16 bytes) of row m of a 16-row, 128-byte tile in LDS: neighbouring
// even and odd rows fill the banks once, the exchange keeps reads of one chunk
// of 16 rows off each other's banks.
__device__ __forceinline__ int tile_at(int m, int c) { return m * 8 + (c ^ ((m >> 1) & 7)); }

// Short segments: 16 tokens a block, RT 16-row tiles of the rank; the waves
// take turns over units of 64 k, each on its own.
template <int RT>
__global__ __launch_bounds__(LORA_THREADS, 2) void lora_shrink_kernel(LoraArgs a, int splits, int k_split, int rank_blocks) {
    __shared__ v4u tiles[4][RT + 1][128];      // a wave's own; then the waves' sums
    // A block's parts lie 8 workgroups apart: on one XCD, whose L2 they share.
    const int parts = splits * rank_blocks, line = blockIdx.x >> 3;
    const int id = (line / parts) * 8 + (blockIdx.x & 7), rest = line % parts;
    const int split = rest / rank_blocks, rank0 = (rest - split * rank_blocks) * (16 * RT);
    const LoraBlock b = lora_block<false>(a, id);
    if (b.t0 >= b.t1 || b.adapter < 0) return;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, m = lane & 15, g = lane >> 4;
    const int k0 = split * k_split, len = min(a.k - k0, k_split);
    // The lane loads chunk lane % 8 of rows lane / 8 and lane / 8 + 8 of a tile.
    // The last 8 rows of a rank that is an odd multiple of 8 are read twice
    // instead of rows that are not there.
    const int lr = lane >> 3, lc = lane & 7;
    const int ranks = min(a.rank - rank0, 16 * RT);
    const uint16_t* A = static_cast<const uint16_t*>(a.A) + ((int64_t)b.adapter * a.rank + rank0 + lr) * a.k + k0 + 8 * lc;
    const uint16_t* x[2];
#pragma unroll
    for (int e = 0; e < 2; e++)
        x[e] = static_cast<const uint16_t*>(a.x) + (int64_t)min(b.t0 + 8 * e + lr, b.t1 - 1) * a.k + k0 + 8 * lc;
    v4f acc[RT];
#pragma unroll
    for (int r = 0; r < RT; r++) acc[r] = v4f{0, 0, 0, 0};
    // Units of 64 of k, AHEAD of them at a time and the next on their way.
    constexpr int AHEAD = RT == 1 ? 4 : RT == 2 ? 2 : 1;
    struct Unit {
        v4u w[RT][2], x[2];
    };
    auto load = [&](Unit& s, int at, bool live) {
#pragma unroll
        for (int e = 0; e < 2; e++) s.x[e] = live ? *reinterpret_cast<const v4u*>(x[e] + at) : v4u{0, 0, 0, 0};
#pragma unroll
        for (int r = 0; r < RT; r++)
#pragma unroll
            for (int e = 0; e < 2; e++)
                s.w[r][e] = live ? *reinterpret_cast<const v4u*>(A + (int64_t)min(16 * r + 8 * e, ranks - 8) * a.k + at) : v4u{0, 0, 0, 0};
    };
    auto multiply = [&](const Unit& s) {
        v4u(*tile)[128] = tiles[wave];
#pragma unroll
        for (int e = 0; e < 2; e++) {
#pragma unroll
            for (int r = 0; r < RT; r++) tile[r][tile_at(8 * e + lr, lc)] = s.w[r][e];
            tile[RT][tile_at(8 * e + lr, lc)] = s.x[e];
        }
#pragma unroll
        for (int j = 0; j < 2; j++) {
            const bf16x8 xf = __builtin_bit_cast(bf16x8, tile[RT][tile_at(m, 4 * j + g)]);
#pragma unroll
            for (int r = 0; r < RT; r++) {
                const bf16x8 w = __builtin_bit_cast(bf16x8, tile[r][tile_at(m, 4 * j + g)]);
                acc[r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, xf, acc[r], 0, 0, 0);
            }
        }
    };
    const int full = len >> 6;
    Unit now[AHEAD];
#pragma unroll
    for (int u = 0; u < AHEAD; u++)
        if (wave + 4 * u < full) load(now[u], 64 * (wave + 4 * u), true);
    for (int i = wave; i < full; i += 4 * AHEAD) {
        Unit next[AHEAD];
#pragma unroll
        for (int u = 0; u < AHEAD; u++)
            if (i + 4 * (AHEAD + u) < full) load(next[u], 64 * (i + 4 * (AHEAD + u)), true);
#pragma unroll
        for (int u = 0; u < AHEAD; u++) {
            if (i + 4 * u < full) multiply(now[u]);
            now[u] = next[u];
        }
    }
    if (wave == (full & 3) && (len & 63)) {         // what is left of k, a multiple of 8
        load(now[0], 64 * full, 64 * full + 8 * lc < len);
        multiply(now[0]);
    }
    // lane: token m, ranks 16 r + 4 g + i.  The waves' sums meet in LDS, in order.
    v4f* sums = reinterpret_cast<v4f*>(tiles);
    __syncthreads();
#pragma unroll
    for (int r = 0; r < RT; r++) sums[(wave * RT + r) * 64 + lane] = acc[r];
    __syncthreads();
    const float scale = a.scale[b.adapter];
    for (int i = threadIdx.x; i < RT * 64; i += LORA_THREADS) {
        const int tile = i >> 6, l = i & 63;
        const v4f h = ((sums[i] + sums[RT * 64 + i]) + (sums[2 * RT * 64 + i] + sums[3 * RT * 64 + i])) * scale;
        const int tok = b.t0 + (l & 15), rank = 16 * tile + 4 * (l >> 4);
        if (tok < b.t1 && rank < ranks)             // ranks is a multiple of 8: 4 of them are inside or outside
            *reinterpret_cast<v4f*>(a.workspace + ((int64_t)split * a.tokens + tok) * a.rank + rank0 + rank) = h;
    }
}

// Long segments: a block of 64 tokens, 16 of them a wave.  The waves share
// the adapter's tile of a unit of 64 k in LDS, so that it crosses the caches
// once a block, and turn their own tokens' tiles around in LDS of their own.
// DEPTH units are in flight in registers.  Blocks of 128 tokens, which read the
// adapter half as often but need more slices of k to fill the chip, took 59 instead of
// 62 us with expand at 8192 tokens, k 8192, rank 64, n 2048, and 37 instead of 34 at 4096
// tokens, k 4096, rank 32, n 5120.
template <int RT>
__global__ __launch_bounds__(LORA_THREADS, 2) void lora_shrink_wide_kernel(LoraArgs a, int splits, int k_split, int rank_blocks) {
    constexpr int DEPTH = 4;
    constexpr int NA = RT * 128 < LORA_THREADS ? 1 : RT * 128 / LORA_THREADS;   // chunks of the adapter's tile a thread
    __shared__ v4u at_tile[2][RT * 128];
    __shared__ v4u x_tile[4][128];
    const int parts = splits * rank_blocks, line = blockIdx.x >> 3;
    const int id = (line / parts) * 8 + (blockIdx.x & 7), rest = line % parts;
    const int split = rest / rank_blocks, rank0 = (rest - split * rank_blocks) * (16 * RT);
    const LoraBlock b = lora_block<true>(a, id);
    if (b.t0 >= b.t1 || b.adapter < 0) return;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, m = lane & 15, g = lane >> 4;
    const int k0 = split * k_split, len = min(a.k - k0, k_split);
    const int lr = lane >> 3, lc = lane & 7, t0 = b.t0 + 16 * wave;
    const int ranks = min(a.rank - rank0, 16 * RT);
    const uint16_t* A = static_cast<const uint16_t*>(a.A) + ((int64_t)b.adapter * a.rank + rank0) * a.k + k0 + 8 * lc;
    const uint16_t *arow[NA], *x[2];
#pragma unroll
    for (int e = 0; e < NA; e++) arow[e] = A + (int64_t)min((int)(threadIdx.x >> 3) + 32 * e, ranks - 1) * a.k;
#pragma unroll
    for (int e = 0; e < 2; e++)
        x[e] = static_cast<const uint16_t*>(a.x) + (int64_t)min(t0 + 8 * e + lr, b.t1 - 1) * a.k + k0 + 8 * lc;
    v4f acc[RT];
#pragma unroll
    for (int r = 0; r < RT; r++) acc[r] = v4f{0, 0, 0, 0};
    struct Unit {
        v4u w[NA], x[2];
    };
    const int units = (len + 63) >> 6;
    auto load = [&](Unit& s, int u) {
        const int at = 64 * u;
        const bool live = at + 8 * lc < len;         // k is a multiple of 8
#pragma unroll
        for (int e = 0; e < 2; e++) s.x[e] = live ? *reinterpret_cast<const v4u*>(x[e] + at) : v4u{0, 0, 0, 0};
#pragma unroll
        for (int e = 0; e < NA; e++) s.w[e] = live ? *reinterpret_cast<const v4u*>(arow[e] + at) : v4u{0, 0, 0, 0};
    };
    Unit ring[DEPTH];
#pragma unroll
    for (int d = 0; d < DEPTH; d++)
        if (d < units) load(ring[d], d);
    for (int u0 = 0; u0 < units; u0 += DEPTH) {
#pragma unroll
        for (int d = 0; d < DEPTH; d++) {
            const int u = u0 + d;
            if (u >= units) break;
            // this buffer was left by every wave before the last barrier
            v4u* const tile = at_tile[u & 1];
#pragma unroll
            for (int e = 0; e < NA; e++) {
                const int r = (threadIdx.x >> 3) + 32 * e;
                if (r < 16 * RT) tile[(r & ~15) * 8 + tile_at(r & 15, lc)] = ring[d].w[e];
            }
#pragma unroll
            for (int e = 0; e < 2; e++) x_tile[wave][tile_at(8 * e + lr, lc)] = ring[d].x[e];
            if (u + DEPTH < units) load(ring[d], u + DEPTH);
            __syncthreads();
#pragma unroll
            for (int j = 0; j < 2; j++) {
                const bf16x8 xf = __builtin_bit_cast(bf16x8, x_tile[wave][tile_at(m, 4 * j + g)]);
#pragma unroll
                for (int r = 0; r < RT; r++) {
                    const bf16x8 w = __builtin_bit_cast(bf16x8, tile[r * 128 + tile_at(m, 4 * j + g)]);
                    acc[r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, xf, acc[r], 0, 0, 0);
                }
            }
        }
    }
    // lane: token m, ranks 16 r + 4 g + i
    const float scale = a.scale[b.adapter];
    const int tok = t0 + m;
    if (tok >= b.t1) return;
    float* dst = a.workspace + ((int64_t)split * a.tokens + tok) * a.rank + rank0 + 4 * g;
#pragma unroll
    for (int r = 0; r < RT; r++)    // ranks is a multiple of 8: 4 of them are inside or outside
        if (16 * r + 4 * g < ranks) *reinterpret_cast<v4f*>(dst + 16 * r) = acc[r] * scale;
}

// 16 bytes of a row of base or out: UNIT consecutive elements, aligned to
// their own size only (a row of odd length starts anywhere).
template <bool F32>
struct LoraOut {
    static constexpr int UNIT = F32 ? 4 : 8, ESZ = F32 ? 4 : 2;
    typedef uint32_t u4 __attribute__((ext_vector_type(4), aligned(2)));
    static __device__ __forceinline__ v4u load(const char* p) {
        const u4 v = *reinterpret_cast<const u4*>(p);
        return v4u{v[0], v[1], v[2], v[3]};
    }
    static __device__ __forceinline__ void store(char* p, v4u v) { *reinterpret_cast<u4*>(p) = u4{v[0], v[1], v[2], v[3]}; }
    static __device__ __forceinline__ v4u add(v4u v, const v4f* d) {
        if constexpr (F32) {
            return __builtin_bit_cast(v4u, __builtin_bit_cast(v4f, v) + d[0]);
        } else {
            v4u r;
#pragma unroll
            for (int i = 0; i < 4; i++)
                r[i] = bf16x2_bits(__builtin_bit_cast(float, v[i] << 16) + d[i >> 1][(2 * i) & 3],
                                   __builtin_bit_cast(float, v[i] & 0xFFFF0000u) + d[i >> 1][(2 * i + 1) & 3]);
            return r;
        }
    }
    static __device__ __forceinline__ void add1(char* dst, const char* src, float d) {
        if constexpr (F32)
            *reinterpret_cast<float*>(dst) = *reinterpret_cast<const float*>(src) + d;
        else
            *reinterpret_cast<uint16_t*>(dst) =
                (uint16_t)bf16x2_bits(__builtin_bit_cast(float, (uint32_t)*reinterpret_cast<const uint16_t*>(src) << 16) + d, 0.0f);
    }
};

// out = base for a block without an adapter.
template <bool F32>
__device__ __forceinline__ void copy_block(const LoraArgs& a, const LoraBlock& b, int n0, int n1) {
    using Out = LoraOut<F32>;
    if (a.out == a.base) return;
    const char* base = static_cast<const char*>(a.base);
    char* out = static_cast<char*>(a.out);
    const int units = (n1 - n0 + Out::UNIT - 1) / Out::UNIT, all = (b.t1 - b.t0) * units;
    constexpr int AHEAD = 8;
    for (int i0 = threadIdx.x; i0 < all; i0 += AHEAD * LORA_THREADS) {
        v4u v[AHEAD];
        int64_t at[AHEAD];
        int left[AHEAD];       // elements of the unit that the row still has
#pragma unroll
        for (int u = 0; u < AHEAD; u++) {
            const int i = i0 + u * LORA_THREADS, t = i / units, c = n0 + (i - t * units) * Out::UNIT;
            left[u] = i < all ? n1 - c : 0;
            at[u] = ((int64_t)(b.t0 + t) * a.n + c) * Out::ESZ;
            if (left[u] >= Out::UNIT) v[u] = Out::load(base + at[u]);
        }
#pragma unroll
        for (int u = 0; u < AHEAD; u++) {
            if (left[u] >= Out::UNIT) {
                Out::store(out + at[u], v[u]);
            } else {
                for (int e = 0; e < left[u]; e++) Out::add1(out + at[u] + e * Out::ESZ, base + at[u] + e * Out::ESZ, -0.0f);
            }
        }
    }
}

// h of a block's tokens in LDS, as bf16 pieces: row = pieces * rank elements up
// to a multiple of `fill`, zeros behind them, and 8 more that keep rows off each
// other's banks.  The slices are summed in order.  All pieces but the last are cut
// to bf16's finite range: what would round to infinity leaves its rest to the next
// one, and an infinite or NaN h passes on to the last (infinity less infinity would
// make a NaN of it).
template <int PIECES, int ITEMS, int SLICES>   // so many loads of a thread in flight
__device__ __forceinline__ void stage_pieces(const LoraArgs& a, const LoraBlock& b, int splits, uint16_t* pieces, int tokens,
                                             int stride, int row) {
    const int quads = a.rank >> 2;
    const int64_t slice = (int64_t)a.tokens * a.rank;
    for (int i0 = threadIdx.x; i0 < tokens * quads; i0 += ITEMS * LORA_THREADS) {
        v4f h[ITEMS];
        const float* p[ITEMS];
        int tok[ITEMS], r[ITEMS];
#pragma unroll
        for (int e = 0; e < ITEMS; e++) {
            const int i = i0 + e * LORA_THREADS;
            tok[e] = i / quads, r[e] = 4 * (i - tok[e] * quads);
            p[e] = a.workspace + (int64_t)min(b.t0 + tok[e], b.t1 - 1) * a.rank + r[e];
            h[e] = v4f{0, 0, 0, 0};
        }
        for (int s = 0; s < splits; s += SLICES) {
            v4f v[SLICES][ITEMS];
#pragma unroll
            for (int u = 0; u < SLICES; u++)
                if (s + u < splits) {
#pragma unroll
                    for (int e = 0; e < ITEMS; e++)
                        if (i0 + e * LORA_THREADS < tokens * quads) v[u][e] = *reinterpret_cast<const v4f*>(p[e] + (s + u) * slice);
                }
#pragma unroll
            for (int u = 0; u < SLICES; u++)
                if (s + u < splits) {
#pragma unroll
                    for (int e = 0; e < ITEMS; e++) h[e] += v[u][e];
                }
        }
#pragma unroll
        for (int e = 0; e < ITEMS; e++) {
            if (i0 + e * LORA_THREADS >= tokens * quads) break;
#pragma unroll
            for (int q = 0; q < PIECES; q++) {
                auto piece = [&](float v) {
                    return q + 1 < PIECES ? __builtin_amdgcn_fmed3f(v, -0x1.FEp127f, 0x1.FEp127f) : v;
                };
                const uint32_t lo = bf16x2_bits(piece(h[e][0]), piece(h[e][1])), hi = bf16x2_bits(piece(h[e][2]), piece(h[e][3]));
                *reinterpret_cast<v2u*>(&pieces[tok[e] * row + q * stride + r[e]]) = v2u{lo, hi};
                h[e] -= v4f{__builtin_bit_cast(float, lo << 16), __builtin_bit_cast(float, lo & 0xFFFF0000u),
                            __builtin_bit_cast(float, hi << 16), __builtin_bit_cast(float, hi & 0xFFFF0000u)};
            }
        }
    }
}

// Short segments: 16 tokens a block, every wave on its own 64 columns, whose
// base and first part of B travel while h is put together.  The pieces of h lie
// side by side along the product's K, against the same ranks of B: a rank of 16
// fills it with two.
template <bool F32>
__global__ __launch_bounds__(LORA_THREADS) void lora_expand_kernel(LoraArgs a, int splits, int col_blocks, int cols) {
    constexpr int PIECES = F32 ? 3 : 2;
    using Out = LoraOut<F32>;
    constexpr int UNITS = 16 / Out::UNIT, ESZ = Out::ESZ;
    extern __shared__ uint16_t pieces[];
    const int id = blockIdx.x / col_blocks, part = blockIdx.x - id * col_blocks;
    const LoraBlock b = lora_block<false>(a, id);
    if (b.t0 >= b.t1) return;
    const int n0 = part * cols, n1 = min(a.n, n0 + cols);
    if (b.adapter < 0) return copy_block<F32>(a, b, n0, n1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, m = lane & 15, g = lane >> 4;
    const char* base = static_cast<const char*>(a.base);
    char* out = static_cast<char*>(a.out);
    const int kk = PIECES * a.rank, steps = (kk + 31) >> 5, row = steps * 32 + 8;
    const uint16_t* B = static_cast<const uint16_t*>(a.B) + (int64_t)b.adapter * a.n * a.rank;
    const int tok = min(b.t0 + m, b.t1 - 1);
    // Tile q, row m of the product is column n + 16 (m / 4) + 4 q + m % 4, so
    // that a lane ends up with 16 consecutive columns of its token.
    v4u w[4], old[UNITS];
    const uint16_t* src[4];
    auto load_w = [&](int f) {       // step f: ranks 32 f + 8 g .. of the pieces, which repeat B's
        int r = 32 * f + 8 * g;
        while (r >= a.rank) r -= a.rank;
#pragma unroll
        for (int q = 0; q < 4; q++) w[q] = *reinterpret_cast<const v4u*>(src[q] + r);
    };
    auto load = [&](int n) {
        const int col = n + 16 * (m >> 2) + (m & 3);
#pragma unroll
        for (int q = 0; q < 4; q++) src[q] = B + (int64_t)min(col + 4 * q, a.n - 1) * a.rank;
        load_w(0);
#pragma unroll
        for (int u = 0; u < UNITS; u++) {
            // the row's last whole unit stands in for one that crosses its end
            const int c = min(n + 16 * g + u * Out::UNIT, max(a.n - Out::UNIT, 0));
            old[u] = a.n >= Out::UNIT ? Out::load(base + ((int64_t)tok * a.n + c) * ESZ) : v4u{0, 0, 0, 0};
        }
    };
    int n = n0 + 64 * wave;
    if (n < n1) load(n);
    stage_pieces<PIECES, 1, 8>(a, b, splits, pieces, 16, a.rank, row);
    const int tail = steps * 32 - kk;
    for (int i = threadIdx.x; i < 16 * tail; i += LORA_THREADS) pieces[(i / tail) * row + kk + i % tail] = 0;
    __syncthreads();
    for (; n < n1; n += 256) {
        v4f acc[4];
#pragma unroll
        for (int q = 0; q < 4; q++) acc[q] = v4f{0, 0, 0, 0};
        for (int f = 0; f < steps; f++) {
            v4u now[4];
            const bool live = 32 * f + 8 * g < kk;    // behind the pieces: nothing, whatever B holds
#pragma unroll
            for (int q = 0; q < 4; q++) now[q] = live ? w[q] : v4u{0, 0, 0, 0};
            if (f + 1 < steps) load_w(f + 1);
            const bf16x8 h = *reinterpret_cast<const bf16x8*>(&pieces[m * row + 32 * f + 8 * g]);
#pragma unroll
            for (int q = 0; q < 4; q++)
                acc[q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, now[q]), h, acc[q], 0, 0, 0);
        }
        if (b.t0 + m < b.t1) {
            const int c0 = n + 16 * g;
            const int64_t at = ((int64_t)tok * a.n + c0) * ESZ;
#pragma unroll
            for (int u = 0; u < UNITS; u++) {
                const int c = c0 + u * Out::UNIT;
                if (c + Out::UNIT <= n1) {
                    Out::store(out + at + 16 * u, Out::add(old[u], &acc[u * (Out::UNIT / 4)]));
                } else {
#pragma unroll
                    for (int i = 0; i < Out::UNIT; i++)
                        if (c + i < n1)
                            Out::add1(out + at + (u * Out::UNIT + i) * ESZ, base + at + (u * Out::UNIT + i) * ESZ,
                                      acc[u * (Out::UNIT / 4) + i / 4][i & 3]);
                }
            }
        }
        if (n + 256 < n1) load(n + 256);
    }
}

// Long segments: 64 tokens a block, 16 of them a wave.  The waves share a tile
// of 128 columns by 64 ranks of B in LDS, the next one on its way in registers;
// h lies in LDS, too.  Here the tokens are the product's M: lane (n, g) gets columns 8 n .. 8 n + 7 (tile q: column 8 n + q) of tokens
// 4 g + i, so that 16 lanes read and write 256 or 512 bytes of a row.
template <bool F32>
__global__ __launch_bounds__(LORA_THREADS, F32 ? 2 : 3) void lora_expand_wide_kernel(LoraArgs a, int splits, int col_blocks, int cols) {
    constexpr int PIECES = F32 ? 3 : 2, TILE = 128;
    using Out = LoraOut<F32>;
    constexpr int UNITS = 8 / Out::UNIT, ESZ = Out::ESZ;
    __shared__ v4u tiles[2][TILE * 8];
    extern __shared__ uint16_t pieces[];
    const int line = blockIdx.x >> 3;      // a block's column parts: on one XCD, which then holds its h
    const int id = (line / col_blocks) * 8 + (blockIdx.x & 7), part = line % col_blocks;
    const LoraBlock b = lora_block<true>(a, id);
    if (b.t0 >= b.t1) return;
    const int n0 = part * cols, n1 = min(a.n, n0 + cols);
    if (b.adapter < 0) return copy_block<F32>(a, b, n0, n1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, m = lane & 15, g = lane >> 4;
    const char* base = static_cast<const char*>(a.base);
    char* out = static_cast<char*>(a.out);
    const uint16_t* B = static_cast<const uint16_t*>(a.B) + (int64_t)b.adapter * a.n * a.rank;
    const int rank_steps = (a.rank + 63) >> 6, strips = (n1 - n0 + TILE - 1) / TILE;
    // B's tile: thread t loads chunk t % 8 of columns t / 8 + 32 e
    const int lc = threadIdx.x & 7, lr = threadIdx.x >> 3;
    v4u w[4];
    auto load = [&](int n, int r0) {
        const bool live = r0 + 8 * lc < a.rank;
#pragma unroll
        for (int e = 0; e < 4; e++)
            w[e] = live ? *reinterpret_cast<const v4u*>(B + (int64_t)min(n + lr + 32 * e, a.n - 1) * a.rank + r0 + 8 * lc) : v4u{0, 0, 0, 0};
    };
    // column c lies in row 16 (c % 8) + c / 8: the 16 columns of a product tile
    // are 16 neighbouring rows
    auto keep = [&](int buffer) {
#pragma unroll
        for (int e = 0; e < 4; e++) {
            const int c = lr + 32 * e, row = 16 * (c & 7) + (c >> 3);
            tiles[buffer][(row & ~15) * 8 + tile_at(row & 15, lc)] = w[e];
        }
    };
    const int tok = b.t0 + 16 * wave;
    v4u old[4][UNITS], soon[4][UNITS];
    auto load_base = [&](v4u (&old)[4][UNITS], int n) {
        const int last = max(a.n - Out::UNIT, 0);
#pragma unroll
        for (int i = 0; i < 4; i++)
#pragma unroll
            for (int u = 0; u < UNITS; u++)
                old[i][u] = a.n >= Out::UNIT ? Out::load(base + ((int64_t)min(tok + 4 * g + i, b.t1 - 1) * a.n +
                                                                 min(n + 8 * m + u * Out::UNIT, last)) * ESZ)
                                             : v4u{0, 0, 0, 0};
    };
    load(n0, 0);
    load_base(old, n0);
    // pieces of h: each from a multiple of 64 on, zeros behind the rank
    const int stride = rank_steps * 64, row = PIECES * stride + 8;
    stage_pieces<PIECES, 4, 2>(a, b, splits, pieces, 64, stride, row);
#pragma unroll
    for (int p = 0; p < PIECES; p++)    // rank and stride are multiples of 8: 16 bytes at a time, 4 threads a token
        for (int r = a.rank + 8 * (threadIdx.x & 3); r < stride; r += 32)
            *reinterpret_cast<v4u*>(&pieces[(threadIdx.x >> 2) * row + p * stride + r]) = v4u{0, 0, 0, 0};
    const uint16_t* h = pieces + (16 * wave + m) * row + 8 * g;
    int buffer = 0;
    for (int strip = 0; strip < strips; strip++) {
        const int n = n0 + strip * TILE;
        if (strip + 1 < strips) load_base(soon, n + TILE);
        v4f acc[8];
#pragma unroll
        for (int q = 0; q < 8; q++) acc[q] = v4f{0, 0, 0, 0};
        for (int rs = 0; rs < rank_steps; rs++, buffer ^= 1) {
            // the other buffer may still be read; this one was left two steps ago
            keep(buffer);
            __syncthreads();
            if (rs + 1 < rank_steps) load(n, 64 * (rs + 1));
            else if (strip + 1 < strips) load(n + TILE, 0);
#pragma unroll
            for (int j = 0; j < 2; j++) {
                if (64 * rs + 32 * j >= a.rank) break;
                bf16x8 x[PIECES];
#pragma unroll
                for (int p = 0; p < PIECES; p++) x[p] = *reinterpret_cast<const bf16x8*>(h + p * stride + 64 * rs + 32 * j);
#pragma unroll
                for (int q = 0; q < 8; q++) {
                    const bf16x8 v = __builtin_bit_cast(bf16x8, tiles[buffer][16 * q * 8 + tile_at(m, 4 * j + g)]);
#pragma unroll
                    for (int p = 0; p < PIECES; p++)
                        acc[q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[p], v, acc[q], 0, 0, 0);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int t = tok + 4 * g + i;
            if (t >= b.t1) continue;
#pragma unroll
            for (int u = 0; u < UNITS; u++) {
                const int c = n + 8 * m + u * Out::UNIT;
                const int64_t at = ((int64_t)t * a.n + c) * ESZ;
                v4f d[2];
#pragma unroll
                for (int e = 0; e < Out::UNIT; e++) d[e >> 2][e & 3] = acc[u * Out::UNIT + e][i];
                if (c + Out::UNIT <= n1) {
                    Out::store(out + at, Out::add(old[i][u], d));
                } else {
#pragma unroll
                    for (int e = 0; e < Out::UNIT; e++)
                        if (c + e < n1) Out::add1(out + at + e * ESZ, base + at + e * ESZ, d[e >> 2][e & 3]);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 4; i++)
#pragma unroll
            for (int u = 0; u < UNITS; u++) old[i][u] = soon[i][u];
    }
}

// Blocks of 16 * tiles tokens: their numbers, and how many certainly have tokens.
static int lora_ids(const LoraArgs& a, int tiles) { return a.tokens / (16 * tiles) + a.segments + 2; }
static int lora_blocks(const LoraArgs& a, int tiles) {
    const int full = (a.tokens + 16 * tiles - 1) / (16 * tiles), some = a.segments < a.tokens ? a.segments : a.tokens;
    return full > some ? full : some;
}
// The forms for long segments, by the average segment.  Shrink + expand, us, wide
// against narrow, k 4096, n 2048 (4096 tokens) or 4096 (the others):
//   4096 tokens, rank 64:  8 tokens a segment 90 / 71, 16: 54 / 66, 64: 33 / 42
//   4096 tokens, rank 16:  16: 42 / 39, 64: 27 / 24, 128: 19 / 24
//   4096 tokens, rank 8:   128: 19 / 25
//   4096 tokens, rank 32:  16: 43 / 44, 32: 27 / 28;  1024 tokens: 64: 20 / 16
//   1024 tokens, rank 64:  128: 19 / 22;  256 tokens in one: 14 / 12;  64: 13 / 11
static bool lora_wide(const LoraArgs& a) {
    const int segment = a.tokens / (a.segments > 0 ? a.segments : 1);
    return a.tokens >= 512 && segment >= (a.rank > 32 ? 16 : 128);
}

struct LoraPlan {
    int tiles, splits, k_split, rank_blocks;
};
static LoraPlan lora_plan(const LoraArgs& a) {
    LoraPlan p;
    p.tiles = lora_wide(a) ? 4 : 1;
    p.rank_blocks = a.rank <= 64 ? 1 : p.tiles > 1 ? (a.rank + 63) / 64 : (a.rank + 127) / 128;
    const int blocks = lora_blocks(a, p.tiles) * p.rank_blocks;
    // two workgroups a CU at once, of at least 256 of k each
    // expand reads every slice of h in each of its column parts: 16 instead of 8
    // cost a wide one 2 to 4 us of 16; with 4 shrink loses what expand gains
    const int max_splits = p.tiles > 1 ? 8 : 16;
    int splits = 512 / blocks;
    int most = (a.k + 255) / 256;
    most = most > max_splits ? max_splits : most;
    splits = splits > most ? most : splits;
    const int64_t room = most_blocks(LORA_THREADS) / (((int64_t)lora_ids(a, p.tiles) + 7) / 8 * 8 * p.rank_blocks);
    splits = splits > room ? (int)room : splits;
    splits = splits < 1 ? 1 : splits;             // k may be 0
    p.k_split = ((a.k + splits - 1) / splits + 127) / 128 * 128;
    p.splits = a.k > 0 ? (a.k + p.k_split - 1) / p.k_split : 0;
    return p;
}

int64_t lora_add_bytes(const LoraArgs& a) {
    if (a.tokens == 0 || a.n == 0 || a.k == 0 || a.rank == 0) return 0;
    return (int64_t)lora_plan(a).splits * a.tokens * a.rank * 4;
}

bool lora_add_fits(const LoraArgs& a) {
    if (a.tokens == 0 || a.n == 0) return true;
    const int tiles = lora_wide(a) ? 4 : 1;
    return ((int64_t)lora_ids(a, tiles) + 7) / 8 * 8 * lora_plan(a).rank_blocks <= most_blocks(LORA_THREADS);
}

template <int RT>
static hipError_t shrink(const LoraArgs& a, const LoraPlan& p, hipStream_t stream) {
    const dim3 grid((unsigned)(((int64_t)lora_ids(a, p.tiles) + 7) / 8 * 8 * p.splits * p.rank_blocks)), block(LORA_THREADS);
    if (p.tiles == 1) {
        lora_shrink_kernel<RT><<<grid, block, 0, stream>>>(a, p.splits, p.k_split, p.rank_blocks);
    } else {
        constexpr int R = RT < 4 ? RT : 4;      // rank blocks of 64
        lora_shrink_wide_kernel<R><<<grid, block, 0, stream>>>(a, p.splits, p.k_split, p.rank_blocks);
    }
    return hipGetLastError();
}

template <bool F32>
static hipError_t expand(const LoraArgs& a, const LoraPlan& p, hipStream_t stream) {
    const bool wide = lora_wide(a);
    const int tiles = wide ? 4 : 1, blocks = lora_blocks(a, tiles), unit = wide ? 128 : 256;
    // wide: what fits on the chip at once, three workgroups a CU (expand of 8192
    // tokens, rank 64, n 4096: 34 us; two a CU 38, four 39).  narrow: 2048 in all,
    // as its workgroups live short (a quarter or half of that is slower).
    int col_blocks = wide ? 768 / blocks : (2048 + blocks - 1) / blocks;
    if (col_blocks < 1) col_blocks = 1;
    const int most = (a.n + unit - 1) / unit;
    col_blocks = col_blocks > most ? most : col_blocks;
    const int ids = lora_ids(a, tiles);
    const int64_t room = most_blocks(LORA_THREADS) / (((int64_t)ids + 7) / 8 * 8);      // more segments than tokens
    col_blocks = col_blocks > room ? (int)room : col_blocks;
    const int cols = ((a.n + col_blocks - 1) / col_blocks + unit - 1) / unit * unit;
    col_blocks = (a.n + cols - 1) / cols;
    const dim3 block(LORA_THREADS);
    const int pieces = F32 ? 3 : 2;
    if (wide) {
        const unsigned lds = 64 * (pieces * ((a.rank + 63) / 64 * 64) + 8) * 2;
        lora_expand_wide_kernel<F32><<<dim3((unsigned)(((int64_t)ids + 7) / 8 * 8 * col_blocks)), block, lds, stream>>>(a, p.splits, col_blocks, cols);
    } else {
        const unsigned lds = 16 * ((pieces * a.rank + 31) / 32 * 32 + 8) * 2;
        lora_expand_kernel<F32><<<dim3((unsigned)((int64_t)ids * col_blocks)), block, lds, stream>>>(a, p.splits, col_blocks, cols);
    }
    return hipGetLastError();
}

hipError_t launch_lora_add(const LoraArgs& in, int f32, hipStream_t stream) {
    LoraArgs a = in;
    if (a.k == 0 || a.rank == 0) a.adapters = 0;   // no low-rank term: every block copies its rows
    const LoraPlan p = lora_plan(a);
    if (a.adapters > 0 && a.segments > 0) {
        const hipError_t e = a.rank <= 16 ? shrink<1>(a, p, stream) : a.rank <= 32 ? shrink<2>(a, p, stream)
                           : a.rank <= 64 ? shrink<4>(a, p, stream) : shrink<8>(a, p, stream);
        if (e != hipSuccess) return e;
    } else if (a.out == a.base) {
        return hipSuccess;
    }
    return f32 ? expand<true>(a, p, stream) : expand<false>(a, p, stream);
}

}  // namespace fp8g
