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
constexpr int LORA_MAX_SPLITS = 16;

// The block's tokens [t0, t1), at most 16 TT, and its adapter (-1: none).
// Tokens in front of the first segment and behind the last are segments
// without an adapter.
struct LoraBlock {
    int t0, t1, adapter;
};
template <int TT>
__device__ __forceinline__ LoraBlock lora_block(const LoraArgs& a, int id) {
    constexpr int LOG2 = TT == 4 ? 6 : TT == 2 ? 5 : 4;
    const int S = a.segments;
    auto start = [&](int v) {   // starts of the S + 2 segments, and the end
        if (v <= 0) return 0;
        if (v > S + 1) return a.tokens;
        return min(max(a.seg_start[v - 1], 0), a.tokens);
    };
    const Sequence q = find_sequence(
        start, [&](int v) { return v >= 1 && v <= S ? a.seg_adapter[v - 1] : -1; }, S + 2, 1, LOG2, id);
    LoraBlock b;
    b.t0 = q.start + (id - ((q.start >> LOG2) + q.index)) * (16 * TT);
    b.t1 = min(q.end, b.t0 + 16 * TT);
    b.adapter = q.word;
    if (b.adapter >= a.adapters) b.adapter = -1;
    return b;
}

template <int RT, int TT>   // 16-row tiles of the rank, 16-token tiles of a block
__global__ __launch_bounds__(LORA_THREADS, 2) void lora_shrink_kernel(LoraArgs a, int splits, int k_split, int rank_blocks) {
    __shared__ v4f part[2][RT * TT][64];
    const int id = blockIdx.x / (splits * rank_blocks), rest = blockIdx.x - id * splits * rank_blocks;
    const int split = rest / rank_blocks, rank0 = (rest - split * rank_blocks) * (16 * RT);
    const LoraBlock b = lora_block<TT>(a, id);
    if (b.t0 >= b.t1 || b.adapter < 0) return;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, m = lane & 15, g = lane >> 4;
    const int k0 = split * k_split, k1 = min(a.k, k0 + k_split);
    // Row 16 r + m of the adapter; the last 8 rows of a rank that is an odd
    // multiple of 8 are read twice instead of rows that are not there.
    const int ranks = min(a.rank - rank0, 16 * RT);
    const uint16_t* A = static_cast<const uint16_t*>(a.A) + ((int64_t)b.adapter * a.rank + rank0) * a.k + k0 + 8 * g;
    const uint16_t *whole = A + (int64_t)m * a.k, *half = A + (int64_t)(m & 7) * a.k;
    const uint16_t* xs[TT];
    v4f acc[RT][TT];
#pragma unroll
    for (int t = 0; t < TT; t++)
        xs[t] = static_cast<const uint16_t*>(a.x) + (int64_t)min(b.t0 + 16 * t + m, b.t1 - 1) * a.k + k0 + 8 * g;
#pragma unroll
    for (int r = 0; r < RT; r++)
#pragma unroll
        for (int t = 0; t < TT; t++) acc[r][t] = v4f{0, 0, 0, 0};
    // The waves take turns over units of 64 of k (a row's 128-byte line), AHEAD
    // of them at a time and the next ones already on their way.
    constexpr int AHEAD = RT + TT <= 2 ? 4 : RT + TT <= 5 ? 2 : 1;
    struct Unit {
        v4u w[2][RT], x[2][TT];
    };
    auto row = [&](int r) { return (16 * r + 16 <= ranks ? whole : half) + (int64_t)min(16 * r, ranks - 8) * a.k; };
    auto load = [&](Unit& s, int at, bool live0, bool live1) {
#pragma unroll
        for (int t = 0; t < TT; t++) {
            s.x[0][t] = live0 ? *reinterpret_cast<const v4u*>(xs[t] + at) : v4u{0, 0, 0, 0};
            s.x[1][t] = live1 ? *reinterpret_cast<const v4u*>(xs[t] + at + 32) : v4u{0, 0, 0, 0};
        }
#pragma unroll
        for (int r = 0; r < RT; r++) {
            s.w[0][r] = live0 ? *reinterpret_cast<const v4u*>(row(r) + at) : v4u{0, 0, 0, 0};
            s.w[1][r] = live1 ? *reinterpret_cast<const v4u*>(row(r) + at + 32) : v4u{0, 0, 0, 0};
        }
    };
    auto multiply = [&](const Unit& s) {
#pragma unroll
        for (int j = 0; j < 2; j++)
#pragma unroll
            for (int r = 0; r < RT; r++)
#pragma unroll
                for (int t = 0; t < TT; t++)
                    acc[r][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                        __builtin_bit_cast(bf16x8, s.w[j][r]), __builtin_bit_cast(bf16x8, s.x[j][t]), acc[r][t], 0, 0, 0);
    };
    const int full = (k1 - k0) >> 6;
    Unit now[AHEAD];
#pragma unroll
    for (int u = 0; u < AHEAD; u++)
        if (wave + 4 * u < full) load(now[u], 64 * (wave + 4 * u), true, true);
    for (int i = wave; i < full; i += 4 * AHEAD) {
        Unit next[AHEAD];
#pragma unroll
        for (int u = 0; u < AHEAD; u++)
            if (i + 4 * (AHEAD + u) < full) load(next[u], 64 * (i + 4 * (AHEAD + u)), true, true);
#pragma unroll
        for (int u = 0; u < AHEAD; u++) {
            if (i + 4 * u < full) multiply(now[u]);
            now[u] = next[u];
        }
    }
    if (wave == (full & 3) && ((k1 - k0) & 63)) {       // what is left of k, a multiple of 8
        const int at = 64 * full + 8 * g;
        load(now[0], 64 * full, at < k1 - k0, at + 32 < k1 - k0);
        multiply(now[0]);
    }
    // lane: token m, ranks 16 r + 4 g + i.  The waves' sums meet in LDS: 0 + 2
    // and 1 + 3, then both.
    auto put = [&](int at) {
#pragma unroll
        for (int r = 0; r < RT; r++)
#pragma unroll
            for (int t = 0; t < TT; t++) part[at][r * TT + t][lane] = acc[r][t];
    };
    auto add = [&](int at) {
#pragma unroll
        for (int r = 0; r < RT; r++)
#pragma unroll
            for (int t = 0; t < TT; t++) acc[r][t] += part[at][r * TT + t][lane];
    };
    if (wave >= 2) put(wave - 2);
    __syncthreads();
    if (wave < 2) add(wave);
    if (wave == 1) put(1);      // its own slice, read before
    __syncthreads();
    if (wave != 0) return;
    add(1);
#pragma unroll
    for (int t = 0; t < TT; t++) {
        const int tok = b.t0 + 16 * t + m;
        if (tok >= b.t1) continue;
        float* dst = a.workspace + ((int64_t)split * a.tokens + tok) * a.rank + rank0 + 4 * g;
#pragma unroll
        for (int r = 0; r < RT; r++)    // the rank is a multiple of 8: 4 of it are inside or outside
            if (16 * r + 4 * g < ranks) *reinterpret_cast<v4f*>(dst + 16 * r) = acc[r][t];
    }
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

template <bool F32, int TT>
__global__ __launch_bounds__(LORA_THREADS) void lora_expand_kernel(LoraArgs a, int splits, int col_blocks, int cols) {
    constexpr int PIECES = F32 ? 3 : 2, ESZ = F32 ? 4 : 2;
    using Out = LoraOut<F32>;
    constexpr int UNITS = 16 / Out::UNIT;
    extern __shared__ uint16_t pieces[];   // [16 TT tokens][kk], kk = PIECES * rank up to a multiple of 32, + 8
    const int id = blockIdx.x / col_blocks, part = blockIdx.x - id * col_blocks;
    const LoraBlock b = lora_block<TT>(a, id);
    if (b.t0 >= b.t1) return;
    const int n0 = part * cols, n1 = min(a.n, n0 + cols);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, m = lane & 15, g = lane >> 4;
    const char* base = static_cast<const char*>(a.base);
    char* out = static_cast<char*>(a.out);
    if (b.adapter < 0) {
        if (a.out == a.base) return;
        for (int t = b.t0 + wave; t < b.t1; t += 4)
            for (int c = n0 + lane * Out::UNIT; c < n1; c += 64 * Out::UNIT) {
                const int64_t at = ((int64_t)t * a.n + c) * ESZ;
                if (c + Out::UNIT <= n1) {
                    Out::store(out + at, Out::load(base + at));
                } else {
                    for (int i = 0; c + i < n1; i++) Out::add1(out + at + i * ESZ, base + at + i * ESZ, -0.0f);
                }
            }
        return;
    }
    const int steps = (PIECES * a.rank + 31) >> 5, row = steps * 32 + 8;
    const uint16_t* B = static_cast<const uint16_t*>(a.B) + (int64_t)b.adapter * a.n * a.rank;
    // Tile q, row m of the product is column n + 16 (m / 4) + 4 q + m % 4, so
    // that a lane ends up with 16 consecutive columns of its token.
    v4u w[4], old[TT][UNITS];
    const uint16_t* src[4];
    auto load_w = [&](int f) {       // step f: ranks 32 f + 8 g .. of the pieces, which repeat B's
        int r = 32 * f + 8 * g;
        while (r >= a.rank) r -= a.rank;
#pragma unroll
        for (int q = 0; q < 4; q++) w[q] = *reinterpret_cast<const v4u*>(src[q] + r);
    };
    auto load = [&](int n) {
        const int col = n + 16 * (m >> 2) + (m & 3), c0 = n + 16 * g;
#pragma unroll
        for (int q = 0; q < 4; q++) src[q] = B + (int64_t)min(col + 4 * q, a.n - 1) * a.rank;
        load_w(0);
#pragma unroll
        for (int t = 0; t < TT; t++) {
            const int tok = b.t0 + 16 * t + m;
#pragma unroll
            for (int u = 0; u < UNITS; u++)
                if (tok < b.t1 && c0 + (u + 1) * Out::UNIT <= n1)
                    old[t][u] = Out::load(base + ((int64_t)tok * a.n + c0) * ESZ + 16 * u);
        }
    };
    int n = n0 + 64 * wave;
    if (n < n1) load(n);             // on their way while h is put together

    const float scale = a.scale[b.adapter];
    const int quads = a.rank >> 2;
    for (int i = threadIdx.x; i < 16 * TT * quads; i += LORA_THREADS) {
        const int tok = i / quads, r = 4 * (i - tok * quads);
        v4f h = {0, 0, 0, 0};
        if (b.t0 + tok < b.t1)
#pragma unroll 4
            for (int s = 0; s < splits; s++)
                h += *reinterpret_cast<const v4f*>(a.workspace + ((int64_t)s * a.tokens + b.t0 + tok) * a.rank + r);
        h *= scale;
#pragma unroll
        for (int p = 0; p < PIECES; p++) {
            const uint32_t lo = bf16x2_bits(h[0], h[1]), hi = bf16x2_bits(h[2], h[3]);
            uint32_t* dst = reinterpret_cast<uint32_t*>(&pieces[tok * row + p * a.rank + r]);
            dst[0] = lo, dst[1] = hi;
            h -= v4f{__builtin_bit_cast(float, lo << 16), __builtin_bit_cast(float, lo & 0xFFFF0000u),
                     __builtin_bit_cast(float, hi << 16), __builtin_bit_cast(float, hi & 0xFFFF0000u)};
        }
    }
    const int tail = steps * 32 - PIECES * a.rank;
    for (int i = threadIdx.x; i < 16 * TT * tail; i += LORA_THREADS)
        pieces[(i / tail) * row + PIECES * a.rank + i % tail] = 0;
    __syncthreads();
    for (; n < n1; n += 256) {
        v4f acc[TT][4];
#pragma unroll
        for (int t = 0; t < TT; t++)
#pragma unroll
            for (int q = 0; q < 4; q++) acc[t][q] = v4f{0, 0, 0, 0};
        for (int f = 0; f < steps; f++) {
            v4u now[4];
            const bool live = 32 * f + 8 * g < PIECES * a.rank;    // behind the pieces: nothing, whatever B holds
#pragma unroll
            for (int q = 0; q < 4; q++) now[q] = live ? w[q] : v4u{0, 0, 0, 0};
            if (f + 1 < steps) load_w(f + 1);
#pragma unroll
            for (int t = 0; t < TT; t++) {
                const bf16x8 h = *reinterpret_cast<const bf16x8*>(&pieces[(16 * t + m) * row + 32 * f + 8 * g]);
#pragma unroll
                for (int q = 0; q < 4; q++)
                    acc[t][q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, now[q]), h, acc[t][q], 0, 0, 0);
            }
        }
        const int c0 = n + 16 * g;
#pragma unroll
        for (int t = 0; t < TT; t++) {
            const int tok = b.t0 + 16 * t + m;
            if (tok >= b.t1) continue;
            const int64_t at = ((int64_t)tok * a.n + c0) * ESZ;
#pragma unroll
            for (int u = 0; u < UNITS; u++) {
                const int c = c0 + u * Out::UNIT;
                if (c + Out::UNIT <= n1) {
                    Out::store(out + at + 16 * u, Out::add(old[t][u], &acc[t][u * (Out::UNIT / 4)]));
                } else {
#pragma unroll
                    for (int i = 0; i < Out::UNIT; i++)
                        if (c + i < n1)
                            Out::add1(out + at + (u * Out::UNIT + i) * ESZ, base + at + (u * Out::UNIT + i) * ESZ,
                                      acc[t][u * (Out::UNIT / 4) + i / 4][i & 3]);
                }
            }
        }
        if (n + 256 < n1) load(n + 256);
    }
}

struct LoraPlan {
    int tiles, ids, splits, k_split, rank_blocks;    // shrink: 16-token tiles of a block
    int out_tiles, out_ids, col_blocks, cols;        // expand
};
// Blocks of 16 * tiles tokens: their numbers, and how many certainly have tokens.
static int lora_ids(const LoraArgs& a, int tiles) { return a.tokens / (16 * tiles) + a.segments + 2; }
static int lora_blocks(const LoraArgs& a, int tiles) {
    const int full = (a.tokens + 16 * tiles - 1) / (16 * tiles), some = a.segments < a.tokens ? a.segments : a.tokens;
    return full > some ? full : some;
}
static LoraPlan lora_plan(const LoraArgs& a) {
    LoraPlan p;
    // Long segments: blocks of up to 64 tokens read the adapter less often; a
    // wave's sums (rank tiles, 8 at most, times token tiles) stay at 16 tiles.
    const bool wide = a.tokens / (a.segments > 0 ? a.segments : 1) >= 32;
    p.rank_blocks = a.rank > 128 ? 2 : 1;
    p.tiles = !wide ? 1 : a.rank > 64 ? 2 : 4;
    p.ids = lora_ids(a, p.tiles);
    int blocks = lora_blocks(a, p.tiles);
    // about two workgroups a CU, of at least 256 of k each
    int splits = (512 + blocks * p.rank_blocks - 1) / (blocks * p.rank_blocks);
    const int most = (a.k + 255) / 256;
    splits = splits > most ? most : splits;
    splits = splits > LORA_MAX_SPLITS ? LORA_MAX_SPLITS : splits < 1 ? 1 : splits;
    p.k_split = ((a.k + splits - 1) / splits + 127) / 128 * 128;
    p.splits = a.k > 0 ? (a.k + p.k_split - 1) / p.k_split : 0;
    p.out_tiles = wide ? 2 : 1;
    p.out_ids = lora_ids(a, p.out_tiles);
    blocks = lora_blocks(a, p.out_tiles);
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

template <int RT, int TT>
static hipError_t shrink(const LoraArgs& a, const LoraPlan& p, hipStream_t stream) {
    lora_shrink_kernel<RT, TT><<<dim3((unsigned)(p.ids * p.splits * p.rank_blocks)), dim3(LORA_THREADS), 0, stream>>>(
        a, p.splits, p.k_split, p.rank_blocks);
    return hipGetLastError();
}

template <bool F32>
static hipError_t expand(const LoraArgs& a, const LoraPlan& p, hipStream_t stream) {
    const int steps = ((F32 ? 3 : 2) * a.rank + 31) / 32;
    const unsigned lds = 16 * p.out_tiles * (steps * 32 + 8) * 2;
    const dim3 grid((unsigned)(p.out_ids * p.col_blocks)), block(LORA_THREADS);
    if (p.out_tiles == 2)
        lora_expand_kernel<F32, 2><<<grid, block, lds, stream>>>(a, p.splits, p.col_blocks, p.cols);
    else
        lora_expand_kernel<F32, 1><<<grid, block, lds, stream>>>(a, p.splits, p.col_blocks, p.cols);
    return hipGetLastError();
}

hipError_t launch_lora_add(const LoraArgs& in, int f32, hipStream_t stream) {
    LoraArgs a = in;
    if (a.k == 0 || a.rank == 0) a.adapters = 0;   // no low-rank term: every block copies its rows
    const LoraPlan p = lora_plan(a);
    if (a.adapters > 0 && a.segments > 0) {
        hipError_t e;
        // the rank's tiles times the block's are what a wave accumulates
        if (a.rank <= 16) e = p.tiles == 4 ? shrink<1, 4>(a, p, stream) : shrink<1, 1>(a, p, stream);
        else if (a.rank <= 32) e = p.tiles == 4 ? shrink<2, 4>(a, p, stream) : shrink<2, 1>(a, p, stream);
        else if (a.rank <= 64) e = p.tiles == 4 ? shrink<4, 4>(a, p, stream) : shrink<4, 1>(a, p, stream);
        else e = p.tiles == 2 ? shrink<8, 2>(a, p, stream) : shrink<8, 1>(a, p, stream);
        if (e != hipSuccess) return e;
    } else if (a.out == a.base) {
        return hipSuccess;
    }
    return f32 ? expand<true>(a, p, stream) : expand<false>(a, p, stream);
}

}  // namespace fp8g
