// kv4_attention: attention over the paged MXFP4 cache.
//
// For a query row q (one query of one head) and the keys it sees,
//   s_j = scale q . k_j,   out = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m)
// in one pass over the keys with the running maximum m and sum l.
//
// A workgroup takes 16 rows -- the group of query heads that share a key head,
// and neighbouring queries of a sequence where that leaves room -- and a chunk
// of the sequence's keys.  Its four waves take 64 keys at a time each, on their
// own (no barrier inside the loop), and join their maxima, sums and outputs at
// the end.  Chunks, cut where few rows would leave the chip idle, leave their
// partial results in the workspace; a second kernel joins them in order.
//
// Both products run transposed on v_mfma_f32_16x16x32_bf16, so that the result
// layout of the first is the operand layout of the second and softmax weights
// never leave their lane:
//   S^T[key, row] = K Q^T,   O^T[dim, row] = V^T P^T
// with the row as the matrix core's N: lane l holds row l % 16, g = l / 16.
// * Keys: lane (m, g) is row m of the first operand and takes the 16 bytes of
//   dims 32 g .. 32 g + 31 (one scale) of a key; the four 8-dim pieces are its
//   operands of four products.  The order of dims along K is free as long as
//   the queries follow it.
// * In a step of 64 keys, product tile i (of 4) takes keys 4 m + i: the lane's
//   four keys are neighbours (4 scales in one load), and the result holds, in
//   lane group g, the 16 neighbouring keys 16 g + 4 r + i.
// * Values: lane (m, g) takes dims 8 m .. 8 m + 7 of those 16 keys (4 bytes
//   each, 16 scales in one load) and turns 8 keys x 8 dims into eight operands
//   with one convert and one byte permute for each pair of elements.
// * Codes come as they lie in memory, 16 keys of a head in one run of 512 to 1536
//   bytes, and each wave turns them around in LDS of its own: loads in operand
//   order touch 64 places each and kept the address unit of a CU busier than
//   its memory.  While a step is computed from LDS the next one's codes travel
//   into the registers that it came from.
// E2M1 with a power-of-two scale is exact in bf16, one convert instruction for
// two elements; only the softmax weights are rounded (to bf16), as the second
// product's operand: in two pieces they would double its matrix instructions.
// Their sum takes them unrounded.  Error against 64 bits, of the size of the result:
// 0.0019 to 0.0023, of which rounding the result to bf16 makes 0.0017.
//
// Measured: 64 sequences of 4165 to 16384 keys, 64 heads over 8 key heads, dims 128:
// 159 us a call over many calls, 164 as the profiler's median of a dispatch: 4.4 to 4.5
// TB/s of codes and scales, where this part reads at up to 6.6.  These loads without the
// arithmetic took 147 us, the arithmetic alone 110: one step of a wave is in flight.
// One query of 32 heads on 2048 keys: 5.8 us and 3.0 to join.

#include "device_common.h"
#include "launch_block.h"
#include "segments.h"

#include <type_traits>

namespace fp8g {

typedef unsigned int v4u __attribute__((ext_vector_type(4)));
typedef unsigned int v2u __attribute__((ext_vector_type(2)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2v __attribute__((ext_vector_type(2)));

constexpr int ATTN_THREADS = 256;
constexpr int ATTN_ROWS_LOG2 = 4, ATTN_ROWS = 1 << ATTN_ROWS_LOG2;
constexpr int ATTN_STEP = 64;                      // keys of a wave's step
constexpr int ATTN_CHUNK = 4 * ATTN_STEP;          // keys of a workgroup's step
constexpr int ATTN_LONGEST = 16384;                // keys of a chunk, where there are splits enough
constexpr float ATTN_SLACK = 8.0f;                 // growth of a maximum that is left to the weights, in powers of two

// fill: chunks of a block's keys that fill the chip; splits: the most that it can have
struct AttnPlan {
    int ids, fill, splits;
    FastDiv page, by_fill, by_splits;
};

// Two E2M1 elements (byte SEL of codes) times 2^(scale - 127), as bf16.
template <int SEL>
__device__ __forceinline__ uint32_t fp4x2(uint32_t codes, float scale) {
    return __builtin_bit_cast(uint32_t, (bf16x2v)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, SEL));
}
__device__ __forceinline__ bf16x8 fp4x8(uint32_t codes, float scale) {
    const v4u r = {fp4x2<0>(codes, scale), fp4x2<1>(codes, scale), fp4x2<2>(codes, scale), fp4x2<3>(codes, scale)};
    return __builtin_bit_cast(bf16x8, r);
}
// UE8M0 code in byte i of w, as a float
template <int I>
__device__ __forceinline__ float scale_of(uint32_t w) {
    uint32_t r;
    if constexpr (I == 3) r = (w >> 1) & 0x7F800000u;
    else if constexpr (I == 2) r = (w << 7) & 0x7F800000u;
    else if constexpr (I == 1) r = (w << 15) & 0x7F800000u;
    else r = (w << 23) & 0x7F800000u;
    return __builtin_bit_cast(float, r);
}
// max over lanes l and l ^ 32: the swap leaves the lower half's values in both
// halves of one register, the upper half's in both of the other
__device__ __forceinline__ float across_halves(float v) {
    const uint32_t u = __builtin_bit_cast(uint32_t, v);
    const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    return __builtin_fmaxf(__builtin_bit_cast(float, (uint32_t)r[0]), __builtin_bit_cast(float, (uint32_t)r[1]));
}

__device__ __forceinline__ float over_groups_max(float v) {
    const uint32_t u = __builtin_bit_cast(uint32_t, v);
    const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);    // lanes l and l ^ 16
    return across_halves(__builtin_fmaxf(__builtin_bit_cast(float, (uint32_t)r[0]), __builtin_bit_cast(float, (uint32_t)r[1])));
}
__device__ __forceinline__ float over_groups_sum(float v) {
    v += __shfl_xor(v, 16, 64);
    return v + __shfl_xor(v, 32, 64);
}

// Chunk `split` of the keys [lo, hi) that a block sees: equal parts of whole
// workgroup steps.  The lengths are known here only; the host knows no more than
// how wide the page table is.
struct AttnPart {
    int begin, end;
};
template <bool SPLIT>
__device__ __forceinline__ AttnPart attn_part(const AttnPlan& p, int split, int lo, int hi) {
    const int from = lo & ~(ATTN_STEP - 1);
    if (!SPLIT) return AttnPart{from, hi};
    const int steps = (max(hi - from, 0) + ATTN_CHUNK - 1) / ATTN_CHUNK;
    int per = (int)divide(steps + p.fill - 1, p.by_fill);
    if (per > ATTN_LONGEST / ATTN_CHUNK) per = max(ATTN_LONGEST / ATTN_CHUNK, (int)divide(steps + p.splits - 1, p.by_splits));
    // in steps, of which there are at most 2^22; known to be the workgroup's, or the
    // 256-row kernel would keep them in vector registers, of which it has none left
    const int first = (int)min((int64_t)split * per, (int64_t)steps), last = min(first + per, steps);
    return AttnPart{__builtin_amdgcn_readfirstlane(from + first * ATTN_CHUNK),
                    __builtin_amdgcn_readfirstlane(last < steps ? from + last * ATTN_CHUNK : hi)};
}

// A maximum of -inf alone does not say that a row has seen nothing: maxima drop
// NaN, and a row of nothing but NaN scores has one, too, with a sum of NaN.  Its
// part goes to the join with a maximum of NaN, where -inf stands for no part.
__device__ __forceinline__ bool saw_nothing(float m, float l) { return m == -INFINITY && l == 0.0f; }
__device__ __forceinline__ float part_max(float m, float l) {
    return m == -INFINITY && !saw_nothing(m, l) ? __builtin_nanf("") : m;
}

// What a block of rows sees.
struct AttnBlock {
    int seq, row0, rows, q0, queries, kv;
};
template <int ROWS_LOG2>
__device__ __forceinline__ bool attn_block(const Kv4AttnArgs& a, int group, int id, AttnBlock& b) {
    auto start = [&](int i) { return min(max(a.q_start[i], 0), a.queries); };
    const Sequence s = find_sequence(start, [&](int i) { return a.kv_len[i]; }, a.batch, group, ROWS_LOG2, id);
    if (s.index < 0) return false;
    b.seq = s.index;
    b.q0 = s.start;
    b.queries = s.end - s.start;
    b.row0 = (id - ((int)(((int64_t)b.q0 * group) >> ROWS_LOG2) + b.seq)) << ROWS_LOG2;
    b.rows = b.queries * group;
    const int64_t room = (int64_t)a.max_pages * a.page_size;
    b.kv = (int)min((int64_t)max(s.word, 0), room);
    return b.row0 < b.rows;
}

// A wave's codes of a step in LDS.  Keys: 16-byte chunks, exchanged within groups
// of 8 or 16 so that reads of one chunk of keys 4 apart meet different banks.
// Values: a run of 16 keys and 64 bytes, so that the four runs do, too.
template <int DK, int DV>
struct AttnTile {
    static constexpr int K_CHUNKS = DK / 32, K_BYTES = ATTN_STEP * DK / 2;
    static constexpr int V_RUN = 16 * DV / 2 + 64, BYTES = K_BYTES + 4 * V_RUN;
    static __device__ __forceinline__ int key_at(int chunk) {      // chunk = key * K_CHUNKS + c
        const int m = chunk / (4 * K_CHUNKS);
        return 16 * (DK == 128 ? chunk ^ (m & 15) : chunk ^ ((m >> 1) & 7));
    }
};

template <int DK, int DV, bool SPLIT>
__global__ __launch_bounds__(ATTN_THREADS, 2) void kv4_attention_kernel(Kv4AttnArgs a, AttnPlan p) {
    constexpr int KW = DK / 32, DT = DV / 16;   // products along the head dim; 16-dim tiles of the output
    typedef AttnTile<DK, DV> Tile;
    // the waves' tiles; at the end their outputs
    constexpr int SHARED = 4 * Tile::BYTES > 4 * ATTN_ROWS * (DV + 4) * 4 ? 4 * Tile::BYTES : 4 * ATTN_ROWS * (DV + 4) * 4;
    __shared__ __attribute__((aligned(16))) uint8_t shared[SHARED];
    __shared__ float s_m[4][ATTN_ROWS], s_l[4][ATTN_ROWS];
    float(*const s_o)[ATTN_ROWS][DV + 4] = reinterpret_cast<float(*)[ATTN_ROWS][DV + 4]>(shared);
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
    const int group = a.q_heads / a.kv_heads;
    // Chunk by chunk: workgroups go to the XCDs in turn, and later chunks, which
    // shorter sequences do not have, would otherwise all fall to the same ones.
    const int blocks = p.ids * a.kv_heads, split = blockIdx.x / blocks, rest = blockIdx.x - split * blocks;
    const int h = rest % a.kv_heads, id = rest / a.kv_heads;
    AttnBlock b;
    if (!attn_block<ATTN_ROWS_LOG2>(a, group, id, b)) return;

    // the lane's row, its query and the keys [lo, hi) that it sees
    const int row = b.row0 + n;
    const bool real = row < b.rows;
    const int qi = min(row, b.rows - 1) / group;
    const int head = h * group + min(row, b.rows - 1) % group;
    const int first = b.kv - b.queries;      // position of query 0
    auto top_of = [&](int q) { return a.causal ? max(0, min(b.kv, first + q + 1)) : b.kv; };
    auto low_of = [&](int q) { return a.window ? max(0, first + q + 1 - a.window) : 0; };
    const int hi = real ? top_of(qi) : 0, lo = low_of(qi);
    const int q_first = b.row0 / group, q_last = (min(b.row0 + ATTN_ROWS, b.rows) - 1) / group;
    const int all_lo = min(low_of(q_first), b.kv), all_hi = top_of(q_last);   // of the union
    const int in_lo = low_of(q_last), in_hi = top_of(q_first);                // of the intersection
    const AttnPart part = attn_part<SPLIT>(p, split, all_lo, all_hi);
    const int begin = part.begin, end = part.end;
    const int64_t out_row = (int64_t)(b.q0 + qi) * a.q_heads + head;
    float* const part_o = a.workspace;
    float* const part_ml = a.workspace + (int64_t)a.queries * a.q_heads * p.splits * DV;
    if (SPLIT && begin >= end) {
        if (threadIdx.x < ATTN_ROWS && real) part_ml[(out_row * p.splits + split) * 2] = -INFINITY;
        return;
    }

    // A negative scale turns the queries' signs, so that the largest product is
    // the largest score; a scale of zero becomes one that changes nothing and
    // keeps -inf * scale at -inf; a scale of NaN becomes that, too, and turns the
    // queries to NaN, so that rows without keys stay without.
    const float c2 = __builtin_fmaxf(__builtin_fabsf(a.scale) * 1.4426950408889634f, 0x1p-120f);
    // queries: dims in the order of the keys' pieces
    bf16x8 q[KW];
    {
        const uint32_t flip = a.scale < 0.0f ? 0x80008000u : 0u, spoil = a.scale != a.scale ? 0x7FFF7FFFu : 0u;
        const uint16_t* src = static_cast<const uint16_t*>(a.q) + (int64_t)(b.q0 + qi) * a.q_stride + (int64_t)head * DK;
#pragma unroll
        for (int j = 0; j < KW; j++) {
            const int d = DK == 64 ? 16 * g + 8 * j : (j < 4 ? 32 * g + 8 * j : 128 + 16 * g + 8 * (j - 4));
            const v4u w = *reinterpret_cast<const v4u*>(src + d);
            q[j] = __builtin_bit_cast(bf16x8, v4u{(w[0] ^ flip) | spoil, (w[1] ^ flip) | spoil, (w[2] ^ flip) | spoil, (w[3] ^ flip) | spoil});
        }
    }

    // A step is four runs of 16 keys, each in one page.  Lane l looks up run l % 4;
    // the entries are asked for a step before the codes, and in front of the
    // codes of the step before, so that waiting for them does not wait for those.
    const int32_t* table = a.page_table + (int64_t)b.seq * a.max_pages;
    // cells (a row of a head) of a page, and of the heads in front of this one
    const int64_t page_cells = (int64_t)a.kv_heads * a.page_size, head_cells = (int64_t)h * a.page_size;
    const uint8_t* const k_codes = a.k_codes + head_cells * (DK / 2);
    const uint8_t* const k_scales = a.k_scales + head_cells * (DK / 32);
    const uint8_t* const v_codes = a.v_codes + head_cells * (DV / 2);
    const uint8_t* const v_scales = a.v_scales + head_cells * (DV / 32);
    const int last_page = a.pages - 1, last_slot = a.max_pages - 1;
    struct Run {
        int64_t cell;      // the page's first
        int at;            // the run's row in the page
    };
    auto look = [&](int base) { return table[min((int)divide(base + 16 * (lane & 3), p.page), last_slot)]; };
    auto run_of = [&](int entry, int base, int r) {
        const int page = min(max(__builtin_amdgcn_readlane(entry, r), 0), last_page), key = base + 16 * r;
        return Run{page * page_cells, key - (int)divide(key, p.page) * a.page_size};
    };
    struct Step {
        v4u k[DK / 32], v[DV / 32], vs;
        uint32_t ks[DK == 192 ? 2 : 1];
    };
    // the lane's scales: keys 4 n .. (run n / 4) of its groups of dims; values: run g
    const int ks0 = (DK == 64 ? g >> 1 : g) * a.page_size + 4 * (n & 3), ks1 = (4 + (g >> 1)) * a.page_size + 4 * (n & 3);
    const int vs0 = (DV == 64 ? n >> 3 : n >> 2) * a.page_size;
    auto pick = [](int64_t x0, int64_t x1, int64_t x2, int64_t x3, int r) {
        const int64_t lo = r & 1 ? x1 : x0, hi = r & 1 ? x3 : x2;
        return r & 2 ? hi : lo;
    };
    int entry = 0;
    auto load = [&](Step& s, int base) {
        Run run[4];
        int64_t ks_at[4], vs_at[4];
#pragma unroll
        for (int r = 0; r < 4; r++) {
            run[r] = run_of(entry, base, r);
            ks_at[r] = run[r].cell * (DK / 32) + run[r].at;
            vs_at[r] = run[r].cell * (DV / 32) + run[r].at;
        }
        entry = look(base + ATTN_CHUNK);        // behind the last page: its last entry, unused
        // load j, half e: 512 bytes, part (2 j + e) % (DIM / 64) of run (2 j + e) / (DIM / 64)
        auto codes = [&](auto dim, const uint8_t* from, v4u* to) {
            constexpr int DIM = decltype(dim)::value, PER = DIM / 64;
#pragma unroll
            for (int j = 0; j < DIM / 32; j++) {
                const Run &r0 = run[2 * j / PER], &r1 = run[(2 * j + 1) / PER];
                const int64_t p0 = (r0.cell + r0.at) * (DIM / 2) + 2 * j % PER * 512;
                const int64_t p1 = (r1.cell + r1.at) * (DIM / 2) + (2 * j + 1) % PER * 512 - 512;
                const uint8_t* src = from + (2 * j / PER == (2 * j + 1) / PER ? p0 : lane < 32 ? p0 : p1);
                to[j] = *reinterpret_cast<const v4u*>(src + (uint32_t)(16 * lane));
            }
        };
        codes(std::integral_constant<int, DK>{}, k_codes, s.k);
        codes(std::integral_constant<int, DV>{}, v_codes, s.v);
        const uint8_t* sc = k_scales + pick(ks_at[0], ks_at[1], ks_at[2], ks_at[3], n >> 2);
        s.ks[0] = *reinterpret_cast<const uint32_t*>(sc + ks0);
        if constexpr (DK == 192) s.ks[1] = *reinterpret_cast<const uint32_t*>(sc + ks1);
        s.vs = *reinterpret_cast<const v4u*>(v_scales + pick(vs_at[0], vs_at[1], vs_at[2], vs_at[3], g) + vs0);
    };
    uint8_t* const tile = shared + wave * Tile::BYTES;
    auto keep = [&](const Step& s) {
#pragma unroll
        for (int j = 0; j < DK / 32; j++) *reinterpret_cast<v4u*>(tile + Tile::key_at(64 * j + lane)) = s.k[j];
#pragma unroll
        for (int j = 0; j < DV / 32; j++) {
            const int half = 2 * j + (lane >> 5), run = half / (DV / 64), part = half % (DV / 64);
            *reinterpret_cast<v4u*>(tile + Tile::K_BYTES + run * Tile::V_RUN + 512 * part + 16 * (lane & 31)) = s.v[j];
        }
    };

    v4f o[DT];
#pragma unroll
    for (int d = 0; d < DT; d++) o[d] = v4f{0, 0, 0, 0};
    float m = -INFINITY, l = 0.0f;

    // what a step still needs beside the codes in LDS
    auto step = [&](const uint32_t (&ks)[DK == 192 ? 2 : 1], v4u vs, int base) {
        // scores
        v4f acc[4];
#pragma unroll
        for (int i = 0; i < 4; i++) acc[i] = v4f{0, 0, 0, 0};
        const float k0[4] = {scale_of<0>(ks[0]), scale_of<1>(ks[0]), scale_of<2>(ks[0]), scale_of<3>(ks[0])};
        uint32_t kc[4][KW];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int chunk = (4 * n + i) * Tile::K_CHUNKS;
            if constexpr (DK == 64) {
                const v2u w = *reinterpret_cast<const v2u*>(tile + Tile::key_at(chunk + (g >> 1)) + 8 * (g & 1));
                kc[i][0] = w[0], kc[i][1] = w[1];
            } else {
                const v4u w = *reinterpret_cast<const v4u*>(tile + Tile::key_at(chunk + g));
#pragma unroll
                for (int j = 0; j < 4; j++) kc[i][j] = w[j];
                if constexpr (DK == 192) {
                    const v2u x = *reinterpret_cast<const v2u*>(tile + Tile::key_at(chunk + 4 + (g >> 1)) + 8 * (g & 1));
                    kc[i][4] = x[0], kc[i][5] = x[1];
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 4; i++) {
#pragma unroll
            for (int j = 0; j < (KW < 4 ? KW : 4); j++)
                acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fp4x8(kc[i][j], k0[i]), q[j], acc[i], 0, 0, 0);
        }
        if constexpr (DK == 192) {
            const float k1[4] = {scale_of<0>(ks[1]), scale_of<1>(ks[1]), scale_of<2>(ks[1]), scale_of<3>(ks[1])};
#pragma unroll
            for (int i = 0; i < 4; i++) {
#pragma unroll
                for (int j = 4; j < 6; j++)
                    acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fp4x8(kc[i][j], k1[i]), q[j], acc[i], 0, 0, 0);
            }
        }
        uint32_t vcode[16];
#pragma unroll
        for (int i = 0; i < 16; i++) {
            const uint8_t* w = tile + Tile::K_BYTES + g * Tile::V_RUN + i * (DV / 2);
            if constexpr (DV == 64)
                vcode[i] = *reinterpret_cast<const uint16_t*>(w + 2 * n);
            else
                vcode[i] = *reinterpret_cast<const uint32_t*>(w + 4 * n);
        }
        // acc[i][r]: key base + 16 g + 4 r + i of row n
        if (base + ATTN_STEP > in_hi || base < in_lo || base + ATTN_STEP > end) {
            asm volatile("");       // a branch: the compiler would compare every score of every step
            // a step that some row sees only a part of.  Values outside the
            // block's keys get a scale of 2^-127: whatever their bytes hold is
            // then finite, and a weight of zero removes it.
            const int top = min(hi, end);
#pragma unroll
            for (int i = 0; i < 4; i++)
#pragma unroll
                for (int r = 0; r < 4; r++) {
                    const int key = base + 16 * g + 4 * r + i;
                    if (key >= top || key < lo) acc[i][r] = -INFINITY;
                }
#pragma unroll
            for (int r = 0; r < 4; r++) {
                uint32_t keep = 0;
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const int key = base + 16 * g + 4 * r + i;
                    if (key < all_hi && key >= all_lo) keep |= 0xFFu << (8 * i);
                }
                vs[r] &= keep;
            }
        }
        float top = acc[0][0];
#pragma unroll
        for (int i = 0; i < 4; i++)
#pragma unroll
            for (int r = 0; r < 4; r++) top = __builtin_fmaxf(top, acc[i][r]);
        top = over_groups_max(top) * c2;
        // the maximum moves where a row's has grown by 2^8: weights up to that
        // lose nothing, and the outputs are rarely scaled
        if (__any(top > m + ATTN_SLACK)) {
            const float m_new = __builtin_fmaxf(m, top);
            const float alpha = __builtin_amdgcn_exp2f(m - (m_new == -INFINITY ? 0.0f : m_new));
            m = m_new;
            l *= alpha;
#pragma unroll
            for (int d = 0; d < DT; d++) o[d] *= alpha;
        }
        const float m_use = m == -INFINITY ? 0.0f : m;      // a row that has seen nothing yet
        float w[4][4];
#pragma unroll
        for (int i = 0; i < 4; i++)
#pragma unroll
            for (int r = 0; r < 4; r++) w[i][r] = __builtin_amdgcn_exp2f(__builtin_fmaf(acc[i][r], c2, -m_use));
#pragma unroll
        for (int r = 0; r < 4; r++) l += (w[0][r] + w[1][r]) + (w[2][r] + w[3][r]);
        // values: 8 keys (16 g + 8 u ..) at a time
#pragma unroll
        for (int u = 0; u < 2; u++) {
            const v4u pw = {bf16x2_bits(w[0][2 * u], w[1][2 * u]), bf16x2_bits(w[2][2 * u], w[3][2 * u]),
                            bf16x2_bits(w[0][2 * u + 1], w[1][2 * u + 1]), bf16x2_bits(w[2][2 * u + 1], w[3][2 * u + 1])};
            const bf16x8 pf = __builtin_bit_cast(bf16x8, pw);
            float sc[8];
#pragma unroll
            for (int e = 0; e < 2; e++) {
                const uint32_t q4 = vs[2 * u + e];
                sc[4 * e + 0] = scale_of<0>(q4), sc[4 * e + 1] = scale_of<1>(q4);
                sc[4 * e + 2] = scale_of<2>(q4), sc[4 * e + 3] = scale_of<3>(q4);
            }
            auto pair = [&](auto sel) {
                constexpr int SEL = decltype(sel)::value;
                uint32_t x[8];
#pragma unroll
                for (int j = 0; j < 8; j++) x[j] = fp4x2<SEL>(vcode[8 * u + j], sc[j]);
                v4u even, odd;
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    even[j] = __builtin_amdgcn_perm(x[2 * j + 1], x[2 * j], 0x05040100u);
                    odd[j] = __builtin_amdgcn_perm(x[2 * j + 1], x[2 * j], 0x07060302u);
                }
                o[2 * SEL] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, even), pf, o[2 * SEL], 0, 0, 0);
                o[2 * SEL + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, odd), pf, o[2 * SEL + 1], 0, 0, 0);
            };
            pair(std::integral_constant<int, 0>{});
            pair(std::integral_constant<int, 1>{});
            if constexpr (DV == 128) {
                pair(std::integral_constant<int, 2>{});
                pair(std::integral_constant<int, 3>{});
            }
        }
    };
    Step s;
    int base = begin + ATTN_STEP * wave;
    if (base < end) {
        entry = look(base);
        load(s, base);
    }
    for (; base < end; base += ATTN_CHUNK) {
        keep(s);
        uint32_t ks[DK == 192 ? 2 : 1];
#pragma unroll
        for (int i = 0; i < (DK == 192 ? 2 : 1); i++) ks[i] = s.ks[i];
        const v4u vs = s.vs;
        if (base + ATTN_CHUNK < end) load(s, base + ATTN_CHUNK);
        step(ks, vs, base);
    }
    // join the waves: o[d][r] is dim DT (4 g + r) + d of row n
    l = over_groups_sum(l);
    __syncthreads();        // the tiles' place becomes the outputs'
#pragma unroll
    for (int r = 0; r < 4; r++)
#pragma unroll
        for (int d = 0; d < DT; d++) s_o[wave][n][DT * (4 * g + r) + d] = o[d][r];
    if (g == 0) s_m[wave][n] = m, s_l[wave][n] = l;
    __syncthreads();
    const int tr = threadIdx.x >> 4, tl = threadIdx.x & 15;     // 16 threads a row
    const int orow = b.row0 + tr;
    if (orow >= b.rows) return;
    float mm = s_m[0][tr];
#pragma unroll
    for (int w = 1; w < 4; w++) mm = __builtin_fmaxf(mm, s_m[w][tr]);
    const float mu = mm == -INFINITY ? 0.0f : mm;
    float fac[4], ll = 0.0f;
#pragma unroll
    for (int w = 0; w < 4; w++) {
        fac[w] = __builtin_amdgcn_exp2f(s_m[w][tr] - mu);
        ll += s_l[w][tr] * fac[w];
    }
    const int64_t target = (int64_t)(b.q0 + orow / group) * a.q_heads + h * group + orow % group;
    float r[DT];
#pragma unroll
    for (int d = 0; d < DT; d++) {
        float x = 0.0f;
#pragma unroll
        for (int w = 0; w < 4; w++) x += s_o[w][tr][DT * tl + d] * fac[w];
        r[d] = x;
    }
    if constexpr (SPLIT) {
        float* dst = part_o + (target * p.splits + split) * DV + DT * tl;
#pragma unroll
        for (int d = 0; d < DT; d += 4) *reinterpret_cast<v4f*>(dst + d) = v4f{r[d], r[d + 1], r[d + 2], r[d + 3]};
        if (tl == 0) {
            part_ml[(target * p.splits + split) * 2] = part_max(mm, ll);
            part_ml[(target * p.splits + split) * 2 + 1] = ll;
        }
    } else {
        // a row without keys may hold NaN from values that others of its block see
        const bool none = saw_nothing(mm, ll);
        const float inv = 1.0f / ll;
#pragma unroll
        for (int d = 0; d < DT; d++) r[d] = none ? 0.0f : r[d] * inv;
        uint16_t* dst = static_cast<uint16_t*>(a.out) + target * DV + DT * tl;
#pragma unroll
        for (int d = 0; d < DT; d += 4)
            *reinterpret_cast<v2u*>(dst + d) = v2u{bf16x2_bits(r[d], r[d + 1]), bf16x2_bits(r[d + 2], r[d + 3])};
        if (a.lse && tl == 0) a.lse[target] = none ? -INFINITY : (mm + __builtin_amdgcn_logf(ll)) * 0.6931471805599453f;
    }
}

// ------------------------------------------------------------------ many rows
//
// Where a sequence has many rows, a workgroup takes 32 of them a wave and all
// of its waves share the keys and values of a step of 64: they are turned into
// bf16 once, in LDS, and read from there as operands of
// v_mfma_f32_32x32x16_bf16, transposed as above:
//   S^T[key, row]: lane l holds row l % 32, half e = l / 32, and in register i
//                  of a 32-key tile the key 8 (i / 4) + 4 e + i % 4
//   O^T[dim, row]: registers 8 u .. 8 u + 7 are the weights' operand for the
//                  keys 16 u + {4 e + 0..3, 8 + 4 e + 0..3}; the values' rows in
//                  LDS (one a dim) hold the keys in that order.
// The two waves of a SIMD take turns: waves 0 .. 3 multiply (the outputs of step
// t and the scores of step t + 1, 32 matrix instructions) while waves 4 .. 7
// work out maxima and weights on the vector unit, then the other way round, a
// barrier between the phases.  Between its matrix instructions a wave has time
// for what is left: it turns codes of step t + 2 (keys) and t + 1 (values) into
// the halves of the LDS that both groups have left, and asks for the next ones.
// Measured: 9663 queries of 32 heads over 3 contexts of up to 8192 keys, dims 128:
// 735 to 776 us a call over many calls, 792 as the profiler's median of a dispatch: 1.02
// to 1.10 PFLOP/s (a bf16 library product of 8192 cubed: up to 1.43).  With the codes turned
// in the vector phase too, its 2350 clocks a step stood against 1260 of the matrix
// phase, and moving them took 68 us of 806 away.  Now counters show the matrix core
// busy in 54% of the clocks and the vector unit in about 65%.
// The running maximum moves only when a row's maximum has grown by 2^8 or more:
// weights up to 2^8 lose nothing in bf16 and float32, and the outputs are
// rarely scaled.

typedef float v16f __attribute__((ext_vector_type(16)));

// 16-byte chunk c of row m, rows of CHUNKS chunks: neighbouring rows (reads of
// one chunk) and rows 2 or 4 apart (writes of values) meet different banks, and
// rows 32 apart are a constant apart.
template <int CHUNKS>
__device__ __forceinline__ int lds_at(int m, int c) {
    if constexpr (CHUNKS == 16) return m * 16 + (c ^ (m & 15));
    return m * CHUNKS + (c ^ (((m >> 1) ^ ((m >> 4) & 1)) & 7));
}

constexpr int WIDE_WAVES = 8, WIDE_THREADS = 64 * WIDE_WAVES;
constexpr int WIDE_ROWS_LOG2 = 8, WIDE_ROWS = 1 << WIDE_ROWS_LOG2;

template <int DK, int DV, bool SPLIT>
__global__ __launch_bounds__(WIDE_THREADS, 2) void kv4_attention_wide_kernel(Kv4AttnArgs a, AttnPlan p) {
    constexpr int THREADS = WIDE_THREADS;
    constexpr int KC = DK / 8, KK = DK / 16, DT = DV / 32;
    // keys: 8 bytes of codes (16 dims) a unit, 8 or 4 of them (a part of 128 or 64
    // dims) side by side; values: 4 dims of 4 keys a unit
    constexpr int KN = DK == 192 ? 2 : 1;
    constexpr int VU = ATTN_STEP / 4 * (DV / 4);
    static_assert(VU <= THREADS && WIDE_ROWS == 32 * WIDE_WAVES, "one unit of values a thread, and a wave's units in one run of 16 keys");
    // the halves as arrays of their own, chosen at compile time: the compiler then
    // knows that writes to one do not meet reads of the other, and moves them
    __shared__ v4u s_k0[ATTN_STEP * KC], s_k1[ATTN_STEP * KC], s_v0[DV * 8], s_v1[DV * 8];
    typedef std::integral_constant<int, 0> Even;
    typedef std::integral_constant<int, 1> Odd;
    auto keys_in = [&](auto half) { if constexpr (decltype(half)::value) return reinterpret_cast<char*>(s_k1); else return reinterpret_cast<char*>(s_k0); };
    auto values_in = [&](auto half) { if constexpr (decltype(half)::value) return reinterpret_cast<char*>(s_v1); else return reinterpret_cast<char*>(s_v0); };
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, n = lane & 31, e = lane >> 5;
    const int group = a.q_heads / a.kv_heads;
    // chunk by chunk, and long blocks (the last rows of a sequence see the most
    // keys) first
    const int blocks = p.ids * a.kv_heads, split = blockIdx.x / blocks, rest = blockIdx.x - split * blocks;
    const int h = rest % a.kv_heads, id = p.ids - 1 - rest / a.kv_heads;
    AttnBlock b;
    if (!attn_block<WIDE_ROWS_LOG2>(a, group, id, b)) return;

    const int first = b.kv - b.queries;
    auto top_of = [&](int q) { return a.causal ? max(0, min(b.kv, first + q + 1)) : b.kv; };
    auto low_of = [&](int q) { return a.window ? max(0, first + q + 1 - a.window) : 0; };
    const int row = b.row0 + 32 * wave + n;
    const bool real = row < b.rows;
    const int qi = min(row, b.rows - 1) / group, head = h * group + min(row, b.rows - 1) % group;
    const int hi = real ? top_of(qi) : 0, lo = low_of(qi);
    // keys that some row of the block sees, and that every row sees
    const int q_first = b.row0 / group, q_last = (min(b.row0 + WIDE_ROWS, b.rows) - 1) / group;
    const int all_lo = min(low_of(q_first), b.kv), all_hi = top_of(q_last);
    const int in_lo = low_of(q_last), in_hi = top_of(q_first);
    const AttnPart part = attn_part<SPLIT>(p, split, all_lo, all_hi);
    const int begin = part.begin, end = part.end;
    const int64_t target = (int64_t)(b.q0 + qi) * a.q_heads + head;
    float* const part_ml = a.workspace + (int64_t)a.queries * a.q_heads * p.splits * DV;
    if (SPLIT && begin >= end) {
        if (e == 0 && real) part_ml[(target * p.splits + split) * 2] = -INFINITY;
        return;
    }
    const int steps = begin < end ? (end - begin + ATTN_STEP - 1) / ATTN_STEP : 0;

    // A negative scale turns the queries' signs, so that the largest product is
    // the largest score; a scale of zero becomes one that changes nothing and
    // keeps -inf * scale at -inf; a scale of NaN becomes that, too, and turns the
    // queries to NaN, so that rows without keys stay without.
    const float c2 = __builtin_fmaxf(__builtin_fabsf(a.scale) * 1.4426950408889634f, 0x1p-120f);
    bf16x8 q[KK];
    {
        const uint16_t* src = static_cast<const uint16_t*>(a.q) + (int64_t)(b.q0 + qi) * a.q_stride + (int64_t)head * DK + 8 * e;
        const uint32_t flip = a.scale < 0.0f ? 0x80008000u : 0u, spoil = a.scale != a.scale ? 0x7FFF7FFFu : 0u;
#pragma unroll
        for (int j = 0; j < KK; j++) {
            const v4u w = *reinterpret_cast<const v4u*>(src + 16 * j);
            q[j] = __builtin_bit_cast(bf16x8, v4u{(w[0] ^ flip) | spoil, (w[1] ^ flip) | spoil, (w[2] ^ flip) | spoil, (w[3] ^ flip) | spoil});
        }
    }

    // Codes of a step.  Keys: unit i of a part of P pieces is piece i % P of key
    // i / P.  Values: thread t has dims 4 (t % (DV / 4)) .. of the keys 4 (t / (DV /
    // 4)) ..  A wave's keys lie in one run of 16, so in one page, and their place
    // is the wave's, not the lane's: 64-bit scalars and 32-bit lane offsets that
    // no step changes.
    struct Keys {
        v2u k[KN];
        uint32_t ks[KN];
    };
    struct Values {
        uint32_t v[4], vs;
    };
    auto pieces = [](int u) { return DK == 64 || u == 1 ? 4 : 8; };
    auto k_live = [&](int u) { return THREADS == ATTN_STEP * pieces(u) || threadIdx.x < ATTN_STEP * pieces(u); };
    auto k_key = [&](int u) { return (int)threadIdx.x / pieces(u); };
    auto k_piece = [&](int u) { return 8 * u + (int)threadIdx.x % pieces(u); };
    const int vq = threadIdx.x % (DV / 4), vkey = threadIdx.x / (DV / 4) * 4;
    // the wave's run of 16 keys of a step, by its first thread's key
    int k_run[KN], k_off[KN], ks_off[KN];
#pragma unroll
    for (int u = 0; u < KN; u++) {
        k_run[u] = __builtin_amdgcn_readfirstlane(k_key(u) & ~15) & (ATTN_STEP - 1);
        k_off[u] = (k_key(u) & 15) * (DK / 2) + 8 * k_piece(u);
        ks_off[u] = (k_piece(u) >> 1) * a.page_size + (k_key(u) & 15);
    }
    const int v_run = __builtin_amdgcn_readfirstlane(vkey & ~15) & (ATTN_STEP - 1);
    const int v_off = (vkey & 15) * (DV / 2) + vq * 2, vs_off = vq / 8 * a.page_size + (vkey & 15);
    const int32_t* table = a.page_table + (int64_t)b.seq * a.max_pages;
    // cells (a row of a head) of a page, and of the heads in front of this one
    const int64_t page_cells = (int64_t)a.kv_heads * a.page_size, head_cells = (int64_t)h * a.page_size;
    const uint8_t* const k_codes = a.k_codes + head_cells * (DK / 2);
    const uint8_t* const k_scales = a.k_scales + head_cells * (DK / 32);
    const uint8_t* const v_codes = a.v_codes + head_cells * (DV / 2);
    const uint8_t* const v_scales = a.v_scales + head_cells * (DV / 32);
    const int last_page = a.pages - 1, last_slot = a.max_pages - 1;
    // The table's entry for a run of keys, and the run's row in the page; looked up
    // a round before it is used.  The entry stays in a vector register until then:
    // were it known to be the wave's, the compiler would move it to a scalar at
    // once and wait for it on the spot, a memory latency a round.
    struct Run {
        int entry, at;
    };
    int opaque;
    asm volatile("v_mov_b32 %0, 0" : "=v"(opaque));
    auto find = [&](int key) {
        const int whole = (int)divide(key, p.page);
        return Run{table[min(whole, last_slot) + opaque], key - whole * a.page_size};
    };
    auto page_cell = [&](const Run& r) {
        return min(max(__builtin_amdgcn_readfirstlane(r.entry), 0), last_page) * page_cells;
    };
    Run k_at[KN], v_at;
    auto find_keys = [&](int base) {
#pragma unroll
        for (int u = 0; u < KN; u++) k_at[u] = u > 0 && k_run[u] == k_run[0] ? k_at[0] : find(base + k_run[u]);
    };
    auto find_values = [&](int base) { v_at = find(base + v_run); };
    auto load_keys = [&](Keys& s) {
#pragma unroll
        for (int u = 0; u < KN; u++) {
            const int64_t cell = page_cell(k_at[u]);
            const uint8_t* c = k_codes + (cell + k_at[u].at) * (DK / 2);
            const uint8_t* sc = k_scales + cell * (DK / 32) + k_at[u].at;
            if (k_live(u)) {
                s.k[u] = *reinterpret_cast<const v2u*>(c + (uint32_t)k_off[u]);
                s.ks[u] = sc[(uint32_t)ks_off[u]];
            }
        }
    };
    auto load_values = [&](Values& s) {
        const int64_t cell = page_cell(v_at);
        const uint8_t* c = v_codes + (cell + v_at.at) * (DV / 2);
        const uint8_t* sc = v_scales + cell * (DV / 32) + v_at.at;
        if (VU == THREADS || threadIdx.x < VU) {
#pragma unroll
            for (int j = 0; j < 4; j++) s.v[j] = *reinterpret_cast<const uint16_t*>(c + (uint32_t)v_off + j * (DV / 2));
            s.vs = *reinterpret_cast<const uint32_t*>(sc + (uint32_t)vs_off);
        }
    };
    // The lane's places in LDS, in bytes.  Every other place of a step is one of
    // these with an exclusive or of a few bits and a constant added: few registers,
    // where the compiler would keep one for each.
    int k_read = 16 * lds_at<KC>(n, e), v_read = 16 * lds_at<8>(n, e), k_write[KN];
#pragma unroll
    for (int u = 0; u < KN; u++) k_write[u] = 16 * lds_at<KC>(k_key(u), 2 * k_piece(u));
    // chunk `part` of each unit
    auto turn_keys = [&](const Keys& s, auto half, int part) {
#pragma unroll
        for (int u = 0; u < KN; u++) {
            if (k_live(u)) {
                const float scale = __builtin_bit_cast(float, s.ks[u] << 23);
                *reinterpret_cast<v4u*>(keys_in(half) + (k_write[u] ^ (16 * part))) = __builtin_bit_cast(v4u, fp4x8(s.k[u][part], scale));
            }
        }
    };
    // A run of 4 keys is half a chunk of the values' rows: runs 0, 2 of 16 keys
    // (e = 0) and 1, 3 (e = 1).
    int v_write = 16 * lds_at<8>(4 * vq, 2 * (vkey >> 4) + ((vkey >> 2) & 1)) + 8 * ((vkey >> 3) & 1);
    auto value_scales = [&](const Values& s, int base, float (&sc)[4]) {
        // values outside the block's keys: a scale of 2^-127 makes whatever they
        // hold finite, and their weight of zero removes it
        auto first_bytes = [](int n) { return n <= 0 ? 0u : n >= 4 ? ~0u : (1u << (8 * n)) - 1u; };
        const uint32_t vs = s.vs & first_bytes(all_hi - base - vkey) & ~first_bytes(all_lo - base - vkey);
        sc[0] = scale_of<0>(vs), sc[1] = scale_of<1>(vs), sc[2] = scale_of<2>(vs), sc[3] = scale_of<3>(vs);
    };
    // dims 2 part, 2 part + 1 of the unit's 4
    auto turn_values = [&](const Values& s, const float (&sc)[4], auto half, auto part) {
        if (VU == THREADS || threadIdx.x < VU) {
            constexpr int SEL = decltype(part)::value;
            uint32_t x[4];
#pragma unroll
            for (int j = 0; j < 4; j++) x[j] = fp4x2<SEL>(s.v[j], sc[j]);
            v2u even, odd;
#pragma unroll
            for (int j = 0; j < 2; j++) {
                even[j] = __builtin_amdgcn_perm(x[2 * j + 1], x[2 * j], 0x05040100u);
                odd[j] = __builtin_amdgcn_perm(x[2 * j + 1], x[2 * j], 0x07060302u);
            }
            // rows 2 SEL and 2 SEL + 1 of the unit's 4, 128 bytes each
            char* const to = values_in(half) + (v_write ^ (16 * SEL)) + 256 * SEL;
            *reinterpret_cast<v2u*>(to) = even;
            *reinterpret_cast<v2u*>(to + 128) = odd;
        }
    };

    v16f o[DT];
#pragma unroll
    for (int d = 0; d < DT; d++)
#pragma unroll
        for (int i = 0; i < 16; i++) o[d][i] = 0.0f;
    float m = -INFINITY, l = 0.0f;

    // operand j, x of the scores (16 dims of 32 keys), and u, d of the outputs
    auto key_operand = [&](auto half, int j, int x) {
        const int flip = DK == 128 ? 2 * j : (2 * j) & 7, add = 2 * j - flip + 32 * KC * x;
        return __builtin_bit_cast(bf16x8, *reinterpret_cast<const v4u*>(keys_in(half) + (k_read ^ (16 * flip)) + 16 * add));
    };
    auto value_operand = [&](auto half, int u, int d) {
        return __builtin_bit_cast(bf16x8, *reinterpret_cast<const v4u*>(values_in(half) + (v_read ^ (32 * u)) + 4096 * d));
    };
    const v16f zero = {0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
    auto scores = [&](v16f (&acc)[2], auto half) {
#pragma unroll
        for (int j = 0; j < KK; j++)
#pragma unroll
            for (int x = 0; x < 2; x++)
                acc[x] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(key_operand(half, j, x), q[j], j ? acc[x] : zero, 0, 0, 0);
    };
    // the largest score of the lane's half of its row, after the mask of an edge step
    auto largest = [&](v16f (&acc)[2], int base, bool edge) {
        if (edge) {
            asm volatile("");        // a branch: the compiler would compare every score of every step
            const int from = lo - base - 4 * e, to = min(hi, end) - base - 4 * e;
#pragma unroll
            for (int x = 0; x < 2; x++)
#pragma unroll
                for (int i = 0; i < 16; i++) {
                    const int key = 32 * x + 8 * (i >> 2) + (i & 3);
                    if (key >= to || key < from) acc[x][i] = -INFINITY;
                }
        }
        float top = acc[0][0];
#pragma unroll
        for (int x = 0; x < 2; x++)
#pragma unroll
            for (int i = 0; i < 16; i++) top = __builtin_fmaxf(top, acc[x][i]);
        return top;
    };
    // the row's maximum moves to the new largest score where that is far above it
    auto raise = [&](float top) {
        top = across_halves(top) * c2;
        if (__any(top > m + ATTN_SLACK)) {
            const float m_new = __builtin_fmaxf(m, top);
            const float alpha = __builtin_amdgcn_exp2f(m - (m_new == -INFINITY ? 0.0f : m_new));
            m = m_new;
            l *= alpha;
#pragma unroll
            for (int d = 0; d < DT; d++) o[d] *= alpha;
        }
    };
    auto weights = [&](const v16f (&acc)[2], bf16x8 (&w)[4]) {
        const float m_use = m == -INFINITY ? 0.0f : m;      // a row that has seen nothing yet
        float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int u = 0; u < 4; u++) {
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; i++) {
                x[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(acc[u >> 1][8 * (u & 1) + i], c2, -m_use));
                sum[i & 3] += x[i];
            }
            const v4u r = {bf16x2_bits(x[0], x[1]), bf16x2_bits(x[2], x[3]), bf16x2_bits(x[4], x[5]), bf16x2_bits(x[6], x[7])};
            w[u] = __builtin_bit_cast(bf16x8, r);
        }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
    };
    auto outputs = [&](const bf16x8 (&w)[4], auto half) {
#pragma unroll
        for (int u = 0; u < 4; u++)
#pragma unroll
            for (int d = 0; d < DT; d++)
                o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(value_operand(half, u, d), w[u], o[d], 0, 0, 0);
    };

    if (steps > 0) {
        // steps [j0, j1) lie inside what every row of the block sees
        const int j0 = in_lo > begin ? (in_lo - begin + ATTN_STEP - 1) / ATTN_STEP : 0;
        const int j1 = min(in_hi, end) > begin ? (min(in_hi, end) - begin) / ATTN_STEP : 0;
        auto base_of = [&](int t) { return begin + t * ATTN_STEP; };
        auto edge = [&](int t) { return t < j0 || t >= j1; };
        const int late = wave >= WIDE_WAVES / 2;      // the waves one phase behind
        Keys keys;
        Values values;
        v16f acc[2];
        bf16x8 w[4];
        find_keys(base_of(0));
        find_values(base_of(0));
        load_keys(keys);
        load_values(values);
        find_keys(base_of(1));
        find_values(base_of(1));
        turn_keys(keys, Even{}, 0);
        turn_keys(keys, Even{}, 1);
        load_keys(keys);
        find_keys(base_of(2));
        float sc[4];
        value_scales(values, base_of(0), sc);
        turn_values(values, sc, Even{}, Even{});
        turn_values(values, sc, Even{}, Odd{});
        load_values(values);
        find_values(base_of(2));
        turn_keys(keys, Odd{}, 0);
        turn_keys(keys, Odd{}, 1);
        load_keys(keys);
        find_keys(base_of(3));
        __syncthreads();
        scores(acc, Even{});
        raise(largest(acc, base_of(0), true));
        weights(acc, w);
        __syncthreads();
        auto round = [&](int t, auto half) {
            typedef std::integral_constant<int, decltype(half)::value ^ 1> Other;
            __builtin_amdgcn_s_setprio(1);
            // The products in eight groups, their operands read 6 or 4 ahead, and with
            // each group a slice of the rest: the compiler's own order waits for
            // each pair of reads and leaves the rest behind the last product.
            constexpr int PRODUCTS = 4 * DT + 2 * KK, AHEAD = DK == 192 ? 4 : 6, GROUP = PRODUCTS / 8;
            // places worked out anew in every round, not kept from before the loop
            asm volatile("" : "+v"(k_read), "+v"(v_read), "+v"(v_write));
#pragma unroll
            for (int u = 0; u < KN; u++) asm volatile("" : "+v"(k_write[u]));
            auto operand = [&](int i) {
                return i < 4 * DT ? value_operand(half, i / DT, i % DT) : key_operand(Other{}, (i - 4 * DT) >> 1, (i - 4 * DT) & 1);
            };
            bf16x8 ring[AHEAD];
#pragma unroll
            for (int i = 0; i < AHEAD; i++) ring[i] = operand(i);
            float sc[4];
#pragma unroll
            for (int gr = 0; gr < 8; gr++) {
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int i = gr * GROUP; i < (gr + 1) * GROUP; i++) {
                    const bf16x8 x = ring[i % AHEAD];
                    if (i < 4 * DT) {
                        o[i % DT] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x, w[i / DT], o[i % DT], 0, 0, 0);
                    } else {
                        const int j = i - 4 * DT;
                        acc[j & 1] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x, q[j >> 1], j < 2 ? zero : acc[j & 1], 0, 0, 0);
                    }
                    if (i + AHEAD < PRODUCTS) ring[i % AHEAD] = operand(i + AHEAD);
                }
                if (gr == 0) turn_keys(keys, half, 0);                       // of step t + 2
                if (gr == 1) turn_keys(keys, half, 1);
                if (gr == 2) value_scales(values, base_of(t + 1), sc);
                if (gr == 3) turn_values(values, sc, Other{}, Even{});
                if (gr == 4) turn_values(values, sc, Other{}, Odd{});
                if (gr == 5) load_keys(keys);                                // of step t + 3
                if (gr == 6) load_values(values);                            // of step t + 2
                if (gr == 7) {
                    find_keys(base_of(t + 4));
                    find_values(base_of(t + 3));
                }
#pragma unroll
                for (int i = 0; i < GROUP; i++) {
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
                    __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);
                    __builtin_amdgcn_sched_group_barrier(0x004, 5, 0);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
            __builtin_amdgcn_s_setprio(0);
            __syncthreads();
            raise(largest(acc, base_of(t + 1), edge(t + 1)));
            weights(acc, w);
            __syncthreads();
        };
        if (late) __syncthreads();
        int t = 0;
        for (; t + 2 < steps; t += 2) {
            round(t, Even{});
            round(t + 1, Odd{});
        }
        if (t + 1 < steps) {
            round(t, Even{});
            outputs(w, Odd{});
        } else {
            outputs(w, Even{});
        }
        if (!late) __syncthreads();
    }
    l += __shfl_xor(l, 32, 64);
    if (!real) return;
    // register i of tile d: dim 32 d + 8 (i / 4) + 4 e + i % 4
    if constexpr (SPLIT) {
        float* dst = a.workspace + (target * p.splits + split) * DV + 4 * e;
#pragma unroll
        for (int d = 0; d < DT; d++)
#pragma unroll
            for (int i = 0; i < 16; i += 4)
                *reinterpret_cast<v4f*>(dst + 32 * d + 2 * i) = v4f{o[d][i], o[d][i + 1], o[d][i + 2], o[d][i + 3]};
        if (e == 0) {
            part_ml[(target * p.splits + split) * 2] = part_max(m, l);
            part_ml[(target * p.splits + split) * 2 + 1] = l;
        }
    } else {
        // A row without keys may hold NaN from values that others of its block see.
        // A select for each value would spill 10 registers at dims 192, this 4.
        const bool none = saw_nothing(m, l);
        const float inv = none ? 0.0f : 1.0f / l;
        if (none) {
#pragma unroll
            for (int d = 0; d < DT; d++) o[d] = zero;
        }
        uint16_t* dst = static_cast<uint16_t*>(a.out) + target * DV + 4 * e;
#pragma unroll
        for (int d = 0; d < DT; d++)
#pragma unroll
            for (int i = 0; i < 16; i += 4)
                *reinterpret_cast<v2u*>(dst + 32 * d + 2 * i) =
                    v2u{bf16x2_bits(o[d][i] * inv, o[d][i + 1] * inv), bf16x2_bits(o[d][i + 2] * inv, o[d][i + 3] * inv)};
        if (a.lse && e == 0) a.lse[target] = none ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * 0.6931471805599453f;
    }
}

// Joins the chunks of every row, in order: DV / 4 lanes a row.
template <int DV>
__global__ __launch_bounds__(ATTN_THREADS) void kv4_attention_join_kernel(Kv4AttnArgs a, AttnPlan p) {
    constexpr int LANES = DV / 4, ROWS = ATTN_THREADS / LANES;
    const int64_t rows = (int64_t)a.queries * a.q_heads;
    const int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / LANES;
    const int lane = threadIdx.x % LANES;
    if (row >= rows) return;
    const int query = (int)(row / a.q_heads);
    if (query < a.q_start[0] || query >= a.q_start[a.batch]) return;   // of no sequence
    const float* part_o = a.workspace + row * p.splits * DV + 4 * lane;
    const float* part_ml = a.workspace + rows * p.splits * DV + row * p.splits * 2;
    constexpr int AHEAD = 8;            // chunks in flight
    float ms[AHEAD], ls[AHEAD];
    v4f os[AHEAD];
    auto load = [&](int s0) {
#pragma unroll
        for (int u = 0; u < AHEAD; u++) {
            const int s = min(s0 + u, p.splits - 1);
            ms[u] = part_ml[2 * s], ls[u] = part_ml[2 * s + 1];
            os[u] = *reinterpret_cast<const v4f*>(part_o + (int64_t)s * DV);
        }
    };
    // The chunks in front of the last that holds keys of the row: a table far
    // wider than the context leaves most of them empty.  Found by the row's lanes
    // together, a maximum each, while the first chunks travel.
    load(0);
    int used = p.splits <= AHEAD ? p.splits : 0;
    for (int s0 = 0; s0 < p.splits && p.splits > AHEAD; s0 += LANES) {
        const bool holds = s0 + lane < p.splits && part_ml[2 * (s0 + lane)] != -INFINITY;
        const uint64_t all = __ballot(holds) >> (threadIdx.x & 63 & ~(LANES - 1)) & ((1ull << LANES) - 1);
        if (all) used = s0 + 64 - __builtin_clzll(all);
    }
    float m = -INFINITY, l = 0.0f;
    v4f o = {0, 0, 0, 0};
    for (int s0 = 0; s0 < used; s0 += AHEAD) {
        if (s0 > 0) load(s0);
        float top = m;
#pragma unroll
        for (int u = 0; u < AHEAD; u++)
            if (s0 + u < used) top = __builtin_fmaxf(top, ms[u]);
        const float mu = top == -INFINITY ? 0.0f : top, f0 = __builtin_amdgcn_exp2f(m - mu);
        l *= f0, o *= f0;
        m = top;
#pragma unroll
        for (int u = 0; u < AHEAD; u++) {
            // a chunk without keys of the row has -inf, and the rest may be anything
            if (s0 + u >= used || ms[u] == -INFINITY) continue;
            const float f = __builtin_amdgcn_exp2f(ms[u] - mu);
            l += ls[u] * f;
            o += os[u] * f;
        }
    }
    const bool none = saw_nothing(m, l);
    const float inv = none ? 0.0f : 1.0f / l;
    *reinterpret_cast<v2u*>(static_cast<uint16_t*>(a.out) + row * DV + 4 * lane) =
        v2u{bf16x2_bits(o[0] * inv, o[1] * inv), bf16x2_bits(o[2] * inv, o[3] * inv)};
    if (a.lse && lane == 0) a.lse[row] = none ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * 0.6931471805599453f;
}

// Many rows a sequence on average: blocks of 256 rows, not 16.  us with blocks of
// 16 / 256, four heads a key head:
//   rows a key head                       64       128       160       192       256       384       512
//   8 x 8192 keys, 8 key heads, 128    48/ 79    74/105   117/109   113/116   132/149   192/159   251/197
//   32 x 4096, 4, 128                  56/101    76/107   100/106   115/117   141/167   198/197   260/204
//   8 x 8192, 16, 192/128              93/220   162/227   201/232   236/239   310/488   457/456   602/508
//   8 x 8192, 8, 64                    43/ 69    73/ 97    73/ 98    73/100    94/135   134/140   175/179
//   1 x 32768, 8, 128                  29/ 54    45/ 60    57/ 62    62/ 66    74/107   136/ 87   137/121
//   3 x 2048, 8, 128                   15/ 19    19/ 24    20/ 27    22/ 28    22/ 42    32/ 44    32/ 46
// At 160 to 192 rows the larger blocks are between 7% faster and 37% slower, at 256 (one
// whole block a sequence) 13 to 90% slower, for a reason that was not found, and from
// 384 on up to a third faster where keys are many.
static bool attn_wide(const Kv4AttnArgs& a) {
    return (int64_t)a.queries * (a.q_heads / a.kv_heads) >= 160 * (int64_t)a.batch;
}

static AttnPlan attn_plan(const Kv4AttnArgs& a) {
    AttnPlan p;
    const int group = a.q_heads / a.kv_heads;
    const bool wide = attn_wide(a);
    const int rows = wide ? WIDE_ROWS : ATTN_ROWS;
    p.ids = (int)((int64_t)a.queries * group / rows) + a.batch;
    p.page = fast_div((uint32_t)a.page_size);
    int64_t keys = (int64_t)a.max_pages * a.page_size;
    const int64_t span = (int64_t)a.window + rows + ATTN_STEP;
    if (a.window && keys > span) keys = span;
    // blocks that certainly have rows
    int64_t blocks = ((int64_t)a.queries * group + rows - 1) / rows;
    const int some = a.batch < a.queries ? a.batch : a.queries;
    if (blocks < some) blocks = some;
    blocks *= a.kv_heads;
    // Two workgroups a CU fill the chip; more and smaller chunks cost more than
    // they balance (measured with 1024 and 2048).
    // A chunk of at most 16384 keys keeps one long sequence among short ones from
    // being the whole time.  64 heads over 8, dims 128, us with 8192 / 16384 / 32768 /
    // 65536: 131072 keys beside 63 sequences of 2048 171 / 171 / 238 / 357; 32 sequences
    // of 32768 to 131072 keys 554 / 570 / 616 / 629; 64 of 4165 to 16384 165 / 161 / 161 /
    // 161.  But a wide table says little about the contexts, and every split has its
    // workgroups, empty or not, and its place in the workspace: at most 16 splits for
    // that, and a workspace of 64 MB, what rows that need splits to fill the chip take
    // at most.  With a table of 2^20 keys and 8 / 16 / 64 splits: the 64 sequences 168 /
    // 172 / 184 us, one of 2^20 keys beside 63 of 2048 1031 / 607 / 617.
    constexpr int64_t full = 512, longest_splits = 16, room = 64 << 20;
    const int64_t steps = (keys + ATTN_CHUNK - 1) / ATTN_CHUNK;
    int64_t fill = blocks >= full ? 1 : full / blocks;
    const int64_t most = most_blocks(wide ? WIDE_THREADS : ATTN_THREADS) / ((int64_t)p.ids * a.kv_heads);
    if (fill > most) fill = most < 1 ? 1 : most;
    if (steps > 0) {
        const int64_t each = (steps + fill - 1) / fill;
        fill = (steps + each - 1) / each;
    } else {
        fill = 1;
    }
    int64_t splits = (keys + ATTN_LONGEST - 1) / ATTN_LONGEST;
    if (splits > longest_splits) splits = longest_splits;
    const int64_t fits = room / ((int64_t)a.queries * a.q_heads * (a.dv + 2) * 4);
    if (splits > fits) splits = fits;
    if (splits > most) splits = most;
    if (splits < fill) splits = fill;
    p.fill = (int)fill;
    p.splits = (int)splits;
    p.by_fill = fast_div((uint32_t)fill);
    p.by_splits = fast_div((uint32_t)splits);
    return p;
}

bool kv4_attention_fits(const Kv4AttnArgs& a) {
    if (a.queries == 0 || a.batch == 0 || a.q_heads == 0) return true;
    return (int64_t)attn_plan(a).ids * a.kv_heads <= most_blocks(attn_wide(a) ? WIDE_THREADS : ATTN_THREADS);
}

int64_t kv4_attention_bytes(const Kv4AttnArgs& a) {
    if (a.queries == 0 || a.batch == 0 || a.q_heads == 0) return 0;
    const AttnPlan p = attn_plan(a);
    return p.splits > 1 ? (int64_t)a.queries * a.q_heads * p.splits * (a.dv + 2) * 4 : 0;
}

template <int DK, int DV, bool SPLIT>
static hipError_t launch_rows(const Kv4AttnArgs& a, const AttnPlan& p, hipStream_t stream) {
    const dim3 grid((unsigned)((int64_t)p.ids * a.kv_heads * p.splits));
    if (attn_wide(a))
        kv4_attention_wide_kernel<DK, DV, SPLIT><<<grid, dim3(WIDE_THREADS), 0, stream>>>(a, p);
    else
        kv4_attention_kernel<DK, DV, SPLIT><<<grid, dim3(ATTN_THREADS), 0, stream>>>(a, p);
    return hipGetLastError();
}

template <int DK, int DV>
static hipError_t launch_dims(const Kv4AttnArgs& a, hipStream_t stream) {
    const AttnPlan p = attn_plan(a);
    if (p.splits == 1) return launch_rows<DK, DV, false>(a, p, stream);
    const hipError_t e = launch_rows<DK, DV, true>(a, p, stream);
    if (e != hipSuccess) return e;
    constexpr int ROWS = ATTN_THREADS / (DV / 4);
    const int64_t rows = (int64_t)a.queries * a.q_heads;
    kv4_attention_join_kernel<DV><<<dim3((unsigned)((rows + ROWS - 1) / ROWS)), dim3(ATTN_THREADS), 0, stream>>>(a, p);
    return hipGetLastError();
}

hipError_t launch_kv4_attention(const Kv4AttnArgs& in, hipStream_t stream) {
    Kv4AttnArgs a = in;
    if (a.pages == 0) a.max_pages = 0;   // no page to read: no sequence has keys
    if (a.dk == 64) return launch_dims<64, 64>(a, stream);
    if (a.dk == 128) return launch_dims<128, 128>(a, stream);
    return launch_dims<192, 128>(a, stream);
}

}  // namespace fp8g
