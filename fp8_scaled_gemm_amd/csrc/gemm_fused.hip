// The fused products and the experts' products on the tile kernel (gemm_tile.h):
// the plan of the experts' tile rows, and the launches.  Products of few rows
// take gemm_rows.hip instead.
//
// Experts' products: which expert has how many rows is known on the device only.
// A small kernel lays the tile rows of all experts end to end (an expert's
// last one may be partly empty), so that the tile kernel walks them as it walks
// the tile rows of one product; and where A's rows are gathered it writes each
// tile row's offsets into A, which the operand loads then take instead of a
// row's own, and puts A's scales (32 or 128 times smaller than A) into the
// slots' order.
//
// Bound by the matrix core at the board's power limit where the tiles fill the CUs
// (8192 x 2 x 11008 x 8192 gated 1032 us, 2.86 PFLOP/s, as without an epilogue);
// experts lose the empty part of each one's last tile (65536 rows of 128 experts x
// 2 x 1024 x 4096: 606 us, 1.81 PFLOP/s).
//
// Compiled once per mode and kind (FP8G_FUSED_PART = 4 * gated + 2 * MX + MOE, or
// 8 + MX for the partial sums of K ranges).

#include <atomic>
#include <type_traits>

#include "gemm_tile.h"
#include "launch_ffn.h"

namespace fp8g {

template <bool MX, bool OUT_F32, bool KTAIL, int TILE, int EPI, bool MOE>
__global__ __launch_bounds__(NTHREADS, 1) void gemm_fused_kernel(int M, int N, int K, const uint8_t* __restrict__ A,
                                                                 const uint8_t* __restrict__ B, const void* __restrict__ sa,
                                                                 const void* __restrict__ sb, void* Dv, TileExtra ex) {
    const float* fa = MX ? nullptr : static_cast<const float*>(sa);
    const float* fb = MX ? nullptr : static_cast<const float*>(sb);
    const uint8_t* ea = MX ? static_cast<const uint8_t*>(sa) : nullptr;
    const uint8_t* eb = MX ? static_cast<const uint8_t*>(sb) : nullptr;
    gemm_tiles<MX, OUT_F32, KTAIL, 0, 0, TILE, false, EPI, MOE>(M, N, K, A, B, fa, fb, ea, eb, Dv, 0, 1, nullptr, nullptr, ex);
}

template <bool MX, bool OUT_F32, bool KTAIL, int TILE, int EPI, bool MOE>
static hipError_t launch_tile(const FusedArgs& a, const TileLaunch& t, hipStream_t stream) {
    auto kern = gemm_fused_kernel<MX, OUT_F32, KTAIL, TILE, EPI, MOE>;
    constexpr int LDS_BYTES = Ring<MX, false, TILE>::LDS_TOTAL;
    // above the default launch limit: raised once per device; setting it twice
    // from racing threads is harmless
    static std::atomic<uint64_t> configured{0};
    const uint64_t bit = t.dev < 64 ? (uint64_t)1 << t.dev : 0;
    if (!bit || !(configured.load(std::memory_order_acquire) & bit)) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kern), hipFuncAttributeMaxDynamicSharedMemorySize,
                                                 LDS_BYTES);
        if (e != hipSuccess) return e;
        configured.fetch_or(bit, std::memory_order_release);
    }
    constexpr int BM = Geo<TILE>::BM, BNO = EPI == EPI_GATED ? Geo<TILE>::BN / 2 : Geo<TILE>::BN;
    const int64_t tiles = (MOE ? t.tile_rows : (a.m + BM - 1) / BM) * ((a.n + BNO - 1) / BNO) * (EPI == EPI_PARTIAL ? t.ranges : 1);
    const TileExtra ex = {a.bias,  a.residual, act_of(a.act), t.plan, t.row_at, t.row_at ? (uint32_t)(a.a_rows * a.k) : 0u,
                          t.ranges, t.pitch, t.part_rows};
    kern<<<dim3((unsigned)(tiles < t.cus ? tiles : t.cus)), dim3(NTHREADS), LDS_BYTES, stream>>>(
        (int)a.m, (int)a.n, (int)a.k, a.A, a.B, t.scale_a, a.scale_b, a.D, ex);
    return hipGetLastError();
}

template <bool MX, bool MOE, int EPI>
hipError_t launch_fused_part(const FusedArgs& a, const TileLaunch& t, hipStream_t stream) {
    auto go = [&](auto tile) {
        constexpr int TILE = decltype(tile)::value;
        if constexpr (EPI == EPI_PARTIAL)
            return a.k % BK ? launch_tile<MX, true, true, TILE, EPI, MOE>(a, t, stream)
                            : launch_tile<MX, true, false, TILE, EPI, MOE>(a, t, stream);
        else if (a.k % BK)
            return a.f32 ? launch_tile<MX, true, true, TILE, EPI, MOE>(a, t, stream)
                         : launch_tile<MX, false, true, TILE, EPI, MOE>(a, t, stream);
        else
            return a.f32 ? launch_tile<MX, true, false, TILE, EPI, MOE>(a, t, stream)
                         : launch_tile<MX, false, false, TILE, EPI, MOE>(a, t, stream);
    };
    if constexpr (!MX) {
        if (t.tile == TILE_64x128) return go(std::integral_constant<int, TILE_64x128>{});
        if constexpr (EPI != EPI_PARTIAL)
            if (t.tile == 256) return launch_tile<MX, false, false, 256, EPI, MOE>(a, t, stream);
    }
    if constexpr (EPI != EPI_PARTIAL)
        if (t.tile == TILE_256x128) return go(std::integral_constant<int, TILE_256x128>{});
    return go(std::integral_constant<int, 128>{});
}

#ifndef FP8G_FUSED_PART
#error "FP8G_FUSED_PART"
#endif
#define FP8G_FUSED(KW, MX, MOE, EPI) \
    KW hipError_t launch_fused_part<MX, MOE, EPI>(const FusedArgs&, const TileLaunch&, hipStream_t);
#if FP8G_FUSED_PART >= 8
FP8G_FUSED(template, (FP8G_FUSED_PART == 9), false, EPI_PARTIAL)
#else
FP8G_FUSED(template, ((FP8G_FUSED_PART & 2) != 0), ((FP8G_FUSED_PART & 1) != 0), ((FP8G_FUSED_PART & 4) ? EPI_GATED : EPI_LINEAR))
#endif

#if FP8G_FUSED_PART == 0
FP8G_FUSED(extern template, false, true, EPI_LINEAR)
FP8G_FUSED(extern template, true, false, EPI_LINEAR)
FP8G_FUSED(extern template, true, true, EPI_LINEAR)
FP8G_FUSED(extern template, false, false, EPI_GATED)
FP8G_FUSED(extern template, false, true, EPI_GATED)
FP8G_FUSED(extern template, true, false, EPI_GATED)
FP8G_FUSED(extern template, true, true, EPI_GATED)
FP8G_FUSED(extern template, false, false, EPI_PARTIAL)
FP8G_FUSED(extern template, true, false, EPI_PARTIAL)

template <bool MX, bool MOE>
static hipError_t launch_fused(const FusedArgs& a, const TileLaunch& t, hipStream_t stream) {
    return a.gated ? launch_fused_part<MX, MOE, EPI_GATED>(a, t, stream) : launch_fused_part<MX, MOE, EPI_LINEAR>(a, t, stream);
}

constexpr int PLAN_THREADS = 256, PLAN_EXPERTS = 1024;

// ---- scale rows of whole dwords, for K not a multiple of 128: 4 bytes for each
// 128 of K, those behind the row 2^0 (the codes there are read as zeros).  A few
// percent of the operands' bytes, where fetching the odd bytes one by one in the
// product halved its rate.
struct PadArgs {
    const uint8_t* from[2];
    uint8_t* to[2];
    int64_t rows[2];
    int nblk, words;             // bytes of a row, dwords of a padded one
};
__device__ __forceinline__ uint32_t padded_word(const uint8_t* row, int c, int nblk) {
    const uint32_t w = scale_word(row, c, nblk), left = (uint32_t)max(nblk - 4 * c, 0);
    return left >= 4 ? w : (w & ((1u << (8 * left)) - 1u)) | (0x7F7F7F7Fu << (8 * left));
}
__global__ __launch_bounds__(PLAN_THREADS) void pad_scales(PadArgs p) {
    const int side = blockIdx.y;
    const int64_t total = p.rows[side] * p.words, step = (int64_t)gridDim.x * PLAN_THREADS;
    for (int64_t i = (int64_t)blockIdx.x * PLAN_THREADS + threadIdx.x; i < total; i += step) {
        const int64_t r = i / p.words;
        const int c = (int)(i - r * p.words);
        reinterpret_cast<uint32_t*>(p.to[side])[i] = padded_word(p.from[side] + r * p.nblk, c, p.nblk);
    }
}
static hipError_t launch_pad(const PadArgs& p, hipStream_t stream) {
    const int64_t most = (p.rows[0] > p.rows[1] ? p.rows[0] : p.rows[1]) * p.words;
    int64_t blocks = (most + PLAN_THREADS - 1) / PLAN_THREADS;
    if (blocks > 4096) blocks = 4096;
    pad_scales<<<dim3((unsigned)blocks, 2), dim3(PLAN_THREADS), 0, stream>>>(p);
    return hipGetLastError();
}
// bytes of a padded scale row; 0: the rows are whole dwords already
static int64_t pad_pitch(const FusedArgs& a) { return a.mx && a.k % BK ? (a.k + BK - 1) / BK * 4 : 0; }
static int64_t up16(int64_t v) { return (v + 15) / 16 * 16; }

// One workgroup per possible tile row t: every one counts the experts' tile
// rows (an expert of c slots has ceil(c / bm)); the expert that holds t writes it down.
// Ascending starts have disjoint experts, sum c <= slots, so that there are at most
// slots / bm + experts tile rows, which is the grid (moe_space).  Starts that fall
// again count slots twice and could have more: the plan ends with the grid, and the
// tile kernel never walks past what is written here.  A planned row lies in [0,
// slots) whatever the starts, as each end is clamped to its own start and to slots.
__global__ __launch_bounds__(PLAN_THREADS) void moe_plan(const int32_t* __restrict__ start, const int32_t* __restrict__ rows,
                                                         const void* __restrict__ sa, int experts, int slots, int a_rows,
                                                         int k, int mx, int bm, int32_t* __restrict__ plan,
                                                         uint32_t* __restrict__ row_at, void* __restrict__ scale) {
    __shared__ int sum[PLAN_THREADS / 64];
    __shared__ int mine[3];
    constexpr int PER = PLAN_EXPERTS / PLAN_THREADS;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, t = blockIdx.x;
    int first[PER], count[PER], tiles = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = tid * PER + i;
        first[i] = count[i] = 0;
        if (e < experts) {
            first[i] = min(max(start[e], 0), slots);
            count[i] = min(max(start[e + 1], first[i]), slots) - first[i];
        }
        tiles += (count[i] + bm - 1) / bm;
    }
    // at most all of the grid each: a thread's 4 x 2^22 tile rows, 256 times, would pass 2^31
    tiles = min(tiles, (int)gridDim.x);
    int upto = tiles;                                     // with this thread's
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const int v = __shfl_up(upto, off, 64);
        if (lane >= off) upto += v;
    }
    if (lane == 63) sum[wave] = upto;
    __syncthreads();
    int total = 0;
#pragma unroll
    for (int w = 0; w < PLAN_THREADS / 64; ++w) {
        if (w < wave) upto += sum[w];
        total += sum[w];
    }
    if (t == 0 && tid == 0) plan[0] = min(total, (int)gridDim.x);
    if (t >= total) return;
    int at = upto - tiles;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int n = (count[i] + bm - 1) / bm;
        if (t >= at && t < at + n) {
            mine[0] = tid * PER + i;
            mine[1] = first[i] + (t - at) * bm;
            mine[2] = min(bm, count[i] - (t - at) * bm);
        }
        at += n;
    }
    __syncthreads();
    const int m0 = mine[1], here = mine[2];
    if (tid < 3) plan[4 + 4 * t + tid] = mine[tid];
    if (!rows) return;
    for (int r = tid; r < bm; r += PLAN_THREADS) {
        uint32_t off = 0x80000000u;                       // past any A: reads 0
        if (r < here) {
            const int a = min(max(rows[m0 + r], 0), a_rows - 1);
            off = (uint32_t)a * (uint32_t)k;
            if (!mx) static_cast<float*>(scale)[m0 + r] = static_cast<const float*>(sa)[a];
        }
        row_at[(int64_t)t * bm + r] = off;
    }
    if (!mx) return;
    const int nblk = k / 32, nw = (k + BK - 1) / BK;      // whole dwords a row
    for (int i = tid; i < here * nw; i += PLAN_THREADS) {
        const int r = i / nw, a = min(max(rows[m0 + r], 0), a_rows - 1);
        static_cast<uint32_t*>(scale)[(int64_t)(m0 + r) * nw + i % nw] =
            padded_word(static_cast<const uint8_t*>(sa) + (int64_t)a * nblk, i % nw, nblk);
    }
}

// ---- one product: which kernel, tile and K ranges.
//
// Times of a launch in us, fitted to measurements on MI355X (256 CUs; weights
// from HBM) and used to choose between
//   the row kernel (gemm_rows.hip), the larger of
//     4 + B at 5.5 TB/s, again at 8 TB/s for every further 64 rows, + A, read by
//     every workgroup, at 9.3 TB/s, and
//     4 + the steps of a wave at 0.35 / 0.6 / 1.1 us with 16 / 32 / 64 rows of A
//     (mode (b): a tenth more of all of it);
//   a tile: 4.5 + rounds of workgroups x (fixed + stages x stage), below, the
//     stage of the small tiles shorter while they fill at most half of the CUs;
//   64x128 or 128x128 tiles with K in ranges, where the tiles leave CUs idle:
//     one round of the longest range, and 4 + the partial sums written and
//     read at 4 TB/s for the kernel that adds them up.
// Measured, mode (a), 2 x 11008 x 8192 gated: rows 37.7 us at m = 8, 51 at 32, 74
// at 64 (64x128 tiles 41, 41, 43); 256x256 tiles 360 at 2500, 555 at 4099.  4096 x
// 14336: rows 14.5 at 8, 35.5 at 64; 64x128 tiles 48 to 54 up to 512 rows, in 4
// ranges 25 at 128; 128x128 tiles 130, 256x128 ones 104 at 1777.
struct TileCost {
    int tile;
    double fixed, stage, idle_stage;
};
constexpr TileCost COST_A[] = {{TILE_64x128, 0.5, 0.38, 0.30}, {128, 0.5, 0.53, 0.43}, {TILE_256x128, 3.4, 0.92, 0.92},
                               {256, 6.0, 1.27, 1.27}};
constexpr TileCost COST_B[] = {{128, 0.3, 0.70, 0.58}, {TILE_256x128, 1.5, 1.04, 1.04}};

static int tile_bm(int tile) { return tile > 1000 ? tile / 1000 : tile; }
static int tile_bn(int tile) { return tile > 1000 ? tile % 1000 : tile; }

struct FusedPlan {
    int tile;                    // 0: the row kernel
    int ranges;                  // of K; 1: not split
    double us;
};
static FusedPlan fused_plan(const FusedArgs& a, int cus) {
    const int64_t b_rows = a.gated ? 2 * a.n : a.n, nk = (a.k + BK - 1) / BK;
    const double b_bytes = (double)b_rows * a.k, work = b_bytes + (double)a.m * a.k;
    const int64_t wgs = (b_rows + 31) / 32, cols = wgs < 512 && !a.gated ? 16 : 32;     // as launch_gemm_rows cuts it
    const double a_read = (double)((b_rows + cols - 1) / cols) * ((a.m + 15) / 16 * 16) * a.k;
    const double again = (double)((a.m + 63) / 64 - 1);
    const double fed = b_bytes / 5.5e6 + again * b_bytes / 8.0e6 + a_read / 9.3e6;
    const double steps = (double)((nk + 3) / 4) * (a.m <= 16 ? 0.35 : a.m <= 32 ? 0.6 : 1.1);
    FusedPlan best = {0, 1, 4.0 + (fed > steps ? fed : steps) * (a.mx ? 1.1 : 1.0)};
    if (a.m <= 16) return best;                       // the tiles are mostly empty
    const double hbm = 6.0 + work / 5.3e6;
    auto consider = [&](const TileCost& c) {
        // 256x256 tiles only where they hold their registers (fp32 output: 256x128 then)
        if (c.tile == 256 && (a.mx || a.k % BK || a.n % 8)) return;
        const int64_t tiles = ((a.m + tile_bm(c.tile) - 1) / tile_bm(c.tile)) * ((b_rows + tile_bn(c.tile) - 1) / tile_bn(c.tile));
        const int64_t rounds = (tiles + cus - 1) / cus;
        const double stage = 2 * tiles <= cus ? c.idle_stage : c.stage;
        double us = 4.5 + (double)rounds * (c.fixed + stage * (double)nk);
        if (us < hbm) us = hbm;
        if (us < best.us) best = {c.tile, 1, us};
        if (c.tile != TILE_64x128 && c.tile != 128) return;
        const double part = (double)tiles * tile_bm(c.tile) * tile_bn(c.tile) * 8.0;     // bytes written and read
        for (int r = 2; r <= 16 && r * tiles <= cus && nk / r >= 4; r *= 2) {
            // gated: the partial sums hold both projections
            const double longest = (double)((nk + r - 1) / r + (a.mx ? 3 : 0));
            us = 4.5 + c.fixed + (2 * r * tiles <= cus ? c.idle_stage : c.stage) * longest;
            if (us < hbm) us = hbm;
            us += 4.0 + r * part / 4.0e6;
            if (us < best.us) best = {c.tile, r, us};
        }
    };
    if (a.mx)
        for (const TileCost& c : COST_B) consider(c);
    else
        for (const TileCost& c : COST_A) consider(c);
    return best;
}

constexpr int PLAN_CUS = 256;    // the workspace's size may not hang on a device

// Partial sums; behind them the padded scale rows of A and B.
struct PartSpace {
    int64_t rows, pitch, scale_a, scale_b, bytes;
};
static PartSpace part_space(const FusedArgs& a, const FusedPlan& p) {
    PartSpace s = {};
    if (!p.tile) return s;
    const int bm = tile_bm(p.tile), bn = tile_bn(p.tile);
    s.rows = (a.m + bm - 1) / bm * bm;
    s.pitch = ((a.gated ? 2 * a.n : a.n) + bn - 1) / bn * bn;
    s.scale_a = p.ranges > 1 ? p.ranges * s.rows * s.pitch * 4 : 0;
    s.scale_b = s.scale_a + up16(a.m * pad_pitch(a));
    s.bytes = s.scale_b + up16((a.gated ? 2 * a.n : a.n) * pad_pitch(a));
    return s;
}
int64_t gemm_fused_bytes(const FusedArgs& a) { return part_space(a, fused_plan(a, PLAN_CUS)).bytes; }

// The ranges' sums added in order, and the epilogue: a thread takes four columns of a row.
struct FinishArgs {
    FusedArgs f;
    Act act;
    int64_t pitch, part;         // elements: of a row, of a range
    int ranges;
};
constexpr int FIN_THREADS = 256;
__global__ __launch_bounds__(FIN_THREADS) void fused_finish(FinishArgs x) {
    const FusedArgs& a = x.f;
    const int N = (int)a.n, n = ((int)blockIdx.x * FIN_THREADS + (int)threadIdx.x) * 4;
    const int64_t m = blockIdx.y;
    if (n >= N) return;
    const int left = min(4, N - n);
    const float* part = static_cast<const float*>(a.workspace) + m * x.pitch;
    const float sm = a.mx ? 1.0f : static_cast<const float*>(a.scale_a)[m];
    float z[2][4] = {};
    for (int h = 0; h <= a.gated; ++h) {
        const int64_t at = (int64_t)h * N + n;
        float t[4] = {};
        for (int r = 0; r < x.ranges; ++r) {
            const float* p = part + r * x.part + at;
            // the up projection's columns are aligned only where N is a multiple of four
            if ((at & 3) == 0) {
                const v4f v = *reinterpret_cast<const v4f*>(p);
#pragma unroll
                for (int c = 0; c < 4; ++c) t[c] = r ? t[c] + v[c] : v[c];
            } else {
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    if (c < left) t[c] = r ? t[c] + p[c] : p[c];
            }
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            if (c >= left) continue;
            float v = t[c];
            if (!a.mx) v = v * sm * static_cast<const float*>(a.scale_b)[at + c];
            if (a.bias) v += a.bias[at + c];
            z[h][c] = v;
        }
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        if (c >= left) continue;
        float v = x.act.on ? activate(z[0][c], x.act.c1, x.act.c3) : z[0][c];
        if (a.gated) v *= z[1][c];
        const int64_t i = m * N + n + c;
        if (a.f32) {
            if (a.residual) v += static_cast<const float*>(a.residual)[i];
            static_cast<float*>(a.D)[i] = v;
        } else {
            if (a.residual) v += __builtin_bit_cast(float, (uint32_t)static_cast<const uint16_t*>(a.residual)[i] << 16);
            static_cast<uint16_t*>(a.D)[i] = (uint16_t)bf16x2_bits(v, 0.0f);
        }
    }
}

// ---- the experts' products.  Up to this many rows an expert on average the
// row kernel reads the weights faster; above, experts of many rows make it read
// theirs again for every 16.  Row kernel / tiles in us, rows spread evenly, and in
// brackets unevenly (the fullest expert has 4 to 14 times the average):
//                                     4 rows            6                 8                 12                16
//   (a) 64 x 2 x 1408 x 4096    136 / 151         139 / 152         142 / 152         145 / 155         153 / 155
//                              (117 / 132)       (119 / 132)       (143 / 137)       (175 / 156)       (211 / 155)
//       60 x 2048 x 1408         36 / 43           37 / 43           38 / 43           42 / 43           45 / 43
//                               (33 / 34)         (37 / 42)         (48 / 42)         (53 / 42)         (67 / 42)
//       128 x 2 x 1024 x 2048    96 / 105          97 / 106         101 / 105         109 / 107         118 / 107
//                               (81 / 91)         (93 / 93)        (111 / 105)       (152 / 105)       (154 / 105)
//   (b) 64 x 2 x 1408 x 4096    137 / 195         139 / 195         141 / 196         148 / 197         160 / 197
//                              (119 / 162)       (143 / 197)       (155 / 197)       (183 / 202)       (227 / 205)
//       60 x 2048 x 1408         40 / 53           40 / 53           42 / 53           44 / 53           47 / 53
//                               (36 / 51)         (39 / 52)         (53 / 53)         (53 / 53)         (79 / 55)
// The bound is mode (a)'s with uneven experts; mode (b), which has no 64x128 tiles,
// would still gain up to about 10 rows.
constexpr int64_t FEW_ROWS_EXPERT = 6;
static bool few_rows(const FusedArgs& a) { return a.m <= FEW_ROWS_EXPERT * a.experts; }

// The tile of the rest, by the costs above: an expert of c rows has ceil(c / bm)
// tile rows, on average c / bm + 1/2 but at least one.  256x256 tiles count a
// tenth more, since ragged experts fill them less evenly, and 128x128 ones in mode
// (b) 0.8 us a stage.  Measured, mode (a), 64x128 / 128x128 / 256x128 / 256x256 in us: 128 experts of
// 2 x 1024 x 4096 with 32 rows 222 / 229 / 253 / 230, with 128 rows 375 / 308 / 327
// / 276, with 512 rows 977 / 723 / 701 / 594; 60 of 2048 x 1408 with 273 rows
// 127 / 98 / 99 / 105.
static int moe_tile(const FusedArgs& a) {
    const int64_t b_rows = a.gated ? 2 * a.n : a.n, nk = (a.k + BK - 1) / BK;
    int best = 0;
    double best_us = 0.0;
    auto consider = [&](const TileCost& c) {
        if (c.tile == 256 && (a.k % BK || a.n % 8)) return;
        double rows = (double)a.m / (double)a.experts / tile_bm(c.tile) + 0.5;      // of an expert
        if (rows < 1.0) rows = 1.0;
        const double tiles = rows * (double)a.experts * (double)((b_rows + tile_bn(c.tile) - 1) / tile_bn(c.tile));
        const double rounds = (double)((int64_t)(tiles / PLAN_CUS) + 1);
        const double stage = a.mx && c.tile == 128 ? 0.8 : c.stage;
        const double us = rounds * (c.fixed + stage * (double)nk) * (c.tile == 256 ? 1.1 : 1.0);
        if (!best || us < best_us) best = c.tile, best_us = us;
    };
    if (a.mx)
        for (const TileCost& c : COST_B) consider(c);
    else
        for (const TileCost& c : COST_A) consider(c);
    return best;
}

bool moe_gemm_fits(const FusedArgs& a) { return !few_rows(a) || gemm_rows_fits(a); }

struct MoeSpace {
    int64_t tile_rows, row_at, scale, scale_b, bytes;      // byte offsets; the plan comes first
};
static MoeSpace moe_space(const FusedArgs& a) {
    const int bm = tile_bm(moe_tile(a));
    MoeSpace s;
    s.tile_rows = a.m / bm + a.experts;           // at most: sum of ceil(c / bm)
    s.row_at = (16 * (1 + s.tile_rows) + 255) / 256 * 256;
    s.scale = s.row_at + (a.rows ? 4 * bm * s.tile_rows : 0);
    const int64_t pad = pad_pitch(a);
    s.scale_b = s.scale + (a.rows || pad ? up16(a.m * (!a.mx ? 4 : pad ? pad : a.k / 32)) : 0);
    s.bytes = s.scale_b + a.experts * (a.gated ? 2 * a.n : a.n) * pad;
    return s;
}

int64_t moe_gemm_bytes(const FusedArgs& a) { return few_rows(a) ? 0 : moe_space(a).bytes; }

static hipError_t launch_product(const FusedArgs& a, hipStream_t stream) {
    FusedPlan p = fused_plan(a, PLAN_CUS);
    if (p.tile <= 1) return launch_gemm_rows(a, stream);
    TileLaunch t = {};
    hipError_t e = hipGetDevice(&t.dev);
    if (e != hipSuccess) return e;
    e = hipDeviceGetAttribute(&t.cus, hipDeviceAttributeMultiprocessorCount, t.dev);
    if (e != hipSuccess) return e;
    t.tile = p.tile == 256 && a.f32 ? TILE_256x128 : p.tile;
    t.scale_a = a.scale_a;
    const int64_t b_rows = a.gated ? 2 * a.n : a.n;
    const int64_t tiles = ((a.m + tile_bm(p.tile) - 1) / tile_bm(p.tile)) * ((b_rows + tile_bn(p.tile) - 1) / tile_bn(p.tile));
    const PartSpace s = part_space(a, p);
    if (p.ranges * tiles > t.cus) p.ranges = 1;      // a device of fewer CUs: an item a workgroup would not fit
    FusedArgs g = a;
    if (pad_pitch(a)) {
        uint8_t *ws = static_cast<uint8_t*>(a.workspace), *pa = ws + s.scale_a, *pb = ws + s.scale_b;
        const PadArgs pad = {{static_cast<const uint8_t*>(a.scale_a), static_cast<const uint8_t*>(a.scale_b)}, {pa, pb},
                             {a.m, b_rows}, (int)(a.k / 32), (int)(pad_pitch(a) / 4)};
        e = launch_pad(pad, stream);
        if (e != hipSuccess) return e;
        t.scale_a = pa, g.scale_b = pb;
    }
    if (p.ranges == 1) return a.mx ? launch_fused<true, false>(g, t, stream) : launch_fused<false, false>(g, t, stream);
    // the plain product of all of B's rows
    g.n = b_rows, g.gated = 0, g.f32 = 1;
    g.bias = nullptr, g.residual = nullptr, g.D = a.workspace;
    t.ranges = p.ranges, t.pitch = (int32_t)s.pitch, t.part_rows = (int32_t)s.rows;
    e = a.mx ? launch_fused_part<true, false, EPI_PARTIAL>(g, t, stream) : launch_fused_part<false, false, EPI_PARTIAL>(g, t, stream);
    if (e != hipSuccess) return e;
    const FinishArgs f = {a, act_of(a.act), s.pitch, s.rows * s.pitch, p.ranges};
    fused_finish<<<dim3((unsigned)((a.n + 4 * FIN_THREADS - 1) / (4 * FIN_THREADS)), (unsigned)a.m), dim3(FIN_THREADS), 0, stream>>>(f);
    return hipGetLastError();
}

hipError_t launch_gemm_fused(const FusedArgs& a, hipStream_t stream) {
    if (!a.expert_start) return launch_product(a, stream);
    if (few_rows(a)) return launch_gemm_rows(a, stream);
    TileLaunch t = {};
    hipError_t e = hipGetDevice(&t.dev);
    if (e != hipSuccess) return e;
    e = hipDeviceGetAttribute(&t.cus, hipDeviceAttributeMultiprocessorCount, t.dev);
    if (e != hipSuccess) return e;
    t.tile = moe_tile(a);
    t.scale_a = a.scale_a;
    const MoeSpace s = moe_space(a);
    uint8_t* ws = static_cast<uint8_t*>(a.workspace);
    t.tile_rows = s.tile_rows;
    t.plan = reinterpret_cast<int32_t*>(ws);
    if (a.rows) {
        t.row_at = reinterpret_cast<uint32_t*>(ws + s.row_at);
        t.scale_a = ws + s.scale;
    }
    moe_plan<<<dim3((unsigned)s.tile_rows), dim3(PLAN_THREADS), 0, stream>>>(
        a.expert_start, a.rows, a.scale_a, (int)a.experts, (int)a.m, (int)a.a_rows, (int)a.k, a.mx, tile_bm(t.tile),
        const_cast<int32_t*>(t.plan), const_cast<uint32_t*>(t.row_at), a.rows ? ws + s.scale : nullptr);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (t.tile == 256 && a.f32) t.tile = TILE_256x128;      // the same rows a tile
    FusedArgs g = a;
    if (pad_pitch(a)) {
        // A's rows, too, unless the plan has put them in order already
        PadArgs pad = {{static_cast<const uint8_t*>(a.scale_a), static_cast<const uint8_t*>(a.scale_b)},
                       {ws + s.scale, ws + s.scale_b}, {a.rows ? 0 : a.m, a.experts * (a.gated ? 2 * a.n : a.n)},
                       (int)(a.k / 32), (int)(pad_pitch(a) / 4)};
        e = launch_pad(pad, stream);
        if (e != hipSuccess) return e;
        t.scale_a = ws + s.scale, g.scale_b = ws + s.scale_b;
    }
    return a.mx ? launch_fused<true, true>(g, t, stream) : launch_fused<false, true>(g, t, stream);
}
#endif  // FP8G_FUSED_PART == 0

}  // namespace fp8g
