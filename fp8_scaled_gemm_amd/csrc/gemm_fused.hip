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
// Compiled once per mode and kind (FP8G_FUSED_PART = 4 * gated + 2 * MX + MOE).

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
    constexpr int LDS_BYTES = Ring<MX, KTAIL, TILE>::LDS_TOTAL;
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
    const int64_t tiles = (MOE ? t.tile_rows : (a.m + BM - 1) / BM) * ((a.n + BNO - 1) / BNO);
    const TileExtra ex = {a.bias, a.residual, act_of(a.act), t.plan, t.row_at, t.row_at ? (uint32_t)(a.a_rows * a.k) : 0u};
    kern<<<dim3((unsigned)(tiles < t.cus ? tiles : t.cus)), dim3(NTHREADS), LDS_BYTES, stream>>>(
        (int)a.m, (int)a.n, (int)a.k, a.A, a.B, t.scale_a, a.scale_b, a.D, ex);
    return hipGetLastError();
}

template <bool MX, bool MOE, int EPI>
hipError_t launch_fused_part(const FusedArgs& a, const TileLaunch& t, hipStream_t stream) {
    auto go = [&](auto tile) {
        constexpr int TILE = decltype(tile)::value;
        if (a.k % BK)
            return a.f32 ? launch_tile<MX, true, true, TILE, EPI, MOE>(a, t, stream)
                         : launch_tile<MX, false, true, TILE, EPI, MOE>(a, t, stream);
        return a.f32 ? launch_tile<MX, true, false, TILE, EPI, MOE>(a, t, stream)
                     : launch_tile<MX, false, false, TILE, EPI, MOE>(a, t, stream);
    };
    if constexpr (!MX) {
        if (t.tile == TILE_64x128) return go(std::integral_constant<int, TILE_64x128>{});
        if constexpr (!MOE)
            if (t.tile == 256) return launch_tile<MX, false, false, 256, EPI, MOE>(a, t, stream);
    }
    if (t.tile == 128) return go(std::integral_constant<int, 128>{});
    return go(std::integral_constant<int, TILE_256x128>{});
}

#ifndef FP8G_FUSED_PART
#error "FP8G_FUSED_PART"
#endif
#define FP8G_FUSED(KW, MX, MOE, EPI) \
    KW hipError_t launch_fused_part<MX, MOE, EPI>(const FusedArgs&, const TileLaunch&, hipStream_t);
FP8G_FUSED(template, ((FP8G_FUSED_PART & 2) != 0), ((FP8G_FUSED_PART & 1) != 0), ((FP8G_FUSED_PART & 4) ? EPI_GATED : EPI_LINEAR))

#if FP8G_FUSED_PART == 0
FP8G_FUSED(extern template, false, true, EPI_LINEAR)
FP8G_FUSED(extern template, true, false, EPI_LINEAR)
FP8G_FUSED(extern template, true, true, EPI_LINEAR)
FP8G_FUSED(extern template, false, false, EPI_GATED)
FP8G_FUSED(extern template, false, true, EPI_GATED)
FP8G_FUSED(extern template, true, false, EPI_GATED)
FP8G_FUSED(extern template, true, true, EPI_GATED)

template <bool MX, bool MOE>
static hipError_t launch_fused(const FusedArgs& a, const TileLaunch& t, hipStream_t stream) {
    return a.gated ? launch_fused_part<MX, MOE, EPI_GATED>(a, t, stream) : launch_fused_part<MX, MOE, EPI_LINEAR>(a, t, stream);
}

constexpr int PLAN_THREADS = 256, PLAN_EXPERTS = 1024;

// One workgroup per possible tile row t: every one counts the experts' tile
// rows (an expert of c slots has ceil(c / bm)); the expert that holds t writes it down.
__global__ __launch_bounds__(PLAN_THREADS) void moe_plan(const int32_t* __restrict__ start, const int32_t* __restrict__ rows,
                                                         const void* __restrict__ sa, int experts, int slots, int a_rows,
                                                         int k, int mx, int bm, int32_t* __restrict__ plan,
                                                         uint32_t* __restrict__ row_at, void* __restrict__ scale) {
    __shared__ int sum[PLAN_THREADS];
    __shared__ int mine[3];
    constexpr int PER = PLAN_EXPERTS / PLAN_THREADS;
    const int tid = threadIdx.x, t = blockIdx.x;
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
    sum[tid] = tiles;
    __syncthreads();
    for (int off = 1; off < PLAN_THREADS; off <<= 1) {
        const int v = tid >= off ? sum[tid - off] : 0;
        __syncthreads();
        sum[tid] += v;
        __syncthreads();
    }
    const int total = sum[PLAN_THREADS - 1];
    if (t == 0 && tid == 0) plan[0] = total;
    if (t >= total) return;
    int at = sum[tid] - tiles;
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
    const int nblk = k / 32;
    if (nblk % 4 == 0) {
        const int nw = nblk / 4;
        for (int i = tid; i < here * nw; i += PLAN_THREADS) {
            const int r = i / nw, a = min(max(rows[m0 + r], 0), a_rows - 1);
            static_cast<uint32_t*>(scale)[(int64_t)(m0 + r) * nw + i % nw] =
                static_cast<const uint32_t*>(sa)[(int64_t)a * nw + i % nw];
        }
    } else {
        for (int i = tid; i < here * nblk; i += PLAN_THREADS) {
            const int r = i / nblk, a = min(max(rows[m0 + r], 0), a_rows - 1);
            static_cast<uint8_t*>(scale)[(int64_t)(m0 + r) * nblk + i % nblk] =
                static_cast<const uint8_t*>(sa)[(int64_t)a * nblk + i % nblk];
        }
    }
}

// Products of at most this many rows (of an expert: on average) go to gemm_rows.hip.
constexpr int64_t FEW_ROWS = 64, FEW_ROWS_EXPERT = 32;

static bool few_rows(const FusedArgs& a) {
    return a.expert_start ? a.m <= FEW_ROWS_EXPERT * a.experts : a.m <= FEW_ROWS;
}

// The experts' tile by the rows an expert has on average.
static int moe_tile(const FusedArgs& a) {
    const int64_t rows = a.m / a.experts;
    if (!a.mx && rows <= 64) return TILE_64x128;
    return rows <= 128 ? 128 : TILE_256x128;
}
static int tile_bm(int tile) { return tile > 1000 ? tile / 1000 : tile; }

struct MoeSpace {
    int64_t tile_rows, row_at, scale, bytes;      // byte offsets behind the plan, which comes first
};
static MoeSpace moe_space(const FusedArgs& a) {
    const int bm = tile_bm(moe_tile(a));
    MoeSpace s;
    s.tile_rows = a.m / bm + a.experts;           // at most: sum of ceil(c / bm)
    s.row_at = (16 * (1 + s.tile_rows) + 255) / 256 * 256;
    s.scale = s.row_at + (a.rows ? 4 * bm * s.tile_rows : 0);
    s.bytes = s.scale + (a.rows ? (a.m * (a.mx ? a.k / 32 : 4) + 15) / 16 * 16 : 0);
    return s;
}

int64_t moe_gemm_bytes(const FusedArgs& a) { return few_rows(a) ? 0 : moe_space(a).bytes; }

hipError_t launch_gemm_fused(const FusedArgs& a, hipStream_t stream) {
    if (few_rows(a)) return launch_gemm_rows(a, stream);
    TileLaunch t = {};
    hipError_t e = hipGetDevice(&t.dev);
    if (e != hipSuccess) return e;
    e = hipDeviceGetAttribute(&t.cus, hipDeviceAttributeMultiprocessorCount, t.dev);
    if (e != hipSuccess) return e;
    t.scale_a = a.scale_a;
    if (!a.expert_start) {
        // the scaled products' choice, but 256x256 tiles only where they hold their
        // registers: per-row scales, bf16 output, K in whole stages
        t.tile = gemm_tile_of(a.m, a.gated ? 2 * a.n : a.n, a.k, a.mx, t.cus);
        if (t.tile == 256 && (a.mx || a.f32 || a.k % BK)) t.tile = TILE_256x128;
        return a.mx ? launch_fused<true, false>(a, t, stream) : launch_fused<false, false>(a, t, stream);
    }
    t.tile = moe_tile(a);
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
    return a.mx ? launch_fused<true, true>(a, t, stream) : launch_fused<false, true>(a, t, stream);
}
#endif  // FP8G_FUSED_PART == 0

}  // namespace fp8g
