// FP8 scaled GEMM: the schedule of a launch, the split workspace and the
// launches of the kernel in gemm_tile.h.

#include <algorithm>
#include <atomic>
#include <map>
#include <mutex>
#include <type_traits>
#include <utility>

#include "gemm_tile.h"
#include "launch.h"

namespace fp8g {

template <bool MX, bool OUT_F32, bool KTAIL, int FA, int FB, int TILE, bool SPLIT>
__global__ __launch_bounds__(NTHREADS, 1) void gemm_fp8_kernel(
    int M, int N, int K, const uint8_t* __restrict__ A, const uint8_t* __restrict__ B,
    const float* __restrict__ sa, const float* __restrict__ sb, const uint8_t* __restrict__ ea,
    const uint8_t* __restrict__ eb, void* __restrict__ Dv, int tiles_whole, int split, float* __restrict__ ws,
    int* __restrict__ cnt) {
    gemm_tiles<MX, OUT_F32, KTAIL, FA, FB, TILE, SPLIT, EPI_NONE, false>(M, N, K, A, B, sa, sb, ea, eb, Dv, tiles_whole,
                                                                          split, ws, cnt, TileExtra{});
}

// ---- split items (mode (a), 128x128 tiles, K a multiple of 128).  When the
// tiles leave a last round at most half full (r = tiles % CUs tiles, 2r <=
// CUs), each of those r tiles may be split over K into S equal ranges of
// stages (S <= min(CUs / r, 4), S dividing the stages, at least 4 stages
// each), one work item per range, so that the last round keeps up to S r CUs
// busy instead of r.  Each item's partial tile then goes through memory (see
// the split reduction in the kernel), so S is chosen by a cost model fitted
// to measurements on MI355X: a stage of a 128x128 tile takes about 0.37 us
// whatever the number of tiles (the loop is latency-bound), and the exchange
// about 1.5 us plus its traffic (every item's 64 KB partial written, S - 1 of
// S read back) at about 4 TB/s.  Measured against unsplit tiles:
// 128x128x4096 16.7 -> 12.2 us (S = 4), 2048x1024x8192 31.2 -> 26.3 us
// (S = 2), 1024x1024x4096 17.1 -> 15.9 us (S = 4); 2048x1024x4096 gained
// nothing (18.2 / 18.4 us: 16 stages saved, 24 MB exchanged) and
// 2048x1024x1024 lost 44%, so neither splits.  (Those two and 1024x1024x4096
// now run on 64x128 tiles; see prefer_tile64.)  The workspace holds the arrival
// counters (one int per split tile, padded to 256 bytes) and the partial
// tiles (S r <= CUs of them).
struct SplitPlan {
    int tiles_whole, split;
};
constexpr double T_STAGE_US = 0.37, T_FIXED_US = 1.5, BYTES_PER_US = 4.0e6;
constexpr double PART_BYTES = 128.0 * 128.0 * 4.0;
// predicted K loop and exchange of r tiles of nk stages split s ways
static double split_us(int64_t r, int s, int64_t nk) {
    const double moved = (double)(s * r) * PART_BYTES * (1.0 + (double)(s - 1) / s);
    return (double)(nk / s) * T_STAGE_US + T_FIXED_US + moved / BYTES_PER_US;
}
static SplitPlan split_plan(int64_t tiles, int cus, int64_t nk) {
    SplitPlan p{(int)tiles, 1};
    const int64_t r = tiles % cus;
    if (r == 0 || 2 * r > cus || nk < 8) return p;
    double best = 0.1 * (double)nk * T_STAGE_US;   // require a predicted gain of 10% at least
    for (int s = 2; s <= 4 && s <= cus / r; ++s) {
        if (nk % s != 0 || nk / s < 4) continue;
        const double gain = (double)nk * T_STAGE_US - split_us(r, s, nk);
        if (gain > best) {
            best = gain;
            p.split = s;
            p.tiles_whole = (int)(tiles - r);
        }
    }
    return p;
}
// 64x128 tiles or 128x128 tiles split over K, for a problem whose 128x128
// tiles fill at most half of the CUs (so its 64x128 tiles fit one round).
// Fitted to measurements on MI355X: one round of 64x128 tiles takes about
// 4.4 us plus 0.26 us per stage, one of 128x128 tiles 5.4 us plus the split
// schedule's predicted loop and exchange; 64x128 tiles are taken when they
// are predicted at least 5% faster.  Measured (split / 64x128 tiles):
// 1024x1024x8192 21.2 / 23.0 us, 512x512x8192 16.0 / 20.8 us, 256x256x16384
// 22.0 / 37.6 us (split taken); 2048x1024x8192 27.1 / 25.2 us, 1024x512x4096
// 13.7 / 12.3 us (64x128 taken).  The model misses the smallest problems by
// a few percent: 128x128x4096 12.9 / 12.1 us and 1024x256x4096 13.0 /
// 12.3 us take the split.
static bool prefer_tile64(int64_t tiles128, int cus, int64_t nk, bool tail) {
    constexpr double T64_FIXED_US = 4.4, T64_STAGE_US = 0.26, T128_FIXED_US = 5.4;
    if (tail) return true;
    const SplitPlan sp = split_plan(tiles128, cus, nk);
    if (sp.split == 1) return true;
    return T64_FIXED_US + (double)nk * T64_STAGE_US <
           0.95 * (T128_FIXED_US + split_us(tiles128 - sp.tiles_whole, sp.split, nk));
}
static int64_t ws_cnt_bytes(int cus) { return ((int64_t)cus * 4 + 255) / 256 * 256; }
// bytes of workspace any split launch on a device with `cus` CUs may use
static int64_t split_ws_bytes(int cus) { return ws_cnt_bytes(cus) + (int64_t)cus * 256 * 256 * 4; }

// Zeroes n ints (the arrival counters of a new split workspace): a kernel
// rather than a memset, so that no memset node can reach a captured graph.
static __global__ __launch_bounds__(256) void clear_counters_kernel(int* __restrict__ p, int n) {
    const int i = (int)(blockIdx.x * 256 + threadIdx.x);
    if (i < n) p[i] = 0;
}

// The calling stream's split workspace (split_ws_bytes), allocated on the
// stream's first split launch and kept for the life of the process; its
// counters are cleared on the stream before the first use.  One workspace per
// (device, stream): launches on one stream run in order, so they never share
// it at the same time, and other streams have their own.  A stream that is
// being captured into a graph gets its workspace if it has one and nullptr
// otherwise (nothing is allocated or cleared during a capture): the launch
// then takes the unsplit schedule.
static hipError_t stream_workspace(int dev, hipStream_t stream, int cus, void** out) {
    static std::mutex mu;
    static std::map<std::pair<int, uintptr_t>, void*> cache;
    hipStreamCaptureStatus cs = hipStreamCaptureStatusNone;
    hipError_t e = hipStreamIsCapturing(stream, &cs);
    if (e != hipSuccess) return e;
    std::lock_guard<std::mutex> lock(mu);
    const auto key = std::make_pair(dev, reinterpret_cast<uintptr_t>(stream));
    const auto it = cache.find(key);
    if (it != cache.end()) {
        *out = it->second;
        return hipSuccess;
    }
    *out = nullptr;
    if (cs != hipStreamCaptureStatusNone) return hipSuccess;
    void* p = nullptr;
    e = hipMalloc(&p, (size_t)split_ws_bytes(cus));
    if (e != hipSuccess) return e;
    const int nc = (int)(ws_cnt_bytes(cus) / 4);
    clear_counters_kernel<<<dim3((unsigned)((nc + 255) / 256)), dim3(256), 0, stream>>>(reinterpret_cast<int*>(p), nc);
    e = hipGetLastError();
    if (e != hipSuccess) {
        (void)hipFree(p);
        return e;
    }
    cache.emplace(key, p);
    *out = p;
    return hipSuccess;
}

template <bool MX, bool OUT_F32, bool KTAIL, int FA, int FB, int TILE, bool SPLIT>
static hipError_t launch_one(int64_t m, int64_t n, int64_t k, const uint8_t* A, const uint8_t* B,
                             const float* sa, const float* sb, const uint8_t* ea, const uint8_t* eb, void* D,
                             int dev, int cus, const SplitPlan& sp, void* ws, hipStream_t stream) {
    auto kern = gemm_fp8_kernel<MX, OUT_F32, KTAIL, FA, FB, TILE, SPLIT>;
    constexpr int LDS_BYTES = Ring<MX, KTAIL, TILE>::LDS_TOTAL;
    // up to 160 KB of dynamic LDS is above the default launch limit; raise it
    // once per device (the attribute is set for the current device).  Setting
    // it twice from racing threads is harmless.
    static std::atomic<uint64_t> configured{0};
    const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;
    if (!bit || !(configured.load(std::memory_order_acquire) & bit)) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kern),
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, LDS_BYTES);
        if (e != hipSuccess) return e;
        configured.fetch_or(bit, std::memory_order_release);
    }
    constexpr int BM = Geo<TILE>::BM, BN = Geo<TILE>::BN;
    const int64_t tiles = ((m + BM - 1) / BM) * ((n + BN - 1) / BN);
    const int64_t items = SPLIT ? sp.tiles_whole + (tiles - sp.tiles_whole) * sp.split : tiles;
    const int64_t grid = items < cus ? items : cus;   // persistent: at most one workgroup per CU
    int* cnt = SPLIT ? reinterpret_cast<int*>(ws) : nullptr;
    float* part = SPLIT ? reinterpret_cast<float*>(reinterpret_cast<char*>(ws) + ws_cnt_bytes(cus)) : nullptr;
    kern<<<dim3((unsigned)grid), dim3(NTHREADS), LDS_BYTES, stream>>>((int)m, (int)n, (int)k, A, B, sa, sb, ea,
                                                                      eb, D, sp.tiles_whole, sp.split, part, cnt);
    return hipGetLastError();
}

// The schedule of a launch on a device with `cus` CUs: the tile shape and,
// for 128x128 tiles in mode (a) with K a multiple of 128, the split plan.  The
// launch and fp8g_gemm_schedule both take it from here.
//   128x128 tiles when 256x256 tiles would leave at least half of the CUs
//   idle: four times the tiles, each at a lower matrix-core rate.  Mode (a)
//   also when the 256x256 tiles spill just past one round (at most an eighth
//   of a second one): 4352x4096 (272 tiles) ran 4-14% faster on 128x128 tiles
//   at K = 1024..8192, while at 1.5 and 2 rounds the 256x256 tiles were
//   4-35% faster.
//   64x128 tiles (mode (a)) when 128x128 tiles would leave at least half of
//   the CUs idle and splitting them over K is not predicted faster
//   (prefer_tile64): twice the workgroups, each with half the matrix-core
//   work per stage.
//   256x128 tiles in place of 256x256 ones when they need at most 1.5 times
//   the rounds: a round of 256x128 tiles costs 0.57-0.66 of a round of
//   256x256 tiles in mode (b) and 0.5-0.65 in mode (a) (measured at 132 to
//   896 tiles of 256x256), so they pay where 256x256 tiles leave a last round
//   partly empty and lose where that round is nearly full.  Measured, mode (b)
//   (256x256 / 256x128 tiles): 2600x2900x1024 22.7 / 17.9 us (132 tiles of
//   256x256; 1 round against 1), 4352x4096x640 25.4 / 23.0 us (272; 2 rounds
//   against 3), 4096x6144x2048 55.9 / 55.2 us (384; 2 against 3);
//   3072x4096x1024 18.5 / 21.4 us (192; 1 against 2), 4096x8192x2048 66.4 /
//   76.0 us (512; 2 against 4), 4096x14336x4096 197.9 / 225.0 us (896; 4
//   against 7).  Mode (a): 2600x2900 at K = 1024 / 4096 / 8192 22.1 / 17.6,
//   45.4 / 35.7, 72.9 / 58.4 us (1 round against 1); 4608x4608x1024 31.5 /
//   29.2 us, 4608x4608x8192 153.0 / 151.2 us, 4096x6144x1024 31.9 / 29.6 us,
//   4864x4096x4096 83.1 / 80.4 us (2 against 3); 3072x4096x1024 18.0 /
//   18.1 us (1 against 2: not taken).  The mode (a) spill shapes above keep
//   128x128 tiles: 4352x4096 at K = 1024 ran 29.3 us on them against 30.9 us
//   on 256x128 tiles.
//   Only 128x128 tiles split: the 256x256 split kernel would spill around its
//   last step.
struct Schedule {
    int tile;       // 256, 128, TILE_64x128 or TILE_256x128
    SplitPlan sp;   // split == 1: no split
};
static Schedule gemm_schedule(int64_t m, int64_t n, int64_t k, bool mx, int cus) {
    const bool tail = (k % BK) != 0;
    const int64_t tiles256 = ((m + 255) / 256) * ((n + 255) / 256);
    const bool spill = !mx && tiles256 > cus && 8 * (tiles256 - cus) <= cus;
    if (2 * tiles256 <= cus || spill) {
        const int64_t tiles128 = ((m + 127) / 128) * ((n + 127) / 128);
        if (!mx) {
            if (!spill && 2 * tiles128 <= cus && prefer_tile64(tiles128, cus, k / BK, tail)) {
                const int64_t tiles64 = ((m + 63) / 64) * ((n + 127) / 128);
                return {TILE_64x128, {(int)tiles64, 1}};
            }
            if (!tail) return {128, split_plan(tiles128, cus, k / BK)};
        }
        return {128, {(int)tiles128, 1}};
    }
    const int64_t tiles_h = ((m + 255) / 256) * ((n + 127) / 128);   // 256x128 tiles
    const int64_t rounds = (tiles256 + cus - 1) / cus, rounds_h = (tiles_h + cus - 1) / cus;
    if (2 * rounds_h <= 3 * rounds) return {TILE_256x128, {(int)tiles_h, 1}};
    return {256, {(int)tiles256, 1}};
}

template <bool MX, int FA, int FB, int TILE>
static hipError_t launch_tiled(int64_t m, int64_t n, int64_t k, const uint8_t* A, const uint8_t* B, const float* sa,
                               const float* sb, const uint8_t* ea, const uint8_t* eb, void* D, int out_f32, int dev,
                               int cus, const SplitPlan& sp, void* fixed_ws, hipStream_t stream) {
    // a K tail (k not a multiple of the 128-byte stage) zero-fills the bytes
    // past K and, in mode (b), reads the scales byte by byte from global memory
    const bool tail = (k % BK) != 0;
    constexpr int BM = Geo<TILE>::BM, BN = Geo<TILE>::BN;
    const int64_t tiles = ((m + BM - 1) / BM) * ((n + BN - 1) / BN);
    if constexpr (!MX && TILE == 128) {
        if (!tail && sp.split > 1) {
            void* ws = fixed_ws;   // the caller's fixed workspace (of split_ws_bytes(cus) at least), or the stream's
            if (!ws) {
                const hipError_t e = stream_workspace(dev, stream, cus, &ws);
                if (e != hipSuccess) return e;
            }
            if (ws)   // none: a capture on a stream without a workspace runs unsplit
                return out_f32 ? launch_one<MX, true, false, FA, FB, TILE, true>(m, n, k, A, B, sa, sb, ea, eb, D,
                                                                                 dev, cus, sp, ws, stream)
                               : launch_one<MX, false, false, FA, FB, TILE, true>(m, n, k, A, B, sa, sb, ea, eb, D,
                                                                                  dev, cus, sp, ws, stream);
        }
    }
    const SplitPlan whole{(int)tiles, 1};
    if (out_f32)
        return tail ? launch_one<MX, true, true, FA, FB, TILE, false>(m, n, k, A, B, sa, sb, ea, eb, D, dev, cus, whole,
                                                                      nullptr, stream)
                    : launch_one<MX, true, false, FA, FB, TILE, false>(m, n, k, A, B, sa, sb, ea, eb, D, dev, cus,
                                                                       whole, nullptr, stream);
    return tail ? launch_one<MX, false, true, FA, FB, TILE, false>(m, n, k, A, B, sa, sb, ea, eb, D, dev, cus, whole,
                                                                   nullptr, stream)
                : launch_one<MX, false, false, FA, FB, TILE, false>(m, n, k, A, B, sa, sb, ea, eb, D, dev, cus, whole,
                                                                    nullptr, stream);
}

template <bool MX, int FA, int FB>
hipError_t launch_fmt(int64_t m, int64_t n, int64_t k, const uint8_t* A, const uint8_t* B, const float* sa,
                      const float* sb, const uint8_t* ea, const uint8_t* eb, void* D, int out_f32, void* fixed_ws,
                      hipStream_t stream) {
    int dev = 0, cus = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    e = hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev);
    if (e != hipSuccess) return e;
    const Schedule sc = gemm_schedule(m, n, k, MX, cus);
    if constexpr (!MX) {
        if (sc.tile == TILE_64x128)
            return launch_tiled<MX, FA, FB, TILE_64x128>(m, n, k, A, B, sa, sb, ea, eb, D, out_f32, dev, cus, sc.sp,
                                                         fixed_ws, stream);
    }
    if (sc.tile == TILE_256x128)
        return launch_tiled<MX, FA, FB, TILE_256x128>(m, n, k, A, B, sa, sb, ea, eb, D, out_f32, dev, cus, sc.sp,
                                                      fixed_ws, stream);
    if (sc.tile == 128)
        return launch_tiled<MX, FA, FB, 128>(m, n, k, A, B, sa, sb, ea, eb, D, out_f32, dev, cus, sc.sp, fixed_ws,
                                             stream);
    return launch_tiled<MX, FA, FB, 256>(m, n, k, A, B, sa, sb, ea, eb, D, out_f32, dev, cus, sc.sp, fixed_ws, stream);
}

// Each operand-format pair's kernels may be compiled in an object of their
// own (FP8G_GEMM_FMT = 2 * FA + FB, set by the library build so that the four
// pairs compile in parallel); the object with FP8G_GEMM_FMT 0 also holds the
// dispatch below.  Without the macro one object holds everything.
#ifndef FP8G_GEMM_FMT
#define FP8G_GEMM_FMT -1
#endif

#define FP8G_FMT_PAIR(KW, FA, FB)                                                                              \
    KW hipError_t launch_fmt<false, FA, FB>(int64_t, int64_t, int64_t, const uint8_t*, const uint8_t*,          \
                                            const float*, const float*, const uint8_t*, const uint8_t*, void*,  \
                                            int, void*, hipStream_t);                                           \
    KW hipError_t launch_fmt<true, FA, FB>(int64_t, int64_t, int64_t, const uint8_t*, const uint8_t*,           \
                                           const float*, const float*, const uint8_t*, const uint8_t*, void*,   \
                                           int, void*, hipStream_t);

#if FP8G_GEMM_FMT >= 0
FP8G_FMT_PAIR(extern template, 0, 0)
FP8G_FMT_PAIR(extern template, 0, 1)
FP8G_FMT_PAIR(extern template, 1, 0)
FP8G_FMT_PAIR(extern template, 1, 1)
#endif
#if FP8G_GEMM_FMT == 0
FP8G_FMT_PAIR(template, 0, 0)
#elif FP8G_GEMM_FMT == 1
FP8G_FMT_PAIR(template, 0, 1)
#elif FP8G_GEMM_FMT == 2
FP8G_FMT_PAIR(template, 1, 0)
#elif FP8G_GEMM_FMT == 3
FP8G_FMT_PAIR(template, 1, 1)
#endif

#if FP8G_GEMM_FMT <= 0
template <bool MX>
static hipError_t launch_mode(int64_t m, int64_t n, int64_t k, const uint8_t* A, int fmt_a, const uint8_t* B,
                              int fmt_b, const float* sa, const float* sb, const uint8_t* ea, const uint8_t* eb,
                              void* D, int out_f32, void* fixed_ws, hipStream_t stream) {
    if ((fmt_a != 0 && fmt_a != 1) || (fmt_b != 0 && fmt_b != 1)) return hipErrorInvalidValue;
    if (fmt_a == 0)
        return fmt_b == 0 ? launch_fmt<MX, 0, 0>(m, n, k, A, B, sa, sb, ea, eb, D, out_f32, fixed_ws, stream)
                          : launch_fmt<MX, 0, 1>(m, n, k, A, B, sa, sb, ea, eb, D, out_f32, fixed_ws, stream);
    return fmt_b == 0 ? launch_fmt<MX, 1, 0>(m, n, k, A, B, sa, sb, ea, eb, D, out_f32, fixed_ws, stream)
                      : launch_fmt<MX, 1, 1>(m, n, k, A, B, sa, sb, ea, eb, D, out_f32, fixed_ws, stream);
}

// 32-bit buffer offsets: a 256-row panel of K bytes stays below 2^31, so the
// out-of-range offset 2^31 plus any scalar offset still fits in 32 bits.
static bool fits(int64_t m, int64_t n, int64_t k) {
    const int64_t tiles = ((m + 127) / 128) * ((n + 127) / 128);
    return m < (1LL << 31) && n < (1LL << 31) && k < (1LL << 23) && tiles < (1LL << 31);
}

hipError_t schedule_gemm(int64_t m, int64_t n, int64_t k, int mx, int cus, int* tile_m, int* tile_n, int* split,
                         int* split_tiles) {
    if (!fits(m, n, k)) return hipErrorInvalidValue;
    const Schedule sc = gemm_schedule(m, n, k, mx != 0, cus);
    *tile_m = sc.tile > 1000 ? sc.tile / 1000 : sc.tile;
    *tile_n = sc.tile > 1000 ? sc.tile % 1000 : sc.tile;
    *split = sc.sp.split;
    const int64_t tiles = ((m + *tile_m - 1) / *tile_m) * ((n + *tile_n - 1) / *tile_n);
    *split_tiles = sc.sp.split > 1 ? (int)(tiles - sc.sp.tiles_whole) : 0;
    return hipSuccess;
}

hipError_t launch_gemm_scaled(int64_t m, int64_t n, int64_t k, const uint8_t* A, int fmt_a, const uint8_t* B,
                              int fmt_b, const float* sa, const float* sb, void* D, int out_f32,
                              hipStream_t stream) {
    if (!fits(m, n, k)) return hipErrorInvalidValue;
    return launch_mode<false>(m, n, k, A, fmt_a, B, fmt_b, sa, sb, nullptr, nullptr, D, out_f32, nullptr, stream);
}

// ---- fixed split workspace, for callers that cannot allocate
// (fp8_gemm_scaled_noalloc).  A file-scope device array, SCRATCH_BYTES =
// split_ws_bytes(256): enough for every split launch on a device of up to 256
// CUs.  It is zero when the library is loaded (its counters must start at
// zero) and every split launch leaves its counters at zero again.  In host
// code the name `scratch` stands for a host-side shadow, not for device
// memory: its address on each device comes from hipGetSymbolAddress, taken
// once per device with that device current, and only that address is passed
// to kernels.  Every call on a device shares that device's array, so calls
// that overlap on one device race.
constexpr int64_t SCRATCH_BYTES = (int64_t)256 * 256 * 256 * 4 + 1024;
static __device__ __align__(256) unsigned char scratch[SCRATCH_BYTES];
static_assert(SCRATCH_BYTES >= (256 * 4 + 255) / 256 * 256 + (int64_t)256 * 256 * 256 * 4, "scratch size");

static hipError_t scratch_address(int dev, void** out) {
    constexpr int MAX_DEV = 64;
    static std::mutex mu;
    static void* addr[MAX_DEV] = {};
    if (dev < 0 || dev >= MAX_DEV) return hipErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu);
    if (!addr[dev]) {
        void* p = nullptr;
        const hipError_t e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
        if (e != hipSuccess) return e;
        addr[dev] = p;
    }
    *out = addr[dev];
    return hipSuccess;
}

hipError_t launch_gemm_scaled_noalloc(int64_t m, int64_t n, int64_t k, const uint8_t* A, const uint8_t* B,
                                      const float* sa, const float* sb, void* D, int out_f32, hipStream_t stream) {
    if (!fits(m, n, k)) return hipErrorInvalidValue;
    int dev = 0, cus = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    e = hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev);
    if (e != hipSuccess) return e;
    if (split_ws_bytes(cus) > SCRATCH_BYTES) return hipErrorOutOfMemory;   // a device of more than 256 CUs
    void* ws = nullptr;
    e = scratch_address(dev, &ws);
    if (e != hipSuccess) return e;
    return launch_mode<false>(m, n, k, A, 0, B, 0, sa, sb, nullptr, nullptr, D, out_f32, ws, stream);
}

hipError_t launch_gemm_mx(int64_t m, int64_t n, int64_t k, const uint8_t* A, int fmt_a, const uint8_t* B,
                          int fmt_b, const uint8_t* ea, const uint8_t* eb, void* D, int out_f32,
                          hipStream_t stream) {
    if (!fits(m, n, k)) return hipErrorInvalidValue;
    return launch_mode<true>(m, n, k, A, fmt_a, B, fmt_b, nullptr, nullptr, ea, eb, D, out_f32, nullptr, stream);
}
#endif  // FP8G_GEMM_FMT <= 0

}  // namespace fp8g
