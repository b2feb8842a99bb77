// FP8 scaled GEMM on the gfx950 matrix cores, two scaling modes, each operand
// E4M3 or E5M2.
//
//   mode (a)  D[m,n] = sa[m] sb[n] sum_k A[m,k] B[n,k]
//             per-token / per-channel fp32 scales, as the DeepGEMM call on the
//             page "FP8 推理基础设施（五）：从 DeepGEMM 到 vLLM".
//   mode (b)  D[m,n] = sum_j 2^(ea[m,j]-127) 2^(eb[n,j]-127) sum_{t<32} A[m,32j+t] B[n,32j+t]
//             MXFP8: one UE8M0 scale per 32 K elements of every row, as on the
//             page "[sglang] FlashInfer v0.6.7 MXFP8 Gemm 통합", sections 1-2.
//
// Operand formats: the matrix-core instruction takes a format per operand
// (E4M3 = "fp8", E5M2 = "bf8"), so each of A and B may be either; the format
// pair is a template parameter and changes nothing else (a zero byte is +0 in
// both, so the zero-filled K tail is the same).
//
// Both operands are K-major bytes (A [M,K], B [N,K]).  The work is a dense
// contraction (2MNK flops at arithmetic intensity in the thousands), so it is
// bound by the matrix cores, not HBM.
//
// Tiling: a 256-thread workgroup (4 waves, 2x2) owns a 256x256 output tile;
// each wave owns 128x128 = 4x4 blocks of the 32x32 matrix-core tile (256 fp32
// accumulators per lane).  Problems with at most half as many 256x256 tiles as
// CUs use 128x128 tiles instead (waves of 64x64 = 2x2 blocks): four times the
// workgroups, each moving twice the operand bytes per flop, which the idle
// CUs more than pay for.  In mode (a), problems whose 128x128 tiles would
// still fill at most half of the CUs (2048 x 1024: 128 tiles for 256 CUs) use
// 64x128 tiles (waves of 32x64 = 1x2 blocks), unless splitting the 128x128
// tiles over K is predicted faster.  In both modes, 256x128 tiles (waves of
// 128x64 = 4x2 blocks) replace 256x256 ones where those leave a last round
// of workgroups partly empty.
//
// K is walked in 64-byte steps, one V_MFMA_SCALE_F32_32X32X64_F8F6F4 per block
// per step; mode (a) passes the neutral scale code 127 (2^0) and applies sa,
// sb in the epilogue, mode (b) passes the operands' block scales.
//
// Persistent workgroups: one per CU, each walking a list of tiles.  Its
// stages (128 bytes of K, two steps) form one stream across its tiles, so the
// loads of the next tile are in flight while the current tile's epilogue runs.
//
// Operand staging: direct global -> LDS loads (buffer_load_dwordx4 ... lds;
// lane L of a wave writes LDS bytes [M0 + 16L, M0 + 16L + 16)).  A stage moves
// 128 bytes of every row: whole 128-byte lines, which the memory system serves
// at twice the rate of 64-byte pieces of rows (measured: 66 vs 33 bytes per
// clock per CU from L2 for rows 8 KB apart).  Each operand of a stage (256 rows
// x 128 B = 32 KB) is one "item" in a ring of NSLOT LDS slots (5 x 32 KB =
// 160 KB; mode (b) with whole scale dwords uses 4 slots, beside its scales).  One item
// is loaded per K step, its 8 loads spread over that step's matrix-core
// instructions, NSLOT-1 items ahead.  The compiler cannot track these loads
// (it would wait for all of them before every LDS read), so they are issued
// from inline assembly and the kernel waits for them itself; vector-memory
// loads complete in order, so a count of outstanding loads identifies the
// item.  Loads past the end of a panel (rows past M or N, bytes past K) read 0
// (buffer range check on voffset + soffset).
//
// LDS layout of a slot: 256 rows of 128 bytes (eight 16-byte chunks); logical
// chunk c of row r sits in slot c ^ ((r >> 1) & 7).  A 128-bit read serves 16
// lanes per LDS cycle (64 banks, 256 bytes): 16 consecutive rows at one logical
// chunk fall in 16 distinct 16-byte bank groups.  A load instruction fills 8
// rows: lane L takes slot L % 8 of row L / 8 and fetches the chunk stored there.
//
// The matrix core reads a lane's 32 operand bytes as two 16-byte halves:
// bytes 0-15 belong to K block 0 of the 64-wide step and bytes 16-31 to block
// 1; lanes 32-63 hold the upper 16 of each block.  So for step h of a stage a
// lane takes chunks 4h + lhi and 4h + 2 + lhi of its row, and the scale of
// block 0 / 1 of the step comes from lanes 0-31 / 32-63.
//
// Operand roles: the matrix-core "A" operand is fed from B's rows (n) and the
// "B" operand from A's rows (m), so each lane's accumulator block holds one m
// and four consecutive n per group of registers: 8-byte (bf16) or 16-byte
// (fp32) row-contiguous stores in the epilogue.
//
// Tile order: workgroup b runs on XCD b % 8; each XCD gets a contiguous run of
// tiles, walked in groups of GROUP_M tile-rows, so the tiles an XCD runs
// together share A and B panels in its own L2.
//
// Matrix-core results must never be consumed under a lane-divergent branch:
// the compiler may then move the instruction into that branch, where it runs
// with a partial EXEC mask yet still writes every lane.  Here they feed only
// the accumulators and the epilogue, under uniform control flow.

#pragma once

#include <type_traits>

#include "device_common.h"
#include "epilogue.h"

namespace fp8g {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef unsigned int v4u __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));

constexpr int BK = 128;        // bytes of K per stage (two matrix-core steps)
constexpr int KSTEP = 64;      // bytes of K per matrix-core step
constexpr int NTHREADS = 256;
constexpr int NUM_XCD = 8;
constexpr int GROUP_M = 8;

// Tile geometry: a BM x BN output tile per workgroup (BM rows of A, BN rows of
// B), 4 waves in 2x2, each wave WTM x WTN = NBM x NBN blocks of 32x32.  TILE
// names the shape: 256 (256x256), 128 (128x128, for problems with few
// tiles), TILE_64x128 (mode (a), for problems whose 128x128 tiles would leave
// at least half of the CUs idle) or TILE_256x128 (for problems whose 256x256
// tiles leave a last round partly empty).
constexpr int TILE_64x128 = 64128, TILE_256x128 = 256128;
template <int TILE>
struct Geo {
    static constexpr int BM = TILE > 1000 ? TILE / 1000 : TILE, BN = TILE > 1000 ? TILE % 1000 : TILE;
    static constexpr int WTM = BM / 2, WTN = BN / 2;           // wave tile
    static constexpr int NBM = WTM / 32, NBN = WTN / 32;       // blocks per wave tile: 4x4, 2x2, 1x2 or 4x2
    // one operand of one stage (an "item"), and its loads per wave (1 KB per
    // wave instruction, 4 waves)
    static constexpr int A_BYTES = BM * BK, B_BYTES = BN * BK;
    static constexpr int LA = A_BYTES / 1024 / 4, LB = B_BYTES / 1024 / 4;
};

// Ring geometry per kernel variant.  256-row items: 5 slots of 32 KB fill the
// LDS, so mode (b) with whole scale dwords (scale groups beside the ring)
// fits only 4 slots.  128-row items: mode (a) 8 slots of 16 KB, loads 7 items
// ahead (against 5 slots: 7-10% faster at 2048x1024x4096 and the other
// 128-tile shapes measured; 6 or 7 slots: the same within 2%); mode (b) 5
// (8 slots ran 5% slower there).  64x128 tiles (A items of 8 KB in slots of
// 16 KB): 6 slots, loads 5 items ahead (at 2048x1024x4096: 13.0 us, against
// 16.8 us with 5 slots, 15.0 us with 8 and 16.4 us with 10 slots of 24 KB
// pairs).  256x128 tiles: 3 pairs of a 32 KB A slot and a 16 KB B slot (6
// slots, loads 5 items ahead), in mode (b) and 12 KB of scale groups; the
// epilogue borrows the B slot that is free then.
template <bool MX, bool KTAIL, int TILE>
struct Ring {
    using G = Geo<TILE>;
    static constexpr bool SCALES = MX && !KTAIL;
    static constexpr int NSLOT =
        TILE == 256 ? (SCALES ? 4 : 5) : (TILE == TILE_64x128 || TILE == TILE_256x128) ? 6 : (MX ? 5 : 8);
    // slot k holds items of index k modulo NSLOT; with slots of two sizes
    // (COMPACT: even slots A items, odd ones B items, NSLOT even) each pair is
    // A_BYTES + B_BYTES, otherwise every slot has the larger item's size
    static constexpr bool COMPACT = TILE == TILE_256x128;
    static_assert(!COMPACT || NSLOT % 2 == 0, "ring");
    static constexpr int SLOT = G::B_BYTES > G::A_BYTES ? G::B_BYTES : G::A_BYTES;
    static constexpr int LDS = COMPACT ? NSLOT / 2 * (G::A_BYTES + G::B_BYTES) : NSLOT * SLOT;
    static constexpr int LA = G::LA, LB = G::LB;   // load instructions per item and wave, A and B
    // 4 slots hold two stages: stage g+2 can be loaded only once stage g's
    // slots are free (its step 1), so both its items are issued in that step
    // (none in step 0) to give them the longest lead.  5 or more slots: one
    // item per step, NSLOT-1 items ahead.
    static constexpr bool PAIRED = NSLOT == 4;
    // mode (b) scale groups after the ring: 2 buffers of BM rows of A and BN
    // rows of B x 16 bytes (the scales of SC_GROUP stages)
    static constexpr int SC_GROUP = 4;
    static constexpr int SC_AREA = LDS;
    static constexpr int SC_A = G::BM * 16, SC_B = G::BN * 16;
    static constexpr int SC_BYTES = SCALES ? 2 * (SC_A + SC_B) : 0;
    // epilogue staging (16 KB; in mode (a) also the tile's sa, sb at
    // +16 KB): with 5 slots of 32 KB, or the 16 KB B slots of 256x128 tiles,
    // the slot that is free during the epilogue is borrowed; otherwise
    // (paired, or 16 KB slots) a region of its own.  Mode (a) on 256x128
    // tiles keeps the tile's sa, sb in 2 KB of their own after the ring
    // (TS_SEPARATE, at TS_AREA), since the borrowed B slot holds only the
    // 16 KB of staging.
    static constexpr bool OWN_STAGE = PAIRED || (TILE != 256 && TILE != TILE_256x128);
    static constexpr int STAGE_AREA = LDS + SC_BYTES;
    static constexpr bool TS_SEPARATE = !MX && TILE == TILE_256x128;
    static constexpr int TS_AREA = STAGE_AREA;
    static constexpr int LDS_TOTAL = STAGE_AREA + (OWN_STAGE ? (MX ? 16 : 18) * 1024 : 0) + (TS_SEPARATE ? 2048 : 0);
};
static_assert(Ring<false, false, 256>::LDS_TOTAL <= 160 * 1024 && Ring<true, false, 256>::LDS_TOTAL <= 160 * 1024 &&
                  Ring<true, false, 128>::LDS_TOTAL <= 160 * 1024 && Ring<false, false, 128>::LDS_TOTAL <= 160 * 1024 &&
                  Ring<false, false, TILE_64x128>::LDS_TOTAL <= 160 * 1024 &&
                  Ring<true, false, TILE_256x128>::LDS_TOTAL <= 160 * 1024 &&
                  Ring<false, false, TILE_256x128>::LDS_TOTAL <= 160 * 1024,
              "LDS");

// The share of n items that slot k of s slots takes: one per slot while they
// last when s >= n, else an even split.
__host__ __device__ constexpr int share_lo(int k, int n, int s) { return s >= n ? (k < n ? k : n) : k * n / s; }
__host__ __device__ constexpr int share_hi(int k, int n, int s) { return s >= n ? (k < n ? k + 1 : n) : (k + 1) * n / s; }

constexpr int BUF_DW3 = 0x00020000;   // raw (untyped) buffer descriptor word 3, 32-bit data format
// Cache policy of the staged epilogues' D stores (each store instruction
// writes 8 rows x 128 contiguous bytes): non-temporal.  Every workgroup writes
// its finished tile at about the same time, 4 MB per XCD for a round of
// 256x256 bf16 tiles.  Measured at 8192x22016x8192: 1.4-2% faster in mode
// (a), 3% in mode (b); at N = 22008 (rows not whole lines) still 0.8%
// (write-through, sc0 sc1: no gain).  The L2 miss traffic of the operand loads
// is unchanged (FETCH_SIZE), so the gain is in how the writes drain, not in the
// operands' reuse.  The epilogue from registers (16 bytes or less in each of
// 32 rows per store) keeps the default policy: non-temporal, it ran 30-50%
// slower.
constexpr int ST_NT = 2;

// ---------------------------------------------------------------- helpers

__device__ __forceinline__ __amdgpu_buffer_rsrc_t panel(const void* p, uint32_t bytes) {
    // buffer over `bytes` bytes at p: loads at or past the end return 0
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, (int)bytes, BUF_DW3);
}

// 16 bytes per lane from buffer rs at (voff + soff) into LDS at lds_addr + 16 * lane.
__device__ __forceinline__ void dma16(uint32_t lds_addr, uint32_t voff, __amdgpu_buffer_rsrc_t rs, uint32_t soff) {
    asm volatile("s_mov_b32 m0, %0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                 :
                 : "s"(lds_addr), "v"(voff), "s"(rs), "s"(soff)
                 : "memory", "m0");
}
// 4 bytes per lane into LDS at lds_addr + 4 * lane.
__device__ __forceinline__ void dma4(uint32_t lds_addr, uint32_t voff, __amdgpu_buffer_rsrc_t rs, uint32_t soff) {
    asm volatile("s_mov_b32 m0, %0\n\tbuffer_load_dword %1, %2, %3 offen lds"
                 :
                 : "s"(lds_addr), "v"(voff), "s"(rs), "s"(soff)
                 : "memory", "m0");
}
template <int N>
__device__ __forceinline__ void wait_vmcnt() {
    asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory");
}

__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __builtin_amdgcn_readfirstlane(v); }

// The lane index, computed afresh (v_mbcnt) inside an opaque statement.  Code
// that runs once per tile (epilogues, the tile's scale loads) derives its
// lane-dependent values from this rather than from the kernel's own lane index:
// the compiler then cannot hoist them to the kernel start, where they would
// stay live through the main loop and be spilled.  Each spill reload is a
// scratch load, and the compiler waits for it with a count that does not know
// about the operand loads issued from inline assembly, so it waited for all of
// them too (measured: two such waits per tile).
__device__ __forceinline__ int fresh_lane() {
    int l;
    asm volatile("v_mbcnt_lo_u32_b32 %0, -1, 0\n\tv_mbcnt_hi_u32_b32 %0, -1, %0" : "=v"(l));
    return l;
}

struct TileCoord {
    int tm, tn;
};

// Tile id -> tile coordinates: groups of GROUP_M tile-rows, columns inside a group.
__device__ __forceinline__ TileCoord tile_coord(int t, int tiles_m, int tiles_n) {
    const int per_group = GROUP_M * tiles_n;
    const int g = t / per_group;
    const int first_m = g * GROUP_M;
    const int gm = min(GROUP_M, tiles_m - first_m);
    const int in = t - g * per_group;
    TileCoord c;
    c.tm = first_m + in % gm;
    c.tn = in / gm;
    return c;
}

// ---------------------------------------------------------------- kernel

// What a fused product (EPI > 0) and the experts' products (MOE) take beside the operands.
constexpr int EPI_NONE = 0, EPI_LINEAR = 1, EPI_GATED = 2, EPI_PARTIAL = 3;
struct TileExtra {
    const float* bias;          // [B's rows], or NULL
    const void* residual;       // as D, or NULL
    Act act;
    // MOE: tile rows found on the device (see moe_plan): plan[0] their number,
    // then 4 words each: expert, first slot, slots; and with gathered A the byte
    // offset of every row of a tile row, BM each (OOB_OFF: none).
    const int32_t* plan;
    const uint32_t* row_at;
    uint32_t a_bytes;           // of all of A, where its rows are gathered
    // EPI_PARTIAL: K ranges, and the partial sums' row pitch (elements) and size (rows)
    int32_t ranges, pitch, part_rows;
};

// Words that no kernel of the launch writes, through the scalar cache.
typedef const __attribute__((address_space(4))) int32_t* const_words;
__device__ __forceinline__ const_words const_at(const void* p) { return (const_words)(uintptr_t)p; }

// FA, FB: format code of A and of B (0 = E4M3, 1 = E5M2, as the instruction's
// format fields).  SPLIT (mode (a), K a multiple of 128): the tiles past
// tiles_whole (the last, at most half-full round of tiles) are split over K
// into `split` equal ranges of stages, one work item each; see the split
// reduction below.  ws: the items' fp32 partial tiles, cnt: one arrival
// counter per split tile (zero between launches).
// EPI: nothing behind the product, bias / activation / residual (EPI_LINEAR), or
// the gated pair (EPI_GATED: B has 2 N rows, and a tile takes BN / 2 output
// columns, so that a wave's first blocks of B's rows hold the gate and its last
// ones the up projection of the same columns, which thus meet in one lane).
// EPI_PARTIAL: K in ex.ranges ranges, one work item each and at most one item a
// workgroup; D takes their unscaled sums, one after the other, in whole tiles.
// MOE: B, its scales and the bias by expert, tile rows from a plan on the device.
template <bool MX, bool OUT_F32, bool KTAIL, int FA, int FB, int TILE, bool SPLIT, int EPI, bool MOE>
__device__ __forceinline__ void gemm_tiles(
    int M, int N, int K, const uint8_t* __restrict__ A, const uint8_t* __restrict__ B,
    const float* __restrict__ sa, const float* __restrict__ sb, const uint8_t* __restrict__ ea,
    const uint8_t* __restrict__ eb, void* __restrict__ Dv, int tiles_whole, int split, float* __restrict__ ws,
    int* __restrict__ cnt, const TileExtra& ex) {
    static_assert(!SPLIT || (!MX && !KTAIL && TILE == 128), "K splits: mode (a), whole stages, 128x128 tiles");
    static_assert(!SPLIT || EPI == EPI_NONE, "no K splits of fused products");
    constexpr bool GATED = EPI == EPI_GATED, PARTIAL = EPI == EPI_PARTIAL;
    // fused products get scale rows of whole dwords (padded where K has a tail)
    constexpr bool PADDED = MX && KTAIL && EPI != EPI_NONE;
    using R = Ring<MX, KTAIL && !PADDED, TILE>;
    static_assert(!PARTIAL || (OUT_F32 && R::OWN_STAGE), "partial sums: fp32, staging of their own");
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    using GEO = Geo<TILE>;
    constexpr int BM = GEO::BM, BN = GEO::BN, WTM = GEO::WTM, WTN = GEO::WTN, NBM = GEO::NBM, NBN = GEO::NBN;
    constexpr int NBX = NBM > NBN ? NBM : NBN;
    constexpr int BNO = GATED ? BN / 2 : BN;              // output columns of a tile
    constexpr int NBO = GATED ? NBN / 2 : NBN;            // blocks of them in a wave tile

    constexpr bool RES = !MOE;                            // experts' products have no residual

    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);   // uniform: kept in scalar registers
    const int wm = wave & 1, wn = wave >> 1;
    const int l32 = lane & 31, lhi = lane >> 5;

    const int tiles_m = MOE ? const_at(ex.plan)[0] : (M + BM - 1) / BM, tiles_n = (N + BNO - 1) / BNO;
    const int tiles = tiles_m * tiles_n, total = PARTIAL ? tiles * ex.ranges : tiles;
    const int nk = (K + BK - 1) / BK;            // stages per tile
    const int nblk = PADDED ? 4 * nk : K / 32;   // MX scale bytes per row

    // ---- this workgroup's work items: XCD x = b % 8 owns a contiguous run of
    // tiles; its W_x workgroups take every W_x-th tile of the run.  SPLIT: only
    // the first tiles_whole tiles are walked so; the split items of the
    // remaining tiles (tile tiles_whole + u, K range s of `split`, item u *
    // split + s) are distributed over the XCDs the same way, at most one per
    // workgroup, after its whole tiles.
    const int G = gridDim.x, b = blockIdx.x;
    const int xcd = b % NUM_XCD, slot = b / NUM_XCD;
    const int wx = (G - xcd + NUM_XCD - 1) / NUM_XCD;                 // workgroups on this XCD
    const int n_whole = SPLIT ? tiles_whole : total;
    const int q = n_whole / NUM_XCD, r = n_whole % NUM_XCD;
    const int run0 = xcd * q + min(xcd, r), runn = q + (xcd < r ? 1 : 0);
    const int my_whole = (slot < runn) ? (runn - slot + wx - 1) / wx : 0;
    int my_split = -1;                                                 // this workgroup's split item, if any
    if constexpr (SPLIT) {
        const int ns = (total - tiles_whole) * split;
        const int q2 = ns / NUM_XCD, r2 = ns % NUM_XCD;
        if (slot < q2 + (xcd < r2 ? 1 : 0)) my_split = xcd * q2 + min(xcd, r2) + slot;
    }
    const int my_tiles = my_whole + (my_split >= 0 ? 1 : 0);          // work items
    const int nks = SPLIT ? nk / split : nk;                           // stages of a split item
    // item t of EPI_PARTIAL: tile t % tiles, K range t / tiles; in mode (b) a range
    // starts at a whole scale group
    auto range_start = [&](int r) __attribute__((always_inline)) {
        const int at = (int)((int64_t)nk * r / ex.ranges);
        return MX && r < ex.ranges ? at & ~3 : at;
    };
    // stages in this workgroup's stream
    const int NS = PARTIAL ? (my_whole ? range_start((run0 + slot) / tiles + 1) - range_start((run0 + slot) / tiles) : 0)
                           : my_whole * nk + (my_split >= 0 ? nks : 0);
    // item j: its tile, first stage (kb) and stages (ns)
    struct Item {
        TileCoord tc;
        int kb, ns;
    };
    auto item_of = [&](int j) __attribute__((always_inline)) -> Item {
        Item it;
        if constexpr (PARTIAL) {
            const int t = run0 + slot + j * wx, r = t / tiles;
            it.tc = tile_coord(t - r * tiles, tiles_m, tiles_n);
            it.kb = range_start(r);
            it.ns = range_start(r + 1) - it.kb;
        } else if (!SPLIT || j < my_whole) {
            it.tc = tile_coord(run0 + slot + j * wx, tiles_m, tiles_n);
            it.kb = 0;
            it.ns = nk;
        } else {
            it.tc = tile_coord(tiles_whole + my_split / split, tiles_m, tiles_n);
            it.kb = (my_split % split) * nks;
            it.ns = nks;
        }
        return it;
    };
    auto tile_of = [&](int j) __attribute__((always_inline)) { return item_of(j).tc; };
    // a tile's rows of A and D and, with MOE, its expert; its first output column
    struct Place {
        int m0, rows, expert, n0;
    };
    auto place_of = [&](TileCoord tc) __attribute__((always_inline)) -> Place {
        Place p;
        if constexpr (MOE) {
            const const_words e = const_at(ex.plan) + 4 + 4 * tc.tm;
            p.expert = e[0], p.m0 = e[1], p.rows = e[2];
        } else {
            p.expert = 0, p.m0 = tc.tm * BM, p.rows = min(BM, M - p.m0);
        }
        p.n0 = tc.tn * BNO;
        return p;
    };
    // B's row block rb (32 rows) of a tile, gated: 32-column block gate_col(rb) of
    // the tile's output columns, of the up projection where gate_up(rb)
    auto gate_col = [](int rb) constexpr { return rb / NBN * NBO + rb % NBO; };
    auto gate_up = [](int rb) constexpr { return rb % NBN >= NBO; };
    const int64_t b_rows = GATED ? 2 * (int64_t)N : N;     // B's rows of one product

    const uint32_t lds0 = (uint32_t)(uintptr_t)smem;   // LDS byte address of the stage buffers

    // ---- loads.  Item i of the stream is operand i & 1 (A, B) of stream stage
    // i >> 1; it goes to LDS slot i % NSLOT.  A cursor (tile, stage, operand)
    // walks the items; descriptors change once per tile.  Past the end of the
    // stream the last stage is loaded again (never read), so every K step
    // issues the same number of loads.
    constexpr int NSLOT = R::NSLOT, SLOT = R::SLOT, LA = R::LA, LB = R::LB;
    static_assert(!R::PAIRED || LA == LB, "paired ring: square tiles");
    // loads of n consecutive items that start with an A item
    auto loads_of = [](int n) constexpr { return (n + 1) / 2 * LA + n / 2 * LB; };
    // LDS byte offset of ring slot k
    auto slot_off = [&](int k) __attribute__((always_inline)) -> uint32_t {
        if constexpr (!R::COMPACT) return (uint32_t)(k * SLOT);
        else return (uint32_t)((k >> 1) * (GEO::A_BYTES + GEO::B_BYTES) + (k & 1) * GEO::A_BYTES);
    };
    // lane L of wave w, instruction p fills row 32p + 8w + L/8, slot L%8, which
    // holds logical chunk (L%8) ^ ((row >> 1) & 7) = (L%8) ^ ((4w + L/16) & 7)
    const uint32_t dma_chunk = (uint32_t)((lane & 7) ^ ((4 * (wave & 1) + (lane >> 4)) & 7));
    const uint32_t dma_voff = (uint32_t)(8 * wave + (lane >> 3)) * (uint32_t)K + dma_chunk * 16u;
    constexpr uint32_t OOB_OFF = 0x80000000u;   // past any panel (panels are < 2^31 bytes)
    int ij = 0, is = 0, iop = 0, ii = 0, islot = 0;   // cursor: work item, stage in it, operand, load item, its slot
    int ikb = 0, ins = nk;                            // the cursor work item's first stage and stages
    __amdgpu_buffer_rsrc_t rsA, rsB, rsU;             // rsU: the up projection's rows
    uint32_t a_voff[MOE ? LA : 1];                    // gathered A: this lane's row of each load
    const bool gather = MOE && ex.row_at != nullptr;
    auto cursor_tile = [&]() __attribute__((always_inline)) {
        const Item it = item_of(min(ij, my_tiles - 1));
        const TileCoord tc = it.tc;
        ikb = it.kb;
        ins = it.ns;
        const Place p = place_of(tc);
        const uint32_t rows_a = (uint32_t)p.rows, rows_b = (uint32_t)min(BNO, N - p.n0);
        const uint8_t* Be = MOE ? B + (int64_t)p.expert * b_rows * K : B;
        rsA = panel(A + (int64_t)p.m0 * K, rows_a * (uint32_t)K);
        rsB = panel(Be + (int64_t)p.n0 * K, rows_b * (uint32_t)K);
        if constexpr (GATED) rsU = panel(Be + (int64_t)(N + p.n0) * K, rows_b * (uint32_t)K);
        if constexpr (MOE) {
            // load q of wave w takes the rows 32 q + 8 w + lane / 8.  One load for all of
            // them, handed to their lanes by permutations, waits once for the operand loads
            // in flight; scalar loads waited longer, for each q's (65536 rows of 128 experts
            // x 2048 x 4096: 588 us, with scalar loads 636 us).
            if (gather) {
                rsA = panel(A, ex.a_bytes);
                const int at = 32 * min(lane >> 3, LA - 1) + 8 * wave + (lane & 7);
                const int rows = (int)ex.row_at[(int64_t)tc.tm * BM + at];
#pragma unroll
                for (int q = 0; q < LA; ++q)
                    a_voff[q] = (uint32_t)__builtin_amdgcn_ds_bpermute(4 * (8 * q + (lane >> 3)), rows) + dma_chunk * 16u;
            } else {
#pragma unroll
                for (int q = 0; q < LA; ++q) a_voff[q] = dma_voff + (uint32_t)(32 * q) * (uint32_t)K;
            }
        }
    };
    // load q (0..LA-1 or 0..LB-1) of the cursor's item
    auto dma_item = [&](int q) __attribute__((always_inline)) {
        const int s_ld = (ii < 2 * NS) ? is : ins - 1;   // past the end: reload the last stage
        const uint32_t sbuf = lds0 + slot_off(islot);
        const uint32_t k0 = (uint32_t)((ikb + s_ld) * BK);
        uint32_t voff = dma_voff;
        if constexpr (MOE) voff = iop ? dma_voff : a_voff[q < LA ? q : 0];
        if constexpr (KTAIL) {
            // bytes past K (the next row's, or past the panel) must read as 0
            if (k0 + dma_chunk * 16u >= (uint32_t)K) voff = OOB_OFF;
        }
        uint32_t row_a = (uint32_t)(32 * q), row_b = (uint32_t)(32 * q);
        if constexpr (MOE) row_a = 0;
        if constexpr (GATED) row_b = (uint32_t)(32 * gate_col(q));
        const uint32_t so = uniform(k0 + (iop ? row_b : row_a) * (uint32_t)K);
        const __amdgpu_buffer_rsrc_t rsOp = iop ? (GATED && gate_up(q) ? rsU : rsB) : rsA;
        dma16(uniform(sbuf + (uint32_t)((4 * q + wave) * 1024)), voff, rsOp, so);
    };

    // ---- mode (b) scale groups (whole scale dwords, K % 128 == 0).  Group gi
    // of a tile covers its stages 4gi .. 4gi+3: bytes 16gi .. 16gi+15 of every
    // scale row.  Stream group number u (tile j: u = j * ngt + gi) goes to
    // buffer u & 1 at SC_AREA + (u & 1) (SC_A + SC_B), A's rows first, then
    // B's (sc_area): row r in the 16 bytes at 16 r, the dword of group stage t at position
    // (t + (r >> 3)) & 3 (rotated so that the 32 rows of one scale read fall in
    // distinct banks).  Load p of an operand fills rows 16p .. 16p+15, lane L
    // row 16p + L/4 at position L % 4: 16 bytes of a row in one or two lines,
    // where loading each stage's dword alone touches a line per row per stage.
    // Wave w issues loads p = w, w+4, ... of both operands: SC_LA of A, then
    // SC_LB of B.
    constexpr int SC_LA = R::SCALES ? BM / 16 / 4 : 0, SC_LB = R::SCALES ? BN / 16 / 4 : 0;
    constexpr int SC_LOADS = SC_LA + SC_LB;   // per wave and group: 8, 4 or 6
    // LDS byte offset of buffer ub's scale rows of operand o
    auto sc_area = [](int ub, int o) constexpr -> int {
        if constexpr (R::SC_A == R::SC_B) return R::SC_AREA + 2 * ub * R::SC_A + o * R::SC_A;
        else return R::SC_AREA + ub * (R::SC_A + R::SC_B) + o * R::SC_A;
    };
    const int ngt = (nk + R::SC_GROUP - 1) / R::SC_GROUP;            // groups per tile
    const uint32_t sc_voff = (uint32_t)(16 * wave + (lane >> 2)) * (uint32_t)nblk +
                             4u * (((uint32_t)(lane & 3) - (uint32_t)(2 * wave + (lane >> 5))) & 3u);
    // gated: a load's 16 rows of B lie in one block of 32, whose place is uniform
    const uint32_t sc_voff_g = sc_voff - (uint32_t)(16 * (wave & 2)) * (uint32_t)nblk;
    __amdgpu_buffer_rsrc_t rsEA, rsEB, rsEU;   // scale panels of the tile of the group loaded last
    auto sc_tile = [&](int j) __attribute__((always_inline)) {
        const Place p = place_of(tile_of(j));
        const uint8_t* eb_e = MOE ? eb + (int64_t)p.expert * b_rows * nblk : eb;
        const uint32_t cols = (uint32_t)min(BNO, N - p.n0);
        rsEA = panel(ea + (int64_t)p.m0 * nblk, (uint32_t)p.rows * (uint32_t)nblk);
        rsEB = panel(eb_e + (int64_t)p.n0 * nblk, cols * (uint32_t)nblk);
        if constexpr (GATED) rsEU = panel(eb_e + (int64_t)(N + p.n0) * nblk, cols * (uint32_t)nblk);
    };
    // load idx of operand B's scale rows, gated
    auto sc_load_gated = [&](uint32_t dst, int idx, int gi) __attribute__((always_inline)) {
        const int rb = 2 * idx + (wave >> 1);
        dma4(uniform(dst), sc_voff_g, gate_up(rb) ? rsEU : rsEB,
             uniform((uint32_t)(16 * gi) + (uint32_t)(32 * gate_col(rb)) * (uint32_t)nblk));
    };
    // load q (0 .. SC_LOADS-1) of group gi (of the tile of rsEA, rsEB) into buffer ub
    auto sc_load = [&](int q, int gi, int ub) __attribute__((always_inline)) {
        if constexpr (R::SCALES) {
            if constexpr (PARTIAL) gi += item_of(0).kb / R::SC_GROUP;
            if constexpr (R::SC_A == R::SC_B) {
                constexpr int PER_OP = SC_LOADS / 2;
                const int o = q / PER_OP, p = wave + 4 * (q % PER_OP);
                const uint32_t dst = lds0 + (uint32_t)(R::SC_AREA + (2 * ub + o) * R::SC_A + 256 * p);
                if (GATED && o) sc_load_gated(dst, q % PER_OP, gi);
                else
                dma4(uniform(dst), sc_voff, o ? rsEB : rsEA,
                     uniform((uint32_t)(16 * gi) + (uint32_t)(64 * (q % PER_OP)) * (uint32_t)nblk));
            } else {
                const int o = q < SC_LA ? 0 : 1, idx = o ? q - SC_LA : q, p = wave + 4 * idx;
                const uint32_t dst = lds0 + (uint32_t)(sc_area(ub, o) + 256 * p);
                if (GATED && o) sc_load_gated(dst, idx, gi);
                else
                dma4(uniform(dst), sc_voff, o ? rsEB : rsEA,
                     uniform((uint32_t)(16 * gi) + (uint32_t)(64 * idx) * (uint32_t)nblk));
            }
        }
    };
    auto advance = [&]() __attribute__((always_inline)) {
        ++ii;
        islot = (islot + 1 == NSLOT) ? 0 : islot + 1;
        if (++iop == 2) {
            iop = 0;
            if (++is == ins) {
                is = 0;
                ++ij;
                cursor_tile();
            }
        }
    };

    // ---- fragment reads: step h of the stage whose items sit in LDS slots
    // sa_off (A) and sb_off (B); this lane's rows, chunks 4h + lhi and 4h + 2 + lhi
    const uint32_t key = (uint32_t)((l32 >> 1) & 7);
    const uint32_t frag_a = (uint32_t)((wm * WTM + l32) * BK);
    const uint32_t frag_b = (uint32_t)((wn * WTN + l32) * BK);
    const uint32_t c0 = ((uint32_t)lhi ^ key) << 4, c1 = ((uint32_t)(2 + lhi) ^ key) << 4;
    auto frag = [&](uint32_t slot_off, uint32_t row_off, int h, int i) __attribute__((always_inline)) -> v8i {
        const uint8_t* p = smem + slot_off + row_off + i * 32 * BK;
        const v4u x0 = *reinterpret_cast<const v4u*>(p + (c0 ^ (uint32_t)(64 * h)));
        const v4u x1 = *reinterpret_cast<const v4u*>(p + (c1 ^ (uint32_t)(64 * h)));
        return (v8i){(int)x0.x, (int)x0.y, (int)x0.z, (int)x0.w, (int)x1.x, (int)x1.y, (int)x1.z, (int)x1.w};
    };
    // slot index + k, modulo NSLOT (k < NSLOT)
    auto slot_add = [&](int slot, int k) __attribute__((always_inline)) -> int {
        return (slot + k >= NSLOT) ? slot + k - NSLOT : slot + k;
    };

    // ---- mode (b) scales for step h of stage s of stream tile j: per lane and
    // row block, the scale byte of this lane half's block in byte 0 (the matrix
    // core reads byte 0).  With whole scale dwords: the stage's dword (blocks
    // 4s .. 4s+3) from the LDS scale group.  Otherwise (rows of nblk bytes, not
    // a multiple of 4): unconditional byte loads from global, 2^0 past the row
    // end; rows past M / N read 0 (their data is zero too).  j < my_tiles.
    auto read_scales = [&](int j, int s, int h, uint32_t* xa, uint32_t* xb) __attribute__((always_inline)) {
        if constexpr (MX) {
            if constexpr (R::SCALES) {
                // the stage's dword holds the scales of its 4 blocks; shifted by
                // this lane half, byte 2h is step h's block (selected in the
                // matrix-core instruction), so one read serves both steps.  The
                // lane-dependent parts come from a fresh lane index: kept live
                // from the kernel start they were spilled.
                const int ln = fresh_lane();
                const int l32s = ln & 31;
                const uint32_t sh = (uint32_t)(8 * (ln >> 5));
                const int ub = (j * ngt + s / R::SC_GROUP) & 1;
                const uint8_t* sca;
                const uint8_t* scb;
                if constexpr (R::SC_A == R::SC_B) {
                    sca = smem + R::SC_AREA + 2 * ub * R::SC_A;
                    scb = sca + R::SC_A;
                } else {
                    sca = smem + sc_area(ub, 0);
                    scb = smem + sc_area(ub, 1);
                }
                // row wm*WTM + 32i + l32: (row >> 3) & 3 == (l32 >> 3) & 3
                const uint32_t pos = (((uint32_t)(s & 3) + (uint32_t)(l32s >> 3)) & 3u) * 4u;
#pragma unroll
                for (int i = 0; i < NBX; ++i) {
                    if (i < NBM)
                        xa[i] = *reinterpret_cast<const uint32_t*>(sca + (wm * WTM + i * 32 + l32s) * 16 + pos) >> sh;
                    if (i < NBN)
                        xb[i] = *reinterpret_cast<const uint32_t*>(scb + (wn * WTN + i * 32 + l32s) * 16 + pos) >> sh;
                }
            } else {
                const Place p = place_of(tile_of(j));
                static_assert(EPI == EPI_NONE, "fused products have scale groups");
                const __amdgpu_buffer_rsrc_t pa = panel(ea + (int64_t)p.m0 * nblk, (uint32_t)p.rows * (uint32_t)nblk);
                const __amdgpu_buffer_rsrc_t pb = panel(eb + (int64_t)p.n0 * nblk, (uint32_t)min(BN, N - p.n0) * (uint32_t)nblk);
                const int kb = 4 * s + 2 * h + lhi;   // this lane half's block
                const bool in = kb < nblk;
                const uint32_t kc = (uint32_t)min(kb, nblk - 1);
#pragma unroll
                for (int i = 0; i < NBX; ++i) {
                    if (i < NBM) {
                        const uint32_t va = __builtin_amdgcn_raw_buffer_load_b8(
                            pa, (uint32_t)(wm * WTM + i * 32 + l32) * (uint32_t)nblk + kc, 0, 0);
                        xa[i] = in ? va : 127u;
                    }
                    if (i < NBN) {
                        const uint32_t vb = __builtin_amdgcn_raw_buffer_load_b8(
                            pb, (uint32_t)(wn * WTN + i * 32 + l32) * (uint32_t)nblk + kc, 0, 0);
                        xb[i] = in ? vb : 127u;
                    }
                }
            }
        }
    };

    // The empty asm after each step pins it where it is written: the builtin has
    // no side effects, so without it the optimizer may sink whole stages of
    // steps past later barriers, leaving the matrix core idle in between.
    // The instruction's first operand is fed from B's rows, so its format
    // field is FB and the second one's FA.
    // OPS: the byte of each scale register that holds this lane's block scale
    auto mfma = [&](v16f& c, const v8i& fbi, const v8i& faj, uint32_t sbi, uint32_t saj, auto ops_tag)
                    __attribute__((always_inline)) {
        constexpr int OPS = decltype(ops_tag)::value;
        if constexpr (MX)
            c = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fbi, faj, c, FB, FA, OPS, (int)sbi, OPS, (int)saj);
        else
            c = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fbi, faj, c, FB, FA, 0, 127, 0, 127);
        asm volatile("" : "+a"(c));
    };

    // ---- epilogue of stream tile j from registers (where no staged epilogue applies):
    // lane holds m = .. + l32 and n = .. + 8g + 4*lhi + t (t = 0..3) in
    // acc[.][.][4g+t].  Stores over the tile's rows of D: out-of-range lanes get
    // an offset past the end, which the hardware drops.  Mode (a) reads the
    // tile's sa, sb from LDS at stage_off + 16 KB / + 17 KB (loaded by
    // tile_scales_to_lds during the tile's last K step, like the staged
    // epilogue): loaded here into registers, the compiler's wait for them would
    // also wait for the next tile's operand loads in flight.
    constexpr int ESZ = OUT_F32 ? 4 : 2;
    constexpr uint32_t SC_OFF = 16384;   // the tile's sa at stage_off + 16 KB, sb at + 17 KB
    // LDS offset of the tile's sa (sb 1 KB after it) for the staging region at stage_off
    auto ts_off = [&](uint32_t stage_off) __attribute__((always_inline)) -> uint32_t {
        if constexpr (R::TS_SEPARATE) return (uint32_t)R::TS_AREA;
        else return stage_off + SC_OFF;
    };
    auto epilogue = [&](int j, v16f (&acc)[NBN][NBM], uint32_t stage_off) __attribute__((always_inline)) {
        const TileCoord tc = tile_of(j);
        const int m0 = tc.tm * BM, n0 = tc.tn * BN;
        const uint32_t rows = (uint32_t)min(BM, M - m0);
        const __amdgpu_buffer_rsrc_t rsD =
            panel(reinterpret_cast<uint8_t*>(Dv) + (int64_t)m0 * N * ESZ, rows * (uint32_t)N * ESZ);
        constexpr uint32_t OOB = 0x80000000u;   // beyond any panel (panels are < 2^31 bytes)
        const int lane_u = fresh_lane();
        const int l32 = lane_u & 31, lhi = lane_u >> 5;
        const float* lsa = reinterpret_cast<const float*>(smem + ts_off(stage_off));
        const float* lsb = reinterpret_cast<const float*>(smem + ts_off(stage_off) + 1024);
        float smv[NBM], snv[NBN][4][4];
#pragma unroll
        for (int jb = 0; jb < NBM; ++jb) {
            smv[jb] = 1.0f;
            if constexpr (!MX) smv[jb] = lsa[wm * WTM + jb * 32 + l32];   // rows past M hold 0 (and are not stored)
        }
#pragma unroll
        for (int i = 0; i < NBN; ++i)
#pragma unroll
            for (int gq = 0; gq < 4; ++gq) {
                if constexpr (!MX) {
                    // a float vector: __builtin_bit_cast of an element of an integer
                    // vector reads element 0 whatever the index (clang)
                    const v4f t4 = *reinterpret_cast<const v4f*>(lsb + wn * WTN + i * 32 + 8 * gq + 4 * lhi);
#pragma unroll
                    for (int t = 0; t < 4; ++t) snv[i][gq][t] = t4[t];
                } else {
#pragma unroll
                    for (int t = 0; t < 4; ++t) snv[i][gq][t] = 1.0f;
                }
            }
        __builtin_amdgcn_sched_barrier(0);
        const bool vec_ok = (N % 4) == 0;
#pragma unroll
        for (int jb = 0; jb < NBM; ++jb) {
            const int mr = wm * WTM + jb * 32 + l32;          // row inside the tile
            const bool mok = m0 + mr < M;
            const uint32_t rowoff = (uint32_t)mr * (uint32_t)N;
#pragma unroll
            for (int i = 0; i < NBN; ++i) {
#pragma unroll
                for (int gq = 0; gq < 4; ++gq) {
                    const int n = n0 + wn * WTN + i * 32 + 8 * gq + 4 * lhi;
                    float v[4];
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        float x = acc[i][jb][4 * gq + t];
                        if constexpr (!MX) x = x * smv[jb] * snv[i][gq][t];
                        v[t] = x;
                    }
                    if (vec_ok) {
                        // n % 4 == 0 and N % 4 == 0: the 4 values are all in or all out
                        const uint32_t off = (mok && n < N) ? (rowoff + (uint32_t)n) * ESZ : OOB;
                        if constexpr (OUT_F32) {
                            const v4u w4 = {__builtin_bit_cast(uint32_t, v[0]), __builtin_bit_cast(uint32_t, v[1]),
                                            __builtin_bit_cast(uint32_t, v[2]), __builtin_bit_cast(uint32_t, v[3])};
                            __builtin_amdgcn_raw_buffer_store_b128(w4, rsD, off, 0, 0);
                        } else {
                            typedef unsigned int v2u __attribute__((ext_vector_type(2)));
                            const v2u w2 = {bf16x2_bits(v[0], v[1]), bf16x2_bits(v[2], v[3])};
                            __builtin_amdgcn_raw_buffer_store_b64(w2, rsD, off, 0, 0);
                        }
                    } else {
#pragma unroll
                        for (int t = 0; t < 4; ++t) {
                            const uint32_t off = (mok && n + t < N) ? (rowoff + (uint32_t)(n + t)) * ESZ : OOB;
                            if constexpr (OUT_F32)
                                __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, v[t]), rsD, off, 0, 0);
                            else
                                __builtin_amdgcn_raw_buffer_store_b16((unsigned short)bf16x2_bits(v[t], 0.0f), rsD, off, 0, 0);
                        }
                    }
                }
            }
        }
    };

    // ---- bf16 epilogue through LDS (N % 8 == 0), in a free 32 KB region at
    // stage_off: the tile's sa, sb sit at stage_off + 16 KB / + 17 KB (loaded by
    // tile_scales_to_lds); each wave stages bands of 32 rows x 64 columns (4 KB,
    // one 128-byte line per row) in its own 4 KB, reads them back row-contiguous
    // and stores 16 bytes per lane, 8 rows x 128 bytes (whole lines) per
    // instruction.  A store instruction that touches 32 rows at 16 bytes each
    // runs about 8x slower.  Band layout: 32 rows of 128 bytes, logical 16-byte
    // chunk c of row r in physical chunk c ^ ((r >> 1) & 7), its 8-byte halves
    // swapped when r >= 16: the 8-byte writes of 32 rows and the 16-byte reads of
    // 2 rows per LDS cycle both hit distinct banks.
    auto tile_scales_to_lds = [&](int j, uint32_t stage_off) __attribute__((always_inline)) {
        if constexpr (!MX) {
            const Place p = place_of(tile_of(j));
            const uint32_t v = (uint32_t)(64 * wave + fresh_lane()) * 4u;   // lane L of wave w: element 64w + L
            dma4(uniform(lds0 + ts_off(stage_off) + (uint32_t)(wave * 256)), v,
                 panel(sa + p.m0, (uint32_t)p.rows * 4u), 0u);
            const float* sbe = (MOE ? sb + (int64_t)p.expert * b_rows : sb) + p.n0;
            if constexpr (GATED) {
                const int r = 64 * wave + fresh_lane(), rb = r >> 5, col = 32 * gate_col(rb) + (r & 31);
                const uint32_t off = (uint32_t)(gate_up(rb) ? N + col : col) * 4u;
                dma4(uniform(lds0 + ts_off(stage_off) + 1024u + (uint32_t)(wave * 256)),
                     r < BN && p.n0 + col < N ? off : OOB_OFF, panel(sbe, (uint32_t)(2 * N - p.n0) * 4u), 0u);
            } else {
                dma4(uniform(lds0 + ts_off(stage_off) + 1024u + (uint32_t)(wave * 256)), v,
                     panel(sbe, (uint32_t)min(BN, N - p.n0) * 4u), 0u);
            }
        }
    };
    auto epilogue_staged = [&](int j, v16f (&acc)[NBN][NBM], uint32_t stage_off) __attribute__((always_inline)) {
        const TileCoord tc = tile_of(j);
        const int m0 = tc.tm * BM, n0 = tc.tn * BN;
        const uint32_t rows = (uint32_t)min(BM, M - m0);
        const __amdgpu_buffer_rsrc_t rsD =
            panel(reinterpret_cast<uint8_t*>(Dv) + (int64_t)m0 * N * 2, rows * (uint32_t)N * 2u);
        constexpr uint32_t OOB = 0x80000000u;
        const int lane_e = fresh_lane();
        const int l32e = lane_e & 31, lhie = lane_e >> 5;
        uint8_t* st = smem + stage_off + wave * 4096;
        const float* lsa = reinterpret_cast<const float*>(smem + ts_off(stage_off));
        const float* lsb = reinterpret_cast<const float*>(smem + ts_off(stage_off) + 1024);
        const uint32_t wkey = (uint32_t)((l32e >> 1) & 7), whalf = (uint32_t)(lhie ^ (l32e >> 4));
        // rows past M need no check: the descriptor covers exactly the tile's rows
        // of D, and offsets past it are dropped
        const uint32_t rc = (uint32_t)(lane_e & 7);        // read-back: 16-byte chunk of the lane
        const int rr = lane_e >> 3;                          // read-back: row within 8
        const uint32_t rd_off = (uint32_t)(rr * 128) + ((rc ^ (uint32_t)((rr >> 1) & 3)) << 4);
#pragma unroll
        for (int ih = 0; ih < NBN / 2; ++ih) {     // 64-column part of the wave tile: blocks i = 2ih, 2ih+1
            float snv[2][4][4];
#pragma unroll
            for (int ii = 0; ii < 2; ++ii)
#pragma unroll
                for (int gq = 0; gq < 4; ++gq) {
                    if constexpr (!MX) {
                        // a float vector: __builtin_bit_cast of an element of an integer
                        // vector reads element 0 whatever the index (clang)
                        const v4f t4 = *reinterpret_cast<const v4f*>(lsb + wn * WTN + (2 * ih + ii) * 32 + 8 * gq + 4 * lhie);
#pragma unroll
                        for (int t = 0; t < 4; ++t) snv[ii][gq][t] = t4[t];
                    } else {
#pragma unroll
                        for (int t = 0; t < 4; ++t) snv[ii][gq][t] = 1.0f;
                    }
                }
#pragma unroll
            for (int jb = 0; jb < NBM; ++jb) {
                float smv = 1.0f;
                if constexpr (!MX) smv = lsa[wm * WTM + jb * 32 + l32e];
#pragma unroll
                for (int ii = 0; ii < 2; ++ii)
#pragma unroll
                    for (int gq = 0; gq < 4; ++gq) {
                        float v[4];
#pragma unroll
                        for (int t = 0; t < 4; ++t) v[t] = acc[2 * ih + ii][jb][4 * gq + t] * smv * snv[ii][gq][t];
                        typedef unsigned int v2u __attribute__((ext_vector_type(2)));
                        const v2u w2 = {bf16x2_bits(v[0], v[1]), bf16x2_bits(v[2], v[3])};
                        const uint32_t pc = (uint32_t)(4 * ii + gq) ^ wkey;
                        *reinterpret_cast<v2u*>(st + l32e * 128 + pc * 16 + whalf * 8) = w2;
                    }
                const int n = n0 + wn * WTN + 64 * ih + 8 * (int)rc;
                // branch-free select (a compare-and-select here becomes a branch)
                uint32_t keep = n < N ? 0xFFFFFFFFu : 0u;
                asm volatile("" : "+v"(keep));
                const uint32_t col_off = (uint32_t)n * 2u;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    // band row r = 8k + rr: (r >> 1) & 7 = 4k + (rr >> 1) (mod 8), so the
                    // physical chunk is rc ^ ((rr >> 1) & 3) ^ 4 (k & 1)
                    v4u d = *reinterpret_cast<const v4u*>(st + k * 1024 + (rd_off ^ (uint32_t)(64 * (k & 1))));
                    if (k >= 2) d = (v4u){d.z, d.w, d.x, d.y};   // rows 16..31: halves swapped
                    const uint32_t mr = (uint32_t)(wm * WTM + jb * 32 + 8 * k + rr);   // row inside the tile
                    const uint32_t off = mr * (uint32_t)N * 2u + col_off;
                    __builtin_amdgcn_raw_buffer_store_b128(d, rsD, (off & keep) | (OOB & ~keep), 0, ST_NT);
                }
            }
        }
    };
    // ---- fp32 epilogue through LDS (mode (a), N % 32 == 0): as the bf16 one, with bands of
    // one 32x32 block (32 rows x 128 bytes, 4 KB per wave).  Lane (l32, lhi)
    // writes the 16-byte chunks 2 gq + lhi (gq = 0..3) of band row l32, logical
    // chunk c of row r at physical chunk c ^ ((r >> 1) & 7): the writes of 16
    // lanes (16 rows, one chunk) and the reads of 16 lanes (2 rows, 8 chunks)
    // both hit 16 distinct 16-byte bank groups.  Read back row-contiguously, 8
    // lanes store one 128-byte row of the band, as whole lines.
    auto epilogue_staged_f32 = [&](int j, v16f (&acc)[NBN][NBM], uint32_t stage_off) __attribute__((always_inline)) {
        const TileCoord tc = tile_of(j);
        const int m0 = tc.tm * BM, n0 = tc.tn * BN;
        const uint32_t rows = (uint32_t)min(BM, M - m0);
        const __amdgpu_buffer_rsrc_t rsD =
            panel(reinterpret_cast<uint8_t*>(Dv) + (int64_t)m0 * N * 4, rows * (uint32_t)N * 4u);
        constexpr uint32_t OOB = 0x80000000u;
        const int lane_e = fresh_lane();
        const int l32e = lane_e & 31, lhie = lane_e >> 5;
        uint8_t* st = smem + stage_off + wave * 4096;
        const float* lsa = reinterpret_cast<const float*>(smem + ts_off(stage_off));
        const float* lsb = reinterpret_cast<const float*>(smem + ts_off(stage_off) + 1024);
        const uint32_t wkey = (uint32_t)((l32e >> 1) & 7);
        // rows past M need no check: the descriptor covers exactly the tile's rows
        // of D, and offsets past it are dropped
        const uint32_t rc = (uint32_t)(lane_e & 7);        // read-back: 16-byte chunk of the lane
        const int rr = lane_e >> 3;                          // read-back: row within 8
        const uint32_t rd_off = (uint32_t)(rr * 128) + ((rc ^ (uint32_t)((rr >> 1) & 3)) << 4);
#pragma unroll
        for (int i = 0; i < NBN; ++i) {     // 32-column block of the wave tile
            float snv[4][4];
#pragma unroll
            for (int gq = 0; gq < 4; ++gq) {
                if constexpr (!MX) {
                    const v4f t4 = *reinterpret_cast<const v4f*>(lsb + wn * WTN + i * 32 + 8 * gq + 4 * lhie);
#pragma unroll
                    for (int t = 0; t < 4; ++t) snv[gq][t] = t4[t];
                } else {
#pragma unroll
                    for (int t = 0; t < 4; ++t) snv[gq][t] = 1.0f;
                }
            }
            const int n = n0 + wn * WTN + 32 * i + 4 * (int)rc;
            // branch-free select (a compare-and-select here becomes a branch)
            uint32_t keep = n < N ? 0xFFFFFFFFu : 0u;
            asm volatile("" : "+v"(keep));
            const uint32_t col_off = (uint32_t)n * 4u;
#pragma unroll
            for (int jb = 0; jb < NBM; ++jb) {
                float smv = 1.0f;
                if constexpr (!MX) smv = lsa[wm * WTM + jb * 32 + l32e];
#pragma unroll
                for (int gq = 0; gq < 4; ++gq) {
                    v4f w4;
#pragma unroll
                    for (int t = 0; t < 4; ++t) w4[t] = acc[i][jb][4 * gq + t] * smv * snv[gq][t];
                    const uint32_t pc = (uint32_t)(2 * gq + lhie) ^ wkey;
                    *reinterpret_cast<v4f*>(st + l32e * 128 + pc * 16) = w4;
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    // band row r = 8k + rr: (r >> 1) & 7 = 4k + (rr >> 1) (mod 8), so the
                    // physical chunk is rc ^ ((rr >> 1) & 3) ^ 4 (k & 1)
                    const v4u d = *reinterpret_cast<const v4u*>(st + k * 1024 + (rd_off ^ (uint32_t)(64 * (k & 1))));
                    const uint32_t mr = (uint32_t)(wm * WTM + jb * 32 + 8 * k + rr);   // row inside the tile
                    const uint32_t off = mr * (uint32_t)N * 4u + col_off;
                    __builtin_amdgcn_raw_buffer_store_b128(d, rsD, (off & keep) | (OOB & ~keep), 0, ST_NT);
                }
                // one block at a time: interleaved across blocks, the schedule kept
                // too many values live and spilled
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    };
    // ---- fused epilogues (EPI > 0).  v = act(z) or act(z_gate) z_up of block i of
    // the wave's output columns, row block jb, group gq: the four columns n ..
    // n + 3 of this lane's row.  bnv: their bias (the up projection's last).
    // The scales come from LDS each time, where every row group needs the same
    // few; the bias from global memory once per tile, waiting for the operand
    // loads in flight before it.
    auto fused_bias = [&](const Place& p, int i, v4f (&b)[GATED ? 2 : 1][4], int lhie) __attribute__((always_inline)) {
#pragma unroll
        for (int h = 0; h < (GATED ? 2 : 1); ++h) {
            const __amdgpu_buffer_rsrc_t rs =
                panel(ex.bias + (MOE ? (int64_t)p.expert * b_rows : 0) + (int64_t)h * N, (uint32_t)N * 4u);
#pragma unroll
            for (int gq = 0; gq < 4; ++gq) {
                const uint32_t n = (uint32_t)(p.n0 + 32 * (wn * NBO + i) + 8 * gq + 4 * lhie);
                if (TILE == 256 || N % 4 == 0) {
                    b[h][gq] = __builtin_bit_cast(v4f, __builtin_amdgcn_raw_buffer_load_b128(rs, 4u * n, 0, 0));
                } else {
                    // the last four may end inside
#pragma unroll
                    for (int t = 0; t < 4; ++t)
                        b[h][gq][t] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rs, 4u * (n + t), 0, 0));
                }
            }
        }
    };
    auto fused_values = [&](v16f (&acc)[NBN][NBM], int i, int jb, int gq, float smv, const float* lsb, int lhie,
                            const v4f (&b)[GATED ? 2 : 1][4], bool with_bias, bool with_act, float* v)
                            __attribute__((always_inline)) {
        float z[GATED ? 2 : 1][4];
#pragma unroll
        for (int h = 0; h < (GATED ? 2 : 1); ++h) {
            v4f sn = {1.0f, 1.0f, 1.0f, 1.0f};
            if constexpr (!MX)
                sn = *reinterpret_cast<const v4f*>(lsb + wn * WTN + (h * NBO + i) * 32 + 8 * gq + 4 * lhie);
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                float x = acc[h * NBO + i][jb][4 * gq + t];
                if constexpr (!MX) x = x * smv * sn[t];
                if (with_bias) x += b[h][gq][t];
                z[h][t] = x;
            }
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            v[t] = with_act ? activate(z[0][t], ex.act.c1, ex.act.c3) : z[0][t];
            if constexpr (GATED) v[t] *= z[1][t];
        }
    };
    // f(with_bias, with_act) with both as compile-time constants
    auto fused_kind = [&](auto f) __attribute__((always_inline)) {
        using Yes = std::integral_constant<bool, true>;
        using No = std::integral_constant<bool, false>;
        if (ex.act.on) {
            if (ex.bias) f(Yes{}, Yes{});
            else f(No{}, Yes{});
        } else {
            if (ex.bias) f(Yes{}, No{});
            else f(No{}, No{});
        }
    };
    // bf16 through LDS, as epilogue_staged: bands of 32 rows x CB blocks of 32
    // columns (CB = 2, or 1 where the wave has one block of output columns), stored
    // row-contiguously.  The residual takes the same way back: read
    // row-contiguously, put into the band, and added by the lane that overwrites it
    // there.  ANY: rows of any length, by units of 8 that start at any element and
    // end at N.
    auto fused_staged = [&](int j, v16f (&acc)[NBN][NBM], uint32_t stage_off, auto any_tag) __attribute__((always_inline)) {
        const Place p = place_of(tile_of(j));
        constexpr int CB = NBO >= 2 ? 2 : 1;                 // blocks of a band
        constexpr bool ANY = decltype(any_tag)::value;
        constexpr int UPR = 4 * CB, RPI = 64 / UPR;   // units of a band row; rows of a store
        constexpr int STEPS = 32 / RPI;
        const uint32_t bytes = (uint32_t)p.rows * (uint32_t)N * 2u;
        const __amdgpu_buffer_rsrc_t rsD = panel(reinterpret_cast<uint8_t*>(Dv) + (int64_t)p.m0 * N * 2, bytes);
        const __amdgpu_buffer_rsrc_t rsR = panel(reinterpret_cast<const uint8_t*>(ex.residual) + (int64_t)p.m0 * N * 2, bytes);
        typedef unsigned int v2u __attribute__((ext_vector_type(2)));
        const int lane_e = fresh_lane();
        const int l32e = lane_e & 31, lhie = lane_e >> 5;
        uint8_t* st = smem + stage_off + wave * 4096;
        const float* lsa = reinterpret_cast<const float*>(smem + ts_off(stage_off));
        const float* lsb = reinterpret_cast<const float*>(smem + ts_off(stage_off) + 1024);
        // chunk c of row r in slot c ^ key(r); 8-byte halves swapped when r >= 16
        auto key = [](int r) { return CB == 2 ? (r >> 1) & 7 : (r >> 2) & 3; };
        const uint32_t wkey = (uint32_t)key(l32e), whalf = (uint32_t)(lhie ^ (l32e >> 4));
        const int rc = lane_e & (UPR - 1), rr = lane_e / UPR;      // read-back: unit, row within RPI
        auto band = [&](int ih, int jb, const v4f (&b)[CB][GATED ? 2 : 1][4], auto bias_tag, auto act_tag)
                        __attribute__((always_inline)) {
            const int n = p.n0 + 32 * (wn * NBO + CB * ih) + 8 * rc;
            // branch-free select (a compare-and-select here becomes a branch)
            uint32_t keep = n < N ? 0xFFFFFFFFu : 0u;
            asm volatile("" : "+v"(keep));
            auto at = [&](int k) __attribute__((always_inline)) -> uint32_t {      // offset in the tile's rows
                const uint32_t mr = (uint32_t)(wm * WTM + jb * 32 + RPI * k + rr);
                return (((mr * (uint32_t)N + (uint32_t)n) * 2u) & keep) | (OOB_OFF & ~keep);
            };
            auto slot = [&](int k) __attribute__((always_inline)) {
                const int r = RPI * k + rr;
                return reinterpret_cast<v4u*>(st + r * (64 * CB) + ((rc ^ key(r)) << 4));
            };
            // element of D and of the residual where ANY unit k starts, how many of its 8 there are
            auto first = [&](int k) __attribute__((always_inline)) {
                return ((int64_t)p.m0 + wm * WTM + jb * 32 + RPI * k + rr) * N + n;
            };
            auto many = [&](int k) __attribute__((always_inline)) {
                return wm * WTM + jb * 32 + RPI * k + rr < p.rows ? N - n : 0;
            };
            if (RES && ex.residual) {
                v4u d[STEPS];
#pragma unroll
                for (int k = 0; k < STEPS; ++k) {
                    if constexpr (ANY) d[k] = load_some(reinterpret_cast<const uint16_t*>(ex.residual) + first(k), many(k));
                    else d[k] = __builtin_amdgcn_raw_buffer_load_b128(rsR, at(k), 0, 0);
                }
#pragma unroll
                for (int k = 0; k < STEPS; ++k) {
                    if (RPI * k >= 16) d[k] = (v4u){d[k].z, d[k].w, d[k].x, d[k].y};
                    *slot(k) = d[k];
                }
            }
            float smv = 1.0f;
            if constexpr (!MX) smv = lsa[wm * WTM + jb * 32 + l32e];
#pragma unroll
            for (int ii = 0; ii < CB; ++ii)
#pragma unroll
                for (int gq = 0; gq < 4; ++gq) {
                    float v[4];
                    fused_values(acc, CB * ih + ii, jb, gq, smv, lsb, lhie, b[ii], decltype(bias_tag)::value,
                                 decltype(act_tag)::value, v);
                    v2u* to = reinterpret_cast<v2u*>(st + l32e * (64 * CB) + (((uint32_t)(4 * ii + gq) ^ wkey) << 4) + whalf * 8);
                    if (RES && ex.residual) {
                        const v2u r = *to;
                        v[0] += __builtin_bit_cast(float, r.x << 16);
                        v[1] += __builtin_bit_cast(float, r.x & 0xFFFF0000u);
                        v[2] += __builtin_bit_cast(float, r.y << 16);
                        v[3] += __builtin_bit_cast(float, r.y & 0xFFFF0000u);
                    }
                    *to = (v2u){bf16x2_bits(v[0], v[1]), bf16x2_bits(v[2], v[3])};
                    // the 256x256 tile's waves have no registers for a second four
                    if constexpr (TILE == 256) __builtin_amdgcn_sched_barrier(0);
                }
#pragma unroll
            for (int k = 0; k < STEPS; ++k) {
                v4u d = *slot(k);
                if (RPI * k >= 16) d = (v4u){d.z, d.w, d.x, d.y};   // rows 16..31: halves swapped
                if constexpr (ANY) store_some(reinterpret_cast<uint16_t*>(Dv) + first(k), many(k), d);
                else __builtin_amdgcn_raw_buffer_store_b128(d, rsD, at(k), 0, ST_NT);
            }
            __builtin_amdgcn_sched_barrier(0);
        };
        fused_kind([&](auto bias_tag, auto act_tag) __attribute__((always_inline)) {
#pragma unroll
            for (int ih = 0; ih < NBO / CB; ++ih) {
                v4f b[CB][GATED ? 2 : 1][4] = {};
                if constexpr (decltype(bias_tag)::value) {
#pragma unroll
                    for (int ii = 0; ii < CB; ++ii) fused_bias(p, CB * ih + ii, b[ii], lhie);
                }
#pragma unroll
                for (int jb = 0; jb < NBM; ++jb) band(ih, jb, b, bias_tag, act_tag);
            }
        });
    };
    // fp32 through LDS, as epilogue_staged_f32; the residual is added where the
    // rows are stored.  ANY: as above, by units of 4.
    auto fused_staged_f32 = [&](int j, v16f (&acc)[NBN][NBM], uint32_t stage_off, auto any_tag) __attribute__((always_inline)) {
        const Place p = place_of(tile_of(j));
        constexpr bool ANY = decltype(any_tag)::value;
        const uint32_t bytes = (uint32_t)p.rows * (uint32_t)N * 4u;
        const __amdgpu_buffer_rsrc_t rsD = panel(reinterpret_cast<uint8_t*>(Dv) + (int64_t)p.m0 * N * 4, bytes);
        const __amdgpu_buffer_rsrc_t rsR = panel(reinterpret_cast<const uint8_t*>(ex.residual) + (int64_t)p.m0 * N * 4, bytes);
        const int lane_e = fresh_lane();
        const int l32e = lane_e & 31, lhie = lane_e >> 5;
        uint8_t* st = smem + stage_off + wave * 4096;
        const float* lsa = reinterpret_cast<const float*>(smem + ts_off(stage_off));
        const float* lsb = reinterpret_cast<const float*>(smem + ts_off(stage_off) + 1024);
        const uint32_t wkey = (uint32_t)((l32e >> 1) & 7);
        const int rc = lane_e & 7, rr = lane_e >> 3;
        fused_kind([&](auto bias_tag, auto act_tag) __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < NBO; ++i) {
                v4f b[GATED ? 2 : 1][4] = {};
                if constexpr (decltype(bias_tag)::value) fused_bias(p, i, b, lhie);
                const int n = p.n0 + 32 * (wn * NBO + i) + 4 * rc;
                uint32_t keep = n < N ? 0xFFFFFFFFu : 0u;
                asm volatile("" : "+v"(keep));
#pragma unroll
                for (int jb = 0; jb < NBM; ++jb) {
                    float smv = 1.0f;
                    if constexpr (!MX) smv = lsa[wm * WTM + jb * 32 + l32e];
#pragma unroll
                    for (int gq = 0; gq < 4; ++gq) {
                        float v[4];
                        fused_values(acc, i, jb, gq, smv, lsb, lhie, b, decltype(bias_tag)::value, decltype(act_tag)::value, v);
                        const uint32_t pc = (uint32_t)(2 * gq + lhie) ^ wkey;
                        *reinterpret_cast<v4f*>(st + l32e * 128 + pc * 16) = (v4f){v[0], v[1], v[2], v[3]};
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int r = 8 * k + rr, mr = wm * WTM + jb * 32 + r;            // row inside the tile
                        v4f d = *reinterpret_cast<const v4f*>(st + r * 128 + ((rc ^ ((r >> 1) & 7)) << 4));
                        if constexpr (ANY) {
                            const int64_t first = ((int64_t)p.m0 + mr) * N + n;
                            const int many = mr < p.rows ? N - n : 0;
                            if (RES && ex.residual) d += __builtin_bit_cast(v4f, load_some(reinterpret_cast<const uint32_t*>(ex.residual) + first, many));
                            store_some(reinterpret_cast<uint32_t*>(Dv) + first, many, __builtin_bit_cast(v4u, d));
                        } else {
                            const uint32_t off = ((((uint32_t)mr * (uint32_t)N + (uint32_t)n) * 4u) & keep) | (OOB_OFF & ~keep);
                            if (RES && ex.residual) d += __builtin_bit_cast(v4f, __builtin_amdgcn_raw_buffer_load_b128(rsR, off, 0, 0));
                            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(v4u, d), rsD, off, 0, ST_NT);
                        }
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        });
    };
    // 256x256 tiles are chosen for whole vectors only: their registers hold no more
    auto fused_any = [&](int j, v16f (&acc)[NBN][NBM], uint32_t stage_off) __attribute__((always_inline)) {
        auto staged = [&](auto any_tag) __attribute__((always_inline)) {
            if constexpr (OUT_F32) fused_staged_f32(j, acc, stage_off, any_tag);
            else fused_staged(j, acc, stage_off, any_tag);
        };
        if constexpr (TILE == 256) {
            staged(std::false_type{});
        } else {
            if (N % (OUT_F32 ? 4 : 8) == 0) staged(std::false_type{});
            else staged(std::true_type{});
        }
    };
    // ---- partial sums (EPI_PARTIAL): the item's accumulators as they are, whole
    // tiles of rows of ex.pitch elements, through LDS as in epilogue_staged_f32
    auto partial_staged = [&](int j, v16f (&acc)[NBN][NBM]) __attribute__((always_inline)) {
        const int t = run0 + slot + j * wx, range = t / tiles;
        const TileCoord tc = tile_of(j);
        const uint32_t pitch = (uint32_t)ex.pitch;
        const __amdgpu_buffer_rsrc_t rsD = panel(
            reinterpret_cast<uint8_t*>(Dv) + (((int64_t)range * ex.part_rows + tc.tm * BM) * pitch + tc.tn * BN) * 4,
            ((uint32_t)(BM - 1) * pitch + BN) * 4u);
        const int lane_e = fresh_lane();
        const int l32e = lane_e & 31, lhie = lane_e >> 5;
        uint8_t* st = smem + R::STAGE_AREA + wave * 4096;
        const uint32_t wkey = (uint32_t)((l32e >> 1) & 7);
        const uint32_t rc = (uint32_t)(lane_e & 7);
        const int rr = lane_e >> 3;
        const uint32_t rd_off = (uint32_t)(rr * 128) + ((rc ^ (uint32_t)((rr >> 1) & 3)) << 4);
#pragma unroll
        for (int i = 0; i < NBN; ++i)
#pragma unroll
            for (int jb = 0; jb < NBM; ++jb) {
#pragma unroll
                for (int gq = 0; gq < 4; ++gq) {
                    const uint32_t pc = (uint32_t)(2 * gq + lhie) ^ wkey;
                    *reinterpret_cast<v4f*>(st + l32e * 128 + pc * 16) =
                        (v4f){acc[i][jb][4 * gq], acc[i][jb][4 * gq + 1], acc[i][jb][4 * gq + 2], acc[i][jb][4 * gq + 3]};
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const v4u d = *reinterpret_cast<const v4u*>(st + k * 1024 + (rd_off ^ (uint32_t)(64 * (k & 1))));
                    const uint32_t mr = (uint32_t)(wm * WTM + jb * 32 + 8 * k + rr);   // row inside the tile
                    const uint32_t col = (uint32_t)(wn * WTN + 32 * i) + 4u * rc;
                    __builtin_amdgcn_raw_buffer_store_b128(d, rsD, (mr * pitch + col) * 4u, 0, 0);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
    };
    // Staged epilogues: bf16 for N % 8 == 0; fp32 in mode (a) for N % 32 == 0,
    // rows of whole 128-byte lines (at N = 22012, rows straddling lines, staged
    // fp32 ran 4% slower than from registers; mode (b) with fp32 output staged
    // spilled in its main loop)
    const bool staged = EPI != EPI_NONE || (OUT_F32 ? (!MX && (N % 32) == 0) : (N % 8) == 0);
    auto epilogue_staged_any = [&](int j, v16f (&acc)[NBN][NBM], uint32_t stage_off) __attribute__((always_inline)) {
        if constexpr (EPI != EPI_NONE) fused_any(j, acc, stage_off);
        else if constexpr (OUT_F32) epilogue_staged_f32(j, acc, stage_off);
        else epilogue_staged(j, acc, stage_off);
    };

    // ---- split reduction (SPLIT: the workgroup's split item, after its last K
    // step).  Every split item stores its fp32 partial tile to ws (item
    // u * split + s; per wave and block 4 KB: accumulators 4c .. 4c+3 of lane
    // L at 1024 c + 16 L, so that every store covers 1 KB in whole lines) and,
    // once those stores have completed, counts itself
    // in cnt[u].  The item that arrives last (count split - 1) reads the other
    // partials and adds all of them in split order, p0 + p1 + ..., its own
    // from registers, so the sum does not depend on the order of arrival; it
    // resets cnt[u] to zero for the next launch and returns true: its
    // workgroup stores the tile.  No workgroup waits for another.
    // Coherence across the XCDs' separate L2 caches comes from the accesses
    // themselves, not from fences: the partials are stored and loaded with
    // device scope (SC1: written through to, and read from, the level all XCDs
    // share) and the counter is a device-scope atomic.  A device-scope fence
    // would instead write back and invalidate the whole L2 of the XCD, taking
    // every other workgroup's operand panels with it (measured: the 2048 x
    // 1024 x 4096 GEMM ran 3.6x slower so).  The LDS word at stage_off (the
    // epilogue's staging area, free here) passes the count to all waves.
    constexpr int CP_SC1 = 16;   // cache policy of the buffer builtins: device scope
    auto split_reduce = [&](v16f (&acc)[NBN][NBM], uint32_t stage_off) __attribute__((always_inline)) -> bool {
        const int u = my_split / split, sidx = my_split % split;
        const int ln = fresh_lane();
        constexpr uint32_t PART = BM * BN * 4;   // bytes per partial tile
        const __amdgpu_buffer_rsrc_t rw = panel(reinterpret_cast<uint8_t*>(ws) + (size_t)my_split * PART, PART);
#pragma unroll
        for (int i = 0; i < NBN; ++i)
#pragma unroll
            for (int jb = 0; jb < NBM; ++jb) {
                const uint32_t off = (uint32_t)((wave * NBN * NBM + i * NBM + jb) * 4096 + ln * 16);
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    __builtin_amdgcn_raw_buffer_store_b128(
                        __builtin_bit_cast(v4u, (v4f){acc[i][jb][4 * c], acc[i][jb][4 * c + 1], acc[i][jb][4 * c + 2],
                                                      acc[i][jb][4 * c + 3]}),
                        rw, off + 1024 * c, 0, CP_SC1);
            }
        asm volatile("s_waitcnt vmcnt(0)" : : : "memory");   // this wave's partial is visible device-wide
        __syncthreads();
        int* flag = reinterpret_cast<int*>(smem + stage_off);
        if (tid == 0) {
            const int old = __hip_atomic_fetch_add(cnt + u, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            *flag = (old == split - 1) ? 1 : 0;
        }
        __syncthreads();
        const bool last = *flag != 0;
        __syncthreads();   // every wave has read the flag before that LDS is used again
        if (!last) return false;
        const __amdgpu_buffer_rsrc_t rr =
            panel(reinterpret_cast<uint8_t*>(ws) + (size_t)(u * split) * PART, PART * (uint32_t)split);
        auto load16 = [&](uint32_t off) __attribute__((always_inline)) -> v16f {
            const v4f a = __builtin_bit_cast(v4f, __builtin_amdgcn_raw_buffer_load_b128(rr, off, 0, CP_SC1));
            const v4f b4 = __builtin_bit_cast(v4f, __builtin_amdgcn_raw_buffer_load_b128(rr, off + 1024, 0, CP_SC1));
            const v4f c = __builtin_bit_cast(v4f, __builtin_amdgcn_raw_buffer_load_b128(rr, off + 2048, 0, CP_SC1));
            const v4f d = __builtin_bit_cast(v4f, __builtin_amdgcn_raw_buffer_load_b128(rr, off + 3072, 0, CP_SC1));
            return (v16f){a.x, a.y, a.z, a.w, b4.x, b4.y, b4.z, b4.w, c.x, c.y, c.z, c.w, d.x, d.y, d.z, d.w};
        };
        // the split count as a constant, so that every partial's loads of a
        // block are issued together (a runtime loop waited for each in turn)
        auto add_parts = [&](auto s_tag) __attribute__((always_inline)) {
            constexpr int S = decltype(s_tag)::value;
#pragma unroll
            for (int i = 0; i < NBN; ++i)
#pragma unroll
                for (int jb = 0; jb < NBM; ++jb) {
                    const uint32_t off = (uint32_t)((wave * NBN * NBM + i * NBM + jb) * 4096 + ln * 16);
                    v16f p[S];
#pragma unroll
                    for (int s2 = 0; s2 < S; ++s2)
                        if (s2 != sidx) p[s2] = load16(s2 * PART + off);
                    v16f t = sidx == 0 ? acc[i][jb] : p[0];
#pragma unroll
                    for (int s2 = 1; s2 < S; ++s2) t += s2 == sidx ? acc[i][jb] : p[s2];
                    acc[i][jb] = t;
                }
        };
        if (split == 2) add_parts(std::integral_constant<int, 2>{});
        else if (split == 3) add_parts(std::integral_constant<int, 3>{});
        else add_parts(std::integral_constant<int, 4>{});
        if (tid == 0) __hip_atomic_store(cnt + u, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        return true;
    };

    if (nk == 0) {   // K == 0: every tile is the empty sum
        for (int j = 0; j < my_tiles; ++j) {
            v16f acc[NBN][NBM];
#pragma unroll
            for (int i = 0; i < NBN; ++i)
#pragma unroll
                for (int jb = 0; jb < NBM; ++jb) acc[i][jb] = (v16f){};
            tile_scales_to_lds(j, 0);
            wait_vmcnt<0>();
            __syncthreads();
            if (staged) epilogue_staged_any(j, acc, 0);
            else epilogue(j, acc, 0);
            __syncthreads();
        }
        return;
    }
    if (NS == 0) return;

    // ---- prologue: items 0 .. NSLOT-2 in flight; stage 0 (items 0, 1) and the
    // first scale group (loaded before them) landed, and the fragments and
    // scales of step 0 read
    cursor_tile();
    if constexpr (R::SCALES) {
        sc_tile(0);
#pragma unroll
        for (int q = 0; q < SC_LOADS; ++q) sc_load(q, 0, 0);
    }
    constexpr int PRO_ITEMS = R::PAIRED ? 4 : NSLOT - 1;   // items in flight before step 0
    for (int i = 0; i < PRO_ITEMS; ++i) {
        const int nq = (i & 1) ? LB : LA;   // item i is operand i & 1
#pragma unroll
        for (int q = 0; q < nq; ++q) dma_item(q);
        advance();
    }
    wait_vmcnt<loads_of(PRO_ITEMS - 2)>();
    __syncthreads();

    // Fragment registers are double-buffered: step t computes from one set
    // while the other receives step t+1's fragments.
    v8i fa0[NBM], fb0[NBN], fa1[NBM], fb1[NBN];
    uint32_t xa[NBM] = {}, xb[NBN] = {};
#pragma unroll
    for (int i = 0; i < NBX; ++i) {
        if (i < NBM) fa0[i] = frag(0, frag_a, 0, i);
        if (i < NBN) fb0[i] = frag(slot_off(1), frag_b, 0, i);
    }
    read_scales(0, 0, 0, xa, xb);
    int rslot = 0;   // LDS slot of the current stage's A item (its B item is the next slot)

    // ---- one K step: step h of stage s of stream tile j (fragments and scales
    // in registers).
    //   the NBM matrix-core steps of row block 0 (4 for 256-row tiles);
    //   h == 1 only: wait until the next stage's items landed (items past them
    //   may be in flight) and sync: they landed for every wave, and every wave's
    //   reads of this stage's items (done during step 0) are finished (the
    //   barrier waits for outstanding LDS reads), so their slots may be refilled;
    //   the remaining (NBN-1)·NBM matrix-core steps ("slots": 12 for 256x256
    //   tiles), each with its share of the loads of the item NSLOT-1 ahead
    //   (into the slot of the item just before this step's) and of the next
    //   step's fragment reads (two 16-byte LDS reads each) into the other
    //   register set.  Spreading the loads keeps the address unit from blocking the
    //   matrix-core steps behind a burst of loads from all four waves.
    //   LAST (the tile's last step): no reads of the next step's fragments (they
    //   are read after the epilogue, which then has their registers to itself).
    // matrix-core steps after row block 0: 12 for 256x256 tiles, 4 for
    // 256x128, 2 for 128x128 and 1 for 64x128; the step's loads and the next
    // step's NBM + NBN fragment reads are spread over them.
    // Mode (b) scales from LDS (once per stage, in its step 1, for the next
    // stage) are read first, in slot 0: LDS reads complete in order, so scales
    // read after the fragments would hold the next step's first matrix-core
    // instruction until every fragment read had landed.
    // Scales loaded byte-wise from global memory (K tail) are read after the
    // step's item loads instead.
    // Mode (b) scale groups: step 0 of a group's first stage loads the next
    // group (the tile's next, or the next tile's first) into the other buffer,
    // whose group was last read in step 0 of the stage before, ahead of the
    // barrier of that stage's step 1.  The paired ring spreads the loads over
    // this step, which loads no items; with 5 or more slots they go first,
    // before the item loads, which the next wait may leave in flight.  Either way they
    // have landed at that wait, the earliest point the group is read.
    constexpr int SLOTS = (NBN - 1) * NBM;
    constexpr int NREAD = NBM + NBN;
    static_assert(SLOTS >= 1, "a matrix-core slot after row block 0");
    constexpr int SCALE_SLOT = R::SCALES ? 0 : (SLOTS > NREAD ? NREAD + 1 : SLOTS - 1);
    // With NSLOT >= 5 slots the ring runs NSLOT - 1 items ahead, one item per
    // step, so step h of every stage loads an item of operand (h + NSLOT - 1) & 1
    // (A: LA loads, B: LB).  LI_LAST: the loads of a stage's step 1 (mode (a)).
    constexpr int LI_LAST = (NSLOT & 1) ? LB : LA;
    auto kstep = [&](v16f (&acc)[NBN][NBM], int j, int s, auto h_tag, auto last_tag, const v8i* fa, const v8i* fb,
                     v8i* na, v8i* nbf) __attribute__((always_inline)) {
        constexpr int h = decltype(h_tag)::value;
        constexpr bool LAST = decltype(last_tag)::value;
        using Ops = std::integral_constant<int, R::SCALES ? 2 * h : 0>;
        constexpr int LI_STEP = ((h + NSLOT - 1) & 1) ? LB : LA;   // this step's loads (unpaired ring)
        // whole scale dwords are read once per stage, in its step 1 for the next stage
        constexpr bool READ_SC = !R::SCALES || h == 1;
        bool sc_go = false;
        int sc_gi = 0, sc_ub = 0;
        if constexpr (R::SCALES) {
            if (h == 0 && s % R::SC_GROUP == 0) {
                const bool in_tile = s + R::SC_GROUP < nk;
                if (in_tile || j + 1 < my_tiles) {
                    if (!in_tile) sc_tile(j + 1);
                    sc_go = true;
                    sc_gi = in_tile ? s / R::SC_GROUP + 1 : 0;
                    sc_ub = (j * ngt + s / R::SC_GROUP + 1) & 1;
                }
            }
        }
#pragma unroll
        for (int jb = 0; jb < NBM; ++jb) mfma(acc[0][jb], fb[0], fa[jb], xb[0], xa[jb], Ops{});
        if (h == 1) {
            __builtin_amdgcn_sched_barrier(0);
            // the next stage's items landed: with NSLOT >= 5 slots the NSLOT-4
            // items issued after them may be in flight; with 4 (paired) none
            wait_vmcnt<R::PAIRED ? 0 : loads_of(NSLOT - 4)>();
            __syncthreads();
            // last stage of a tile: the slot of its B item is now free until the
            // next tile's first step; load the tile's scales into it for the
            // epilogue (before this step's item loads, so that waiting for all
            // but those leaves the scales landed)
            if constexpr (!MX && LAST && !PARTIAL) {
                tile_scales_to_lds(j, R::OWN_STAGE ? (uint32_t)R::STAGE_AREA : slot_off(slot_add(rslot, 1)));
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        const int sn = h ? s + 1 : s, hn = h ^ 1;
        const int na_slot = h ? slot_add(rslot, 2) : rslot;   // slots of the items read next
        const uint32_t sa_off = slot_off(na_slot), sb_off = slot_off(slot_add(na_slot, 1));
        uint32_t nxa[NBM], nxb[NBN];
#pragma unroll
        for (int k = 0; k < SLOTS; ++k) {
            const int i = 1 + k / NBM, jb = k % NBM;
            mfma(acc[i][jb], fb[i], fa[jb], xb[i], xa[jb], Ops{});
            if constexpr (R::SCALES) {
                if (sc_go) {
                    if constexpr (R::PAIRED) {
#pragma unroll
                        for (int q = share_lo(k, SC_LOADS, SLOTS); q < share_hi(k, SC_LOADS, SLOTS); ++q)
                            sc_load(q, sc_gi, sc_ub);
                    } else if (k == 0) {
#pragma unroll
                        for (int q = 0; q < SC_LOADS; ++q) sc_load(q, sc_gi, sc_ub);
                    }
                }
            }
            if constexpr (!R::PAIRED) {
#pragma unroll
                for (int q = share_lo(k, LI_STEP, SLOTS); q < share_hi(k, LI_STEP, SLOTS); ++q) dma_item(q);
            } else if (h == 1) {
                // the stage's two items: the first over the first half of the slots, the second over the rest
                constexpr int HALF = SLOTS / 2;
                const int kk = k % HALF;
#pragma unroll
                for (int q = kk * LA / HALF; q < (kk + 1) * LA / HALF; ++q) dma_item(q);
                if (k == HALF - 1) advance();
            }
            // reads in order of first use: row block 0 of B, the NBM of A, then the rest of B
            if constexpr (!LAST) {
                if (R::SCALES && READ_SC && k == SCALE_SLOT) read_scales(j, sn, hn, nxa, nxb);
#pragma unroll
                for (int e = share_lo(k, NREAD, SLOTS); e < share_hi(k, NREAD, SLOTS); ++e) {
                    if (e == 0) nbf[0] = frag(sb_off, frag_b, hn, 0);
                    else if (e <= NBM) na[e - 1] = frag(sa_off, frag_a, hn, e - 1);
                    else nbf[e - NBM] = frag(sb_off, frag_b, hn, e - NBM);
                }
                if (!R::SCALES && k == SCALE_SLOT) read_scales(j, sn, hn, nxa, nxb);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        if (!R::PAIRED || h == 1) advance();
        if (h) rslot = na_slot;
        // keep this step's operand registers allocated to its end
#pragma unroll
        for (int i = 0; i < NBX; ++i) {
            if (i < NBM && i < NBN) asm volatile("" : : "v"(fa[i]), "v"(fb[i]));
            else if (i < NBM) asm volatile("" : : "v"(fa[i]));
            else asm volatile("" : : "v"(fb[i]));
        }
        if constexpr (!LAST && READ_SC) {
#pragma unroll
            for (int i = 0; i < NBX; ++i) {
                if (i < NBM) xa[i] = nxa[i];
                if (i < NBN) xb[i] = nxb[i];
            }
        }
    };
    using Step0 = std::integral_constant<int, 0>;
    using Step1 = std::integral_constant<int, 1>;
    using NotLast = std::integral_constant<bool, false>;
    using Last = std::integral_constant<bool, true>;

    for (int j = 0; j < my_tiles; ++j) {
        v16f acc[NBN][NBM];   // [n block][m block]
#pragma unroll
        for (int i = 0; i < NBN; ++i)
#pragma unroll
            for (int jb = 0; jb < NBM; ++jb) acc[i][jb] = (v16f){};
        const int nsj = SPLIT || PARTIAL ? item_of(j).ns : nk;   // stages of this work item
        for (int s = 0; s < nsj - 1; ++s) {
            kstep(acc, j, s, Step0{}, NotLast{}, fa0, fb0, fa1, fb1);
            kstep(acc, j, s, Step1{}, NotLast{}, fa1, fb1, fa0, fb0);
        }
        kstep(acc, j, nsj - 1, Step0{}, NotLast{}, fa0, fb0, fa1, fb1);
        kstep(acc, j, nsj - 1, Step1{}, Last{}, fa1, fb1, fa0, fb0);
        // the slot of the last stage's B item is free until the next K step
        // loads into it (every wave finished reading it before the last barrier)
        const uint32_t stage_off = R::OWN_STAGE ? (uint32_t)R::STAGE_AREA : slot_off(slot_add(rslot, NSLOT - 1));
        if constexpr (SPLIT) {
            // the split item is the workgroup's last: the one that does not add
            // up the tile has no epilogue and nothing after it
            if (j == my_whole && !split_reduce(acc, stage_off)) break;
        }
        if constexpr (PARTIAL) {
            partial_staged(j, acc);
        } else if (staged) {
            if constexpr (!MX) wait_vmcnt<LI_LAST>();   // the tile's scales (only the last item's loads may be in flight)
            __syncthreads();
            epilogue_staged_any(j, acc, stage_off);
            __syncthreads();   // staging reads done before that slot is loaded again
        } else {
            if constexpr (!MX) {
                wait_vmcnt<LI_LAST>();
                __syncthreads();
            }
            epilogue(j, acc, stage_off);
            if constexpr (!MX) __syncthreads();   // scale reads done before that slot is loaded again
        }
        // the next stage's step-0 fragments and scales (its items landed before
        // the last barrier; the slots of this stage's items are not refilled
        // before the next barrier).  After the last tile the fragment reads
        // (LDS) are harmless and unused; the scales are read only for a tile
        // that exists (the K-tail path reads them from global memory).
#pragma unroll
        for (int i = 0; i < NBX; ++i) {
            if (i < NBM) fa0[i] = frag(slot_off(rslot), frag_a, 0, i);
            if (i < NBN) fb0[i] = frag(slot_off(slot_add(rslot, 1)), frag_b, 0, i);
        }
        if (j + 1 < my_tiles) read_scales(j + 1, 0, 0, xa, xb);
    }
    wait_vmcnt<0>();   // the past-the-end loads must land before the workgroup exits
}

}  // namespace fp8g
