// Fused FP8 products for few rows, one product or one for every expert.
//
//   z[m, j] = sa[m] sb[j] sum_k A[m, k] B[j, k] + bias[j]      (or block scales)
//   D[m, n] = act(z[m, n]) (* z[m, N + n] where gated) + residual[m, n]
//
// With few rows the weights' bytes are the bound, so nothing stands between
// them and the matrix core: a wave loads a 16 x 128-byte piece of B straight
// into the operand registers (lane L holds chunks L/16 and 4 + L/16, 16 bytes
// each, of row L % 16; rows of 128 bytes are whole lines), and A's pieces, which
// all workgroups share and the L2 holds, the same way.
//
// The four waves of a workgroup split K: wave w takes the 128-byte steps w, w + 4,
// ..., so that together they read 512 bytes of each row in turn, and every wave has
// the loads of `AHEAD` steps in flight.  Their sums meet in LDS, added in the
// order of the waves, and a thread finishes four neighbouring columns of a row.
// Bound by the weights: 64 experts of 2 x 1408 x 4096 with six rows each, 738 MB,
// 133 us (5.6 TB/s).
//
// The instruction is V_MFMA_SCALE_F32_16X16X128_F8F6F4 with B's rows as its
// first operand, so a lane's four results are four neighbouring columns n of one
// row m.  A lane's first 16 operand bytes are elements 16 g .. 16 g + 15 of the
// 128 (g = lane / 16), its second 64 + 16 g ..; lane group g brings the scale of
// the 32-element block g.  Block scales pass through LDS where a workgroup's fit
// (SC_LDS): fetched by the step they are a load each for a byte a lane, half as
// many again as the operands' (64 experts of 2 x 1408 x 4096, 6 rows: 168 us so).

#include <atomic>
#include <type_traits>

#include "epilogue.h"
#include "launch_ffn.h"

namespace fp8g {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef unsigned int v4u __attribute__((ext_vector_type(4)));
typedef unsigned int v2u __attribute__((ext_vector_type(2)));
typedef float v4f __attribute__((ext_vector_type(4)));

constexpr int RW_WAVES = 4;
constexpr int RW_THREADS = 64 * RW_WAVES;
constexpr uint32_t RW_OOB = 0x80000000u;      // past any panel (panels are < 2^31 bytes)

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rw_panel(const void* p, int64_t bytes) {
    // loads at or past the end return 0
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, (int)bytes, 0x00020000);
}

struct RowsArgs {
    FusedArgs f;
    Act act;
};

// Bytes between the scale rows in LDS: whole 16 bytes, an odd number of them, so
// that the 16 rows of a read lie in different banks.
__host__ __device__ constexpr int scale_pitch(int nblk) { return ((nblk + 15) / 16 | 1) * 16; }
constexpr int SC_LIMIT = 40 * 1024;       // of a workgroup, beside 4 to 32 KB of sums: two or three on a CU at least

// B's rows of a workgroup: NB blocks of 16; gated: the first half of them the
// gate's, the others the up projection's.  MB: blocks of 16 rows of A.  AHEAD:
// steps in flight.  WPE: waves of a SIMD that the registers are to allow.
template <bool MX, bool SC_LDS, bool GATED, int NB, int MB, int AHEAD, int WPE>
__global__ __launch_bounds__(RW_THREADS, WPE) void gemm_rows_kernel(RowsArgs args) {
    const FusedArgs& a = args.f;
    constexpr int H = GATED ? 2 : 1;                      // projections
    constexpr int NO = NB / H;                            // blocks of one
    constexpr int COLS = 16 * NO;                         // output columns
    constexpr int UNITS = COLS / 4 * 16 * MB;             // threads that finish: four columns of a row each
    static_assert(NB % H == 0 && UNITS <= RW_THREADS, "one unit a thread");
    static_assert(MX || !SC_LDS, "block scales");
    __shared__ v4f red[RW_WAVES][NB * MB][64];
    extern __shared__ __attribute__((aligned(16))) uint8_t scales[];      // SC_LDS: B's rows, then A's
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int l16 = lane & 15, g = lane >> 4;
    const int N = (int)a.n, K = (int)a.k, nblk = K / 32;
    const int n0 = (int)blockIdx.x * COLS;                // first output column
    const int64_t b_rows = GATED ? 2 * (int64_t)N : N;    // B's rows of a product
    const uint8_t* B = a.B;
    int64_t s0 = (int64_t)blockIdx.y * (16 * MB), s1 = a.m, step = (int64_t)gridDim.y * (16 * MB);
    int64_t b_row = 0;                                    // this product's first row of scale_b and bias
    if (a.expert_start) {
        const int e = blockIdx.y, S = (int)a.m;
        s0 = min(max(a.expert_start[e], 0), S);
        s1 = min(max(a.expert_start[e + 1], (int)s0), S);
        s0 += (int64_t)blockIdx.z * (16 * MB);            // the expert's blocks of rows, in turn
        if (s0 >= s1) return;
        step = (int64_t)gridDim.z * (16 * MB);
        b_row = e * b_rows;
        B += b_row * K;
    }
    const int steps = (K + 127) / 128;
    const bool gather = a.rows != nullptr;

    const int cols = min(COLS, N - n0);
    __amdgpu_buffer_rsrc_t rsB[H], rsEB[H];
#pragma unroll
    for (int h = 0; h < H; h++) {
        const int64_t first = n0 + (int64_t)h * N;
        rsB[h] = rw_panel(B + first * K, (int64_t)cols * K);
        if constexpr (MX)
            rsEB[h] = rw_panel(static_cast<const uint8_t*>(a.scale_b) + (b_row + first) * nblk, (int64_t)cols * nblk);
    }
    uint32_t vb[NO], veb[NO];
#pragma unroll
    for (int i = 0; i < NO; i++) {
        vb[i] = (uint32_t)(16 * i + l16) * (uint32_t)K + 16u * g;
        veb[i] = (uint32_t)(16 * i + l16) * (uint32_t)nblk + g;
    }

    // SC_LDS: `rows` rows of nblk scale bytes into LDS from row `at` on; from(r): row
    // r's, or nullptr
    const int pitch = scale_pitch(nblk);
    auto fetch_scales = [&](int at, int rows, auto from) __attribute__((always_inline)) {
        if (nblk % 16 == 0) {
            const int per = nblk / 16;
            for (int i = threadIdx.x; i < rows * per; i += RW_THREADS) {
                const int r = i / per, c = i - r * per;
                const uint8_t* p = from(r);
                if (p) reinterpret_cast<v4u*>(scales + (at + r) * pitch)[c] = reinterpret_cast<const v4u*>(p)[c];
            }
            return;
        }
        const int per = (nblk + 3) / 4;
        for (int i = threadIdx.x; i < rows * per; i += RW_THREADS) {
            const int r = i / per, c = i - r * per;
            const uint8_t* p = from(r);
            if (p) reinterpret_cast<uint32_t*>(scales + (at + r) * pitch)[c] = scale_word(p, c, nblk);
        }
    };
    if constexpr (SC_LDS) {
        fetch_scales(0, 16 * NB, [&](int r) {
            const int h = r / (16 * NO), c = r % (16 * NO);
            return c < cols ? static_cast<const uint8_t*>(a.scale_b) + (b_row + (int64_t)h * N + n0 + c) * nblk : nullptr;
        });
    }

    for (; s0 < s1; s0 += step) {
        const int count = (int)min((int64_t)(16 * MB), s1 - s0);
        // A: this chunk's rows, or with `rows` all of A
        const __amdgpu_buffer_rsrc_t rsA = gather ? rw_panel(a.A, a.a_rows * K) : rw_panel(a.A + s0 * K, (int64_t)count * K);
        __amdgpu_buffer_rsrc_t rsEA;
        if constexpr (MX) {
            const uint8_t* ea = static_cast<const uint8_t*>(a.scale_a);
            rsEA = gather ? rw_panel(ea, a.a_rows * nblk) : rw_panel(ea + s0 * nblk, (int64_t)count * nblk);
        }
        uint32_t va[MB], vea[MB];
#pragma unroll
        for (int j = 0; j < MB; j++) {
            int r = min(16 * j + l16, count - 1);         // rows past the end: the last one again, not stored
            if (gather) r = min(max(a.rows[s0 + r], 0), (int)a.a_rows - 1);
            va[j] = (uint32_t)r * (uint32_t)K + 16u * g;
            vea[j] = (uint32_t)r * (uint32_t)nblk + g;
        }
        if constexpr (SC_LDS) {
            fetch_scales(16 * NB, count, [&](int r) {
                const int64_t row = gather ? min(max(a.rows[s0 + r], 0), (int)a.a_rows - 1) : s0 + r;
                return static_cast<const uint8_t*>(a.scale_a) + row * nblk;
            });
        }

        struct Frag {
            v8i b[NB], a[MB];
            uint32_t eb[NB], ea[MB];
        };
        auto load16 = [&](__amdgpu_buffer_rsrc_t rs, uint32_t off, int st) __attribute__((always_inline)) -> v8i {
            const int kc = 128 * st + 16 * g;             // bytes past K read 0
            const uint32_t so = 128u * (uint32_t)st;
            const v4u x = __builtin_amdgcn_raw_buffer_load_b128(rs, kc < K ? off : RW_OOB, so, 0);
            const v4u y = __builtin_amdgcn_raw_buffer_load_b128(rs, kc + 64 < K ? off + 64u : RW_OOB, so, 0);
            return (v8i){(int)x.x, (int)x.y, (int)x.z, (int)x.w, (int)y.x, (int)y.y, (int)y.z, (int)y.w};
        };
        auto load = [&](int st, Frag& f) __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < NB; i++) f.b[i] = load16(rsB[i / NO], vb[i % NO], st);
#pragma unroll
            for (int j = 0; j < MB; j++) f.a[j] = load16(rsA, va[j], st);
            if constexpr (MX && !SC_LDS) {
                const bool in = 4 * st + g < nblk;
#pragma unroll
                for (int i = 0; i < NB; i++)
                    f.eb[i] = __builtin_amdgcn_raw_buffer_load_b8(rsEB[i / NO], in ? veb[i % NO] : RW_OOB, 4u * st, 0);
#pragma unroll
                for (int j = 0; j < MB; j++)
                    f.ea[j] = __builtin_amdgcn_raw_buffer_load_b8(rsEA, in ? vea[j] : RW_OOB, 4u * st, 0);
            }
        };
        v4f acc[NB][MB];
#pragma unroll
        for (int i = 0; i < NB; i++)
#pragma unroll
            for (int j = 0; j < MB; j++) acc[i][j] = (v4f){0.f, 0.f, 0.f, 0.f};

        // Steps past the last one load and add zeros.  The barriers keep each step's
        // loads behind the step before: reordered, the loop waited for all of them.
        Frag f[AHEAD];
#pragma unroll
        for (int u = 0; u < AHEAD; u++) {
            load(wave + RW_WAVES * u, f[u]);
            __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (SC_LDS) __syncthreads();
        for (int st = wave; st < steps; st += RW_WAVES * AHEAD) {
#pragma unroll
            for (int u = 0; u < AHEAD; u++) {
                if constexpr (SC_LDS) {
                    // blocks past K: some byte of the row; the codes there are zeros
                    const int c = min(4 * (st + RW_WAVES * u) + g, nblk - 1);
#pragma unroll
                    for (int i = 0; i < NB; i++) f[u].eb[i] = scales[(16 * i + l16) * pitch + c];
#pragma unroll
                    for (int j = 0; j < MB; j++) f[u].ea[j] = scales[(16 * NB + min(16 * j + l16, count - 1)) * pitch + c];
                }
#pragma unroll
                for (int i = 0; i < NB; i++)
#pragma unroll
                    for (int j = 0; j < MB; j++) {
                        if constexpr (MX)
                            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(f[u].b[i], f[u].a[j], acc[i][j], 0, 0, 0,
                                                                                         (int)f[u].eb[i], 0, (int)f[u].ea[j]);
                        else
                            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(f[u].b[i], f[u].a[j], acc[i][j], 0, 0, 0,
                                                                                         127, 0, 127);
                    }
                __builtin_amdgcn_sched_barrier(0);
                load(st + RW_WAVES * (u + AHEAD), f[u]);
                __builtin_amdgcn_sched_barrier(0);
            }
        }

        // a thread's unit: output columns n .. n + 3 of row mr; its scales and bias are
        // asked for before the sums meet
        const int i = wave / MB, j = wave % MB, mr = 16 * j + l16, nc = 16 * i + 4 * g;
        const bool mine = wave < NO * MB && mr < count && nc < cols;
        const int n = n0 + nc, left = min(4, cols - nc);
        const int64_t slot = s0 + mr;
        float sm = 1.0f, sn[H][4], bs[H][4];
        if (mine) {
            if constexpr (!MX) {
                int64_t r = slot;
                if (gather) r = min(max(a.rows[slot], 0), (int)a.a_rows - 1);
                sm = static_cast<const float*>(a.scale_a)[r];
            }
#pragma unroll
            for (int h = 0; h < H; h++)
#pragma unroll
                for (int c = 0; c < 4; c++) {
                    const int64_t row = b_row + (int64_t)h * N + n + min(c, left - 1);
                    sn[h][c] = MX ? 1.0f : static_cast<const float*>(a.scale_b)[row];
                    bs[h][c] = a.bias ? a.bias[row] : 0.0f;
                }
        }
#pragma unroll
        for (int x = 0; x < NB; x++)
#pragma unroll
            for (int y = 0; y < MB; y++) red[wave][x * MB + y][lane] = acc[x][y];
        __syncthreads();
        if (mine) {
            float z[H][4];
#pragma unroll
            for (int h = 0; h < H; h++) {
                const int from = (h * NO + i) * MB + j;
                v4f t = red[0][from][lane];
#pragma unroll
                for (int w = 1; w < RW_WAVES; w++) t += red[w][from][lane];
#pragma unroll
                for (int c = 0; c < 4; c++) z[h][c] = (MX ? t[c] : t[c] * sm * sn[h][c]) + bs[h][c];
            }
            float v[4];
#pragma unroll
            for (int c = 0; c < 4; c++) {
                v[c] = args.act.on ? activate(z[0][c], args.act.c1, args.act.c3) : z[0][c];
                if constexpr (GATED) v[c] *= z[1][c];
            }
            const int64_t at = slot * N + n;
            if (a.f32) {
                float* D = static_cast<float*>(a.D);
                const float* res = static_cast<const float*>(a.residual);
                for (int c = 0; c < left; c++) D[at + c] = res ? v[c] + res[at + c] : v[c];
            } else {
                uint16_t* D = static_cast<uint16_t*>(a.D);
                const uint16_t* res = static_cast<const uint16_t*>(a.residual);
                for (int c = 0; c < left; c++) {
                    const float r = res ? __builtin_bit_cast(float, (uint32_t)res[at + c] << 16) : 0.0f;
                    D[at + c] = (uint16_t)bf16x2_bits(res ? v[c] + r : v[c], 0.0f);
                }
            }
        }
        __syncthreads();       // the sums are read before the next chunk's are written
    }
}

constexpr int64_t RW_GROUPS = ((int64_t)1 << 32) / RW_THREADS;      // of a launch, fewer than this

// two workgroups share an expert's blocks of rows, should it have several: 200 rows
// of 128 experts, 2 x 1024 x 2048, in four of them 36 -> 25 us; spread evenly 89 both
static unsigned row_shares(const FusedArgs& f, int mb) { return f.expert_start && f.m > 16 * mb ? 2 : 1; }

// Experts have a workgroup for every 16 (gated) or 32 columns of each.
bool gemm_rows_fits(const FusedArgs& f) {
    const int64_t cols = f.gated ? 16 : 32;
    return !f.expert_start || (f.n + cols - 1) / cols * f.experts * row_shares(f, 1) < RW_GROUPS;
}

template <bool MX, bool GATED, int NB, int MB, int AHEAD, int WPE>
static hipError_t launch_one_rows(const FusedArgs& f, hipStream_t stream) {
    constexpr int COLS = GATED ? 8 * NB : 16 * NB;
    const int64_t gx = (f.n + COLS - 1) / COLS;
    int64_t gy = f.expert_start ? f.experts : (f.m + 16 * MB - 1) / (16 * MB);
    if (gy > 65535) gy = 65535;
    // a workgroup of one product goes round as many blocks of rows as are left
    if (!f.expert_start && gx * gy >= RW_GROUPS) gy = (RW_GROUPS - 1) / gx;
    RowsArgs args{f, act_of(f.act)};
    const unsigned gz = row_shares(f, MB);
    const dim3 grid((unsigned)gx, (unsigned)gy, gz), threads(RW_THREADS);
    if constexpr (MX) {
        const int64_t lds = (int64_t)scale_pitch((int)(f.k / 32)) * 16 * (NB + MB);
        if (lds <= SC_LIMIT && f.k > 0) {
            auto kern = gemm_rows_kernel<true, true, GATED, NB, MB, AHEAD, WPE>;
            // with the sums above the default launch limit: raised once per device; setting
            // it twice from racing threads is harmless
            if constexpr (RW_WAVES * NB * MB * 64 * (int)sizeof(v4f) + SC_LIMIT > 64 * 1024) {
                static std::atomic<uint64_t> configured{0};
                int dev = 0;
                hipError_t e = hipGetDevice(&dev);
                if (e != hipSuccess) return e;
                const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;
                if (!bit || !(configured.load(std::memory_order_acquire) & bit)) {
                    e = hipFuncSetAttribute(reinterpret_cast<const void*>(kern), hipFuncAttributeMaxDynamicSharedMemorySize, SC_LIMIT);
                    if (e != hipSuccess) return e;
                    configured.fetch_or(bit, std::memory_order_release);
                }
            }
            kern<<<grid, threads, (unsigned)lds, stream>>>(args);
            return hipGetLastError();
        }
    }
    gemm_rows_kernel<MX, false, GATED, NB, MB, AHEAD, WPE><<<grid, threads, 0, stream>>>(args);
    return hipGetLastError();
}

// NB, MB, AHEAD, WPE.  Up to 16 rows: gated, 2 x 11008 x 8192, one row: 35.9 us (5.0
// TB/s); the same with one column block less in flight or eight waves 40 to 65 us.
// Plain products of few column blocks (below 512 workgroups of 32 columns) take 16
// columns a workgroup and four steps in flight, wider ones 32 and one.  More rows than
// 16 come in blocks of 32 or 64, where registers allow two waves of a SIMD (one
// product only: experts come here with few rows on average, see gemm_fused.hip).
template <bool MX, bool GATED>
static hipError_t launch_rows(const FusedArgs& f, hipStream_t stream) {
    const int64_t rows = f.expert_start ? (f.m + f.experts - 1) / f.experts : f.m;   // of a product, on average
    if constexpr (GATED) {
        if (rows <= 16) return launch_one_rows<MX, true, 2, 1, 1, 4>(f, stream);
        if (rows <= 32) return launch_one_rows<MX, true, 2, 2, 2, 2>(f, stream);
        return launch_one_rows<MX, true, 2, 4, 2, 2>(f, stream);
    } else {
        if (rows > 32) return launch_one_rows<MX, false, 1, 4, 2, 2>(f, stream);
        if (rows > 16) return launch_one_rows<MX, false, 1, 2, 4, 2>(f, stream);
        const int64_t blocks = (f.n + 31) / 32 * (f.expert_start ? f.experts : 1);
        if (blocks < 512) return launch_one_rows<MX, false, 1, 1, 4, 4>(f, stream);
        return launch_one_rows<MX, false, 2, 1, 1, 4>(f, stream);
    }
}

hipError_t launch_gemm_rows(const FusedArgs& f, hipStream_t stream) {
    if (f.mx) return f.gated ? launch_rows<true, true>(f, stream) : launch_rows<true, false>(f, stream);
    return f.gated ? launch_rows<false, true>(f, stream) : launch_rows<false, false>(f, stream);
}

}  // namespace fp8g
