// moe_combine: the routed rows back to their tokens.
//
//   out[t] = round( residual[t] + sum_j w[t, j] y[slot[t, j]] )
//
// HBM-bound: every routed row is read once, every token's row written once.  A
// wave holds 64 x 16 bytes of a token's row; its slots and weights are the
// wave's own, read once, and four rows are in flight together.  8192 tokens x 8 rows
// of 4096 bf16, 671 MB: 129 us (5.2 TB/s).

#include "launch_ffn.h"
#include "rows16.h"

namespace fp8g {

constexpr int CB_THREADS = 256;
constexpr int CB_AHEAD = 4;          // rows in flight

template <bool F32>
__global__ __launch_bounds__(CB_THREADS) void combine_rows(CombineArgs a) {
    using R = Row16<F32>;
    constexpr int VEC = R::VEC;
    const int lane = threadIdx.x & 63;
    const int nv = a.width / VEC, parts = (nv + 63) / 64;      // waves a row
    const int64_t wave = (int64_t)blockIdx.x * (CB_THREADS / 64) + (threadIdx.x >> 6);
    const int64_t t = wave / parts;
    const int v = (int)(wave - t * parts) * 64 + lane;
    if (t >= a.tokens || v >= nv) return;
    const v4u* y = reinterpret_cast<const v4u*>(a.y);
    float acc[VEC] = {};
    if (a.residual) R::unpack(reinterpret_cast<const v4u*>(a.residual)[t * nv + v], acc);
    const int32_t* slots = a.slots + t * a.top_k;
    const float* weights = a.weights + t * a.top_k;
    for (int j = 0; j < a.top_k; j += CB_AHEAD) {
        v4u r[CB_AHEAD];
        float w[CB_AHEAD];
#pragma unroll
        for (int i = 0; i < CB_AHEAD; i++) {
            const bool in = j + i < a.top_k;
            const int s = in ? slots[j + i] : -1;
            const bool ok = s >= 0 && s < a.y_rows;
            w[i] = ok ? weights[j + i] : 0.0f;
            r[i] = ok ? y[(int64_t)s * nv + v] : (v4u){0, 0, 0, 0};
        }
#pragma unroll
        for (int i = 0; i < CB_AHEAD; i++) {
            float f[VEC];
            R::unpack(r[i], f);
#pragma unroll
            for (int c = 0; c < VEC; c++) acc[c] = __builtin_fmaf(w[i], f[c], acc[c]);
        }
    }
    reinterpret_cast<v4u*>(a.out)[t * nv + v] = R::pack(acc);
}

static int64_t combine_blocks(const CombineArgs& a, int f32) {
    const int64_t nv = a.width / (f32 ? 4 : 8), parts = (nv + 63) / 64;
    return (a.tokens * parts + CB_THREADS / 64 - 1) / (CB_THREADS / 64);
}
bool moe_combine_fits(const CombineArgs& a, int f32) { return combine_blocks(a, f32) < ((int64_t)1 << 32) / CB_THREADS; }

hipError_t launch_moe_combine(const CombineArgs& a, int f32, hipStream_t stream) {
    const dim3 grid((unsigned)combine_blocks(a, f32)), threads(CB_THREADS);
    if (f32) combine_rows<true><<<grid, threads, 0, stream>>>(a);
    else combine_rows<false><<<grid, threads, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace fp8g
