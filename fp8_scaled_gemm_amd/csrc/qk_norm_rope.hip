// qk_norm_rope: per-head RMS norm of queries and keys and the position
// rotation, in one pass over the rows.
//
//   y = x * rsqrt(mean x^2 + eps) * w;   (y_a, y_b) -> (y_a c - y_b s, y_b c + y_a s)
//
// HBM-bound: every element is read and written once.  One head row is held by
// L lanes (a power of two, 16 bytes a lane), so the sum of squares needs only
// log2(L) lane exchanges and no shared memory.  A slot of L lanes stays with
// one token and walks over its heads: the token's cosines and sines (per axis
// gathered, 2 loads a pair) then stay in registers for all of them.
//
// Where a pair is (i, i + rotary_dim / 2) the lane that holds i needs its
// partner's 16 bytes too; it loads them a second time (they hit the cache that
// the row just passed through) instead of exchanging them over the lanes.
// Both loads of a row come before its store in the same wave, so a row may be
// written in place.

#include "device_common.h"
#include "launch_block.h"

namespace fp8g {

typedef unsigned int v4u __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));

constexpr int QK_THREADS = 256;

template <bool F32>
struct QkRow {
    static constexpr int VEC = F32 ? 4 : 8;   // elements of 16 bytes
    static __device__ __forceinline__ void unpack(v4u r, float* f) {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            if constexpr (F32) {
                // the vector as a whole: a bit cast of one element of it reads element 0
                f[i] = __builtin_bit_cast(v4f, r)[i];
            } else {
                f[2 * i] = __builtin_bit_cast(float, r[i] << 16);
                f[2 * i + 1] = __builtin_bit_cast(float, r[i] & 0xFFFF0000u);
            }
        }
    }
    static __device__ __forceinline__ v4u pack(const float* f) {
        v4u r;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            if constexpr (F32)
                r[i] = __builtin_bit_cast(uint32_t, f[i]);
            else
                r[i] = bf16x2_bits(f[2 * i], f[2 * i + 1]);
        }
        return r;
    }
};

// Sum over aligned groups of L lanes, in every lane of the group.
template <int L>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int off = 1; off < L; off <<= 1) v += __shfl_xor(v, off, 64);
    return v;
}

template <bool F32, int L>
__global__ __launch_bounds__(QK_THREADS) void qk_norm_rope_kernel(QkArgs a, int tokens_per_wg, int row_blocks) {
    using Row = QkRow<F32>;
    constexpr int VEC = Row::VEC, SLOTS = QK_THREADS / L;
    const int rows = a.q_heads + a.k_heads;
    const int slot = threadIdx.x / L, lane = threadIdx.x % L;
    // a slot's token and first row; with several row blocks a token's rows are
    // dealt out over them
    const int tile = blockIdx.x / row_blocks, part = blockIdx.x - tile * row_blocks;
    int64_t t = tile;
    int row = part * SLOTS + slot, step = row_blocks * SLOTS;
    if (tokens_per_wg > 1) {
        const int sub = slot / rows;
        t = (int64_t)tile * tokens_per_wg + sub;
        row = sub < tokens_per_wg ? slot - sub * rows : rows;
        step = rows;
    }
    if (t >= a.tokens) row = rows;
    // the lane's 16 bytes of a row; lanes past the row's end repeat the last
    // ones and count for nothing
    const int chunks = a.head_dim / VEC;
    const bool live = lane < chunks;
    const int e0 = (live ? lane : chunks - 1) * VEC;
    const int half = a.rotary_dim >> 1;
    const bool turns = e0 < a.rotary_dim;
    const bool second = turns && !a.interleaved && e0 >= half;
    const int partner = a.interleaved || !turns ? e0 : (second ? e0 - half : e0 + half);
    // cosines and sines of the lane's pairs; sines with the sign of the term
    // that the partner adds.  Interleaved: VEC / 2 pairs, each twice.
    float c[VEC], s[VEC];
#pragma unroll
    for (int j = 0; j < VEC; j++) c[j] = 1.0f, s[j] = 0.0f;
    if (turns && row < rows) {
        const int i0 = a.interleaved ? e0 >> 1 : (second ? e0 - half : e0);
        if (a.axes == 1) {
            const int p = min(max(a.positions[t], 0), a.max_position - 1);
            const float* table = a.cos_sin + (int64_t)p * a.rotary_dim;
#pragma unroll
            for (int j = 0; j < VEC; j++) {
                const int i = i0 + (a.interleaved ? j >> 1 : j);
                c[j] = table[i];
                s[j] = table[half + i];
            }
        } else {
#pragma unroll
            for (int j = 0; j < VEC; j++) {
                const int i = i0 + (a.interleaved ? j >> 1 : j);
                const int ax = min(max(a.axis[i], 0), a.axes - 1);
                const int p = min(max(a.positions[(int64_t)ax * a.tokens + t], 0), a.max_position - 1);
                const float* table = a.cos_sin + (int64_t)p * a.rotary_dim;
                c[j] = table[i];
                s[j] = table[half + i];
            }
        }
#pragma unroll
        for (int j = 0; j < VEC; j++)
            if (a.interleaved ? !(j & 1) : !second) s[j] = -s[j];
    }
    const float inv_dim = 1.0f / (float)a.head_dim;
    for (; row < rows; row += step) {
        const bool is_k = row >= a.q_heads;
        const int h = is_k ? row - a.q_heads : row;
        const int64_t esz = F32 ? 4 : 2;
        const char* src = static_cast<const char*>(is_k ? a.k : a.q) +
                          (t * (is_k ? a.k_stride : a.q_stride) + (int64_t)h * a.head_dim) * esz;
        char* dst = static_cast<char*>(is_k ? a.k_out : a.q_out) +
                    (t * (is_k ? a.k_out_stride : a.q_out_stride) + (int64_t)h * a.head_dim) * esz;
        const float* w = is_k ? a.k_weight : a.q_weight;
        float x[VEC], y[VEC], wx[VEC], wy[VEC];
        Row::unpack(*reinterpret_cast<const v4u*>(src + e0 * esz), x);
        Row::unpack(*reinterpret_cast<const v4u*>(src + partner * esz), y);
#pragma unroll
        for (int j = 0; j < VEC; j++) {
            wx[j] = w ? w[e0 + j] : 1.0f;
            wy[j] = w ? w[partner + j] : 1.0f;
        }
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < VEC; j++) sum += x[j] * x[j];
        sum = group_sum<L>(live ? sum : 0.0f);
        const float r = 1.0f / __builtin_sqrtf(sum * inv_dim + a.eps);
        float o[VEC];
#pragma unroll
        for (int j = 0; j < VEC; j++) {
            const int jp = a.interleaved ? j ^ 1 : j;
            o[j] = x[j] * r * wx[j] * c[j] + (a.interleaved ? x[jp] * r * wx[jp] : y[j] * r * wy[j]) * s[j];
        }
        if (live) *reinterpret_cast<v4u*>(dst + e0 * esz) = Row::pack(o);
    }
}

template <bool F32, int L>
static hipError_t launch_l(const QkArgs& a, hipStream_t stream) {
    constexpr int SLOTS = QK_THREADS / L;
    const int rows = a.q_heads + a.k_heads;
    int tokens_per_wg = 1, row_blocks = 1;
    if (rows <= SLOTS) {
        tokens_per_wg = SLOTS / rows;
    } else {
        // few tokens: a row for every slot; many: up to 4 rows a slot, so that
        // the token's cosines and sines serve them all
        const int most = (rows + SLOTS - 1) / SLOTS;
        row_blocks = a.tokens >= 2048 ? (most + 3) / 4 : most;
    }
    const int64_t grid = ((int64_t)a.tokens + tokens_per_wg - 1) / tokens_per_wg * row_blocks;
    qk_norm_rope_kernel<F32, L><<<dim3((unsigned)grid), dim3(QK_THREADS), 0, stream>>>(a, tokens_per_wg, row_blocks);
    return hipGetLastError();
}

hipError_t launch_qk_norm_rope(const QkArgs& a, int f32, hipStream_t stream) {
    const int bytes = a.head_dim * (f32 ? 4 : 2);
    if (f32) {
        if (bytes <= 128) return launch_l<true, 8>(a, stream);
        if (bytes <= 256) return launch_l<true, 16>(a, stream);
        if (bytes <= 512) return launch_l<true, 32>(a, stream);
        return launch_l<true, 64>(a, stream);
    }
    if (bytes <= 128) return launch_l<false, 8>(a, stream);
    if (bytes <= 256) return launch_l<false, 16>(a, stream);
    return launch_l<false, 32>(a, stream);
}

}  // namespace fp8g
