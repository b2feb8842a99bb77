// qk_norm_rope: per-head RMS norm of queries and keys and the position
// rotation, in one pass over the rows.
//
//   y = x * rsqrt(mean x^2 + eps) * w;   (y_a, y_b) -> (y_a c - y_b s, y_b c + y_a s)
//
// With r = 1 / sqrt(mean x^2 + eps) and p(e) the other element of e's pair,
//   out_e = r * (x_e C_e + x_p(e) S_e),   C_e = w_e c,  S_e = -/+ w_p(e) s
// (C_e = w_e, S_e = 0 behind rotary_dim), so a row needs two products an
// element once its token's C and S are there.  A workgroup works them out once
// for its tokens, for queries and for keys, in LDS, one element a thread: the
// look-ups (axis -> position -> cosine, sine) are a chain of three loads that
// would otherwise stand in front of every row.
//
// HBM-bound: every element is read and written once.  A row is held by L lanes
// (a power of two, 16 bytes a lane), so its sum of squares takes log2(L) lane
// exchanges.  Where a pair is (i, i + rotary_dim / 2), a lane loads its
// partner's 16 bytes a second time (they are in the cache that the row just
// passed through) instead of exchanging them over the lanes.  The loads of a
// row come before its store in the same wave, and a wave holds whole rows, so
// a row may be written in place.
//
// Measured: 8192 tokens x 72 heads x 128 bf16, three axes, 67 us, 4.6 TB/s (copies on
// this part reach 5.8); 411 us before C and S lay in LDS and rows were in
// flight while others are worked out.

#include "device_common.h"
#include "launch_block.h"

namespace fp8g {

typedef unsigned int v4u __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));

constexpr int QK_THREADS = 256;
constexpr int QK_AHEAD = 4;          // rows of a slot in flight
constexpr int QK_LDS = 16384;        // C and S of a workgroup's tokens: 16 bytes an element of head_dim

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

// How a launch is cut: `tokens` of a workgroup, all of their rows or, with row
// blocks, `part` rows of its one token.
struct QkPlan {
    int tokens, row_blocks, part;
};

template <bool F32, int L, bool INTERLEAVED>
__global__ __launch_bounds__(QK_THREADS) void qk_norm_rope_kernel(QkArgs a, QkPlan p) {
    using Row = QkRow<F32>;
    constexpr int VEC = Row::VEC, SLOTS = QK_THREADS / L;
    constexpr int64_t ESZ = F32 ? 4 : 2;
    extern __shared__ float coef[];            // [token][q: C, S; k: C, S][head_dim]
    const int D = a.head_dim, half = a.rotary_dim >> 1;
    const int tile = blockIdx.x / p.row_blocks, block = blockIdx.x - tile * p.row_blocks;
    const int64_t t0 = (int64_t)tile * p.tokens;
    const int tokens = (int)min((int64_t)p.tokens, a.tokens - t0);
    const int rows = a.q_heads + a.k_heads;
    const int first = block * p.part, last = min(rows, first + p.part);   // rows of each token
    const int slot = threadIdx.x / L, lane = threadIdx.x % L;
    const int total = tokens * (last - first);
    // the lane's 16 bytes of a row; lanes past the row's end repeat the last
    // ones and count for nothing
    const int chunks = D / VEC;
    const bool live = lane < chunks;
    const int e0 = (live ? lane : chunks - 1) * VEC;
    const int partner = INTERLEAVED || e0 >= a.rotary_dim ? e0 : (e0 >= half ? e0 - half : e0 + half);

    // a row's place, and the next one of the slot
    const int span = last - first, step_token = SLOTS / span, step_row = SLOTS % span;
    int token = slot / span, row = first + slot % span;
    auto next = [&] {
        row += step_row, token += step_token;
        if (row >= last) row -= span, token++;
    };
    v4u x[QK_AHEAD], y[QK_AHEAD];
    char* dst[QK_AHEAD];
    const float* cs[QK_AHEAD];
    int f = slot;
    auto load = [&] {
        int g = f;
#pragma unroll
        for (int u = 0; u < QK_AHEAD; u++, g += SLOTS) {
            if (g < total) {
                const bool is_k = row >= a.q_heads;
                const int h = is_k ? row - a.q_heads : row;
                const int64_t t = t0 + token;
                const char* src = static_cast<const char*>(is_k ? a.k : a.q) +
                                  (t * (is_k ? a.k_stride : a.q_stride) + (int64_t)h * D) * ESZ;
                dst[u] = static_cast<char*>(is_k ? a.k_out : a.q_out) +
                         (t * (is_k ? a.k_out_stride : a.q_out_stride) + (int64_t)h * D) * ESZ + e0 * ESZ;
                cs[u] = coef + (token * 4 + (is_k ? 2 : 0)) * D + e0;
                x[u] = *reinterpret_cast<const v4u*>(src + e0 * ESZ);
                if constexpr (!INTERLEAVED) y[u] = *reinterpret_cast<const v4u*>(src + partner * ESZ);
                next();
            }
        }
    };
    load();      // the first rows travel while C and S are worked out

    for (int i = threadIdx.x; i < tokens * D; i += QK_THREADS) {
        const int tok = i / D, e = i - tok * D;
        float c = 1.0f, s = 0.0f;
        int other = e;
        if (e < a.rotary_dim) {
            const bool second = INTERLEAVED ? (e & 1) : e >= half;
            const int pair = INTERLEAVED ? e >> 1 : (second ? e - half : e);
            other = INTERLEAVED ? e ^ 1 : (second ? e - half : e + half);
            const int ax = a.axes > 1 ? min(max(a.axis[pair], 0), a.axes - 1) : 0;
            const int pos = min(max(a.positions[(int64_t)ax * a.tokens + t0 + tok], 0), a.max_position - 1);
            const float* table = a.cos_sin + (int64_t)pos * a.rotary_dim + pair;
            c = table[0];
            s = second ? table[half] : -table[half];
        }
        float* dc = coef + tok * 4 * D + e;
        dc[0] = (a.q_weight ? a.q_weight[e] : 1.0f) * c;
        dc[D] = (a.q_weight ? a.q_weight[other] : 1.0f) * s;
        dc[2 * D] = (a.k_weight ? a.k_weight[e] : 1.0f) * c;
        dc[3 * D] = (a.k_weight ? a.k_weight[other] : 1.0f) * s;
    }
    __syncthreads();

    const float inv_dim = 1.0f / (float)D;
    for (; f < total; f += QK_AHEAD * SLOTS) {
        v4u xs[QK_AHEAD], ys[QK_AHEAD];
        char* ds[QK_AHEAD];
        const float* cc[QK_AHEAD];
#pragma unroll
        for (int u = 0; u < QK_AHEAD; u++) xs[u] = x[u], ys[u] = y[u], ds[u] = dst[u], cc[u] = cs[u];
        const int now = f;
        f += QK_AHEAD * SLOTS;
        load();
        f = now;
#pragma unroll
        for (int u = 0; u < QK_AHEAD; u++) {
            if (now + u * SLOTS >= total) continue;     // a slot's lanes stay together
            float v[VEC], w[VEC], o[VEC];
            Row::unpack(xs[u], v);
            if constexpr (!INTERLEAVED) Row::unpack(ys[u], w);
            float sum = 0.0f;
#pragma unroll
            for (int j = 0; j < VEC; j++) sum += v[j] * v[j];
            sum = group_sum<L>(live ? sum : 0.0f);
            const float r = 1.0f / __builtin_sqrtf(sum * inv_dim + a.eps);
#pragma unroll
            for (int j = 0; j < VEC; j++)
                o[j] = r * (v[j] * cc[u][j] + (INTERLEAVED ? v[j ^ 1] : w[j]) * cc[u][D + j]);
            if (live) *reinterpret_cast<v4u*>(ds[u]) = Row::pack(o);
        }
    }
}

// lanes of a row: a power of two, 16 bytes a lane
static int qk_lanes(const QkArgs& a, int f32) {
    const int bytes = a.head_dim * (f32 ? 4 : 2);
    return bytes <= 128 ? 8 : bytes <= 256 ? 16 : bytes <= 512 ? 32 : 64;
}

static QkPlan qk_plan(const QkArgs& a, int lanes, int64_t* blocks) {
    const int SLOTS = QK_THREADS / lanes;
    const int rows = a.q_heads + a.k_heads;
    QkPlan p;
    p.part = rows, p.row_blocks = 1;
    const int64_t passes = ((int64_t)a.tokens * rows + SLOTS - 1) / SLOTS;
    if (passes <= 2048) {
        // few rows: one pass of them a workgroup, over the whole chip
        p.tokens = rows < SLOTS ? SLOTS / rows : 1;
        p.row_blocks = (rows + SLOTS - 1) / SLOTS;
        p.part = (rows + p.row_blocks - 1) / p.row_blocks;
    } else {
        // many: about 16 passes a workgroup, at least 2048 workgroups
        int64_t each = passes / 2048;
        each = each > 16 ? 16 : each;
        p.tokens = (int)((each * SLOTS + rows - 1) / rows);
    }
    const int most = QK_LDS / (a.head_dim * 16);
    if (p.tokens > most) p.tokens = most;
    *blocks = ((int64_t)a.tokens + p.tokens - 1) / p.tokens * p.row_blocks;
    return p;
}

bool qk_norm_rope_fits(const QkArgs& a, int f32) {
    int64_t blocks;
    qk_plan(a, qk_lanes(a, f32), &blocks);
    return blocks <= most_blocks(QK_THREADS);
}

template <bool F32, int L>
static hipError_t launch_l(const QkArgs& a, hipStream_t stream) {
    int64_t grid;
    const QkPlan p = qk_plan(a, L, &grid);
    const unsigned lds = p.tokens * a.head_dim * 16;
    if (a.interleaved)
        qk_norm_rope_kernel<F32, L, true><<<dim3((unsigned)grid), dim3(QK_THREADS), lds, stream>>>(a, p);
    else
        qk_norm_rope_kernel<F32, L, false><<<dim3((unsigned)grid), dim3(QK_THREADS), lds, stream>>>(a, p);
    return hipGetLastError();
}

hipError_t launch_qk_norm_rope(const QkArgs& a, int f32, hipStream_t stream) {
    const int lanes = qk_lanes(a, f32);
    if (f32) {
        if (lanes == 8) return launch_l<true, 8>(a, stream);
        if (lanes == 16) return launch_l<true, 16>(a, stream);
        if (lanes == 32) return launch_l<true, 32>(a, stream);
        return launch_l<true, 64>(a, stream);
    }
    if (lanes == 8) return launch_l<false, 8>(a, stream);
    if (lanes == 16) return launch_l<false, 16>(a, stream);
    return launch_l<false, 32>(a, stream);
}

}  // namespace fp8g
