// moe_route: the experts of every token, and the routed rows sorted by expert.
//
//   p = softmax or sigmoid of the logits, choice = p + bias; groups by the sum
//   of their largest choices; the top_k of the kept groups' experts
//
// A wave scores a token: lane L holds the experts L, L + 64, ...  Scores and sums
// are fp64, so that two experts change places only where their choices agree to
// 2^-50 or so: an fp32 choice would hang on the order of a sum and on the
// exponential at hand.  Each of the top_k rounds takes the wave's largest
// choice, and among equals the lowest expert.
//
// The rows are sorted by counting, stably and without order-dependent atomics:
// a workgroup counts the experts of its run of tokens (integer additions in
// LDS); the counts are summed over the workgroups, expert by expert; and each
// workgroup then places its tokens' rows behind those of the workgroups before
// it, a row's rank within the run being the number of rows of the same expert
// ahead of it.

#include "launch_ffn.h"
#include "rows16.h"

namespace fp8g {

constexpr int RT_THREADS = 256, RT_WAVES = RT_THREADS / 64;
constexpr int RT_MAX_EXPERTS = 1024;
constexpr int RT_ENTRIES = 512;          // routed rows of a workgroup's run, at most

struct RoutePlan {
    int chunk, blocks;                   // tokens of a run, runs
};
static RoutePlan route_plan(const RouteArgs& a) {
    RoutePlan p;
    p.chunk = RT_WAVES;
    while (p.chunk < 64 && (int64_t)p.chunk * 256 < a.tokens && 2 * p.chunk * a.top_k <= RT_ENTRIES) p.chunk *= 2;
    p.blocks = (a.tokens + p.chunk - 1) / p.chunk;
    return p;
}

__device__ __forceinline__ double wave_max_f64(double v) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) v = __builtin_fmax(v, __shfl_xor(v, off, 64));
    return v;
}
__device__ __forceinline__ double wave_sum_f64(double v) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
    return v;
}

// The token's experts and weights: in lane j < top_k the j-th.
template <bool F32, int VPL>
__device__ __forceinline__ void route_token(const RouteArgs& a, int64_t t, int& id, float& weight) {
    const int lane = threadIdx.x & 63, E = a.experts;
    const double NEG = -__builtin_inf();
    double p[VPL], key[VPL];
    bool there[VPL];
    double most = NEG;
#pragma unroll
    for (int i = 0; i < VPL; i++) {
        const int e = lane + 64 * i;
        float x = -__builtin_inff();
        if (e < E) {
            if constexpr (F32) x = static_cast<const float*>(a.logits)[t * E + e];
            else x = __builtin_bit_cast(float, (uint32_t)static_cast<const uint16_t*>(a.logits)[t * E + e] << 16);
        }
        there[i] = x > -__builtin_inff();                 // NaN: not there
        key[i] = there[i] ? (double)x + 0.0 : NEG;        // -0 as +0
        most = __builtin_fmax(most, key[i]);
    }
    if (a.sigmoid) {
#pragma unroll
        for (int i = 0; i < VPL; i++) p[i] = there[i] ? 1.0 / (1.0 + exp(-key[i])) : 0.0;
    } else {
        most = wave_max_f64(most);
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < VPL; i++) {
            // the largest itself without a difference, which is NaN between infinities
            p[i] = there[i] ? (key[i] == most ? 1.0 : exp(key[i] - most)) : 0.0;
            sum += p[i];
        }
        sum = wave_sum_f64(sum);
#pragma unroll
        for (int i = 0; i < VPL; i++) p[i] = sum > 0.0 ? p[i] / sum : 0.0;
    }
    if (a.bias) {
#pragma unroll
        for (int i = 0; i < VPL; i++) {
            const int e = lane + 64 * i;
            if (there[i]) key[i] = p[i] + (double)a.bias[e];
            there[i] = there[i] && key[i] > NEG;          // a bias of -inf or NaN: not there
        }
    }
    if (a.groups > 1) {
        const int width = E / a.groups;
        double mine = NEG;                                // lane q: group q's value
        for (int q = 0; q < a.groups; q++) {
            double top = NEG, v[VPL];
#pragma unroll
            for (int i = 0; i < VPL; i++) {
                const int e = lane + 64 * i;
                v[i] = there[i] && e / width == q ? (a.bias ? key[i] : p[i]) : NEG;
                top = __builtin_fmax(top, v[i]);
            }
            top = wave_max_f64(top);
            double value = top;
            if (a.group_top == 2) {
                bool gone = false;                        // one of the largest taken out
                double second = NEG;
#pragma unroll
                for (int i = 0; i < VPL; i++) {
                    const uint64_t b = __ballot(v[i] == top);
                    if (!gone && b) {
                        if (lane == __builtin_ctzll(b)) v[i] = NEG;
                        gone = true;
                    }
                    second = __builtin_fmax(second, v[i]);
                }
                value = top + wave_max_f64(second);
            }
            if (lane == q) mine = value;
        }
        int rank = 0;
        for (int q = 0; q < a.groups; q++) {
            const double other = __shfl(mine, q, 64);
            rank += other > mine || (other == mine && q < lane) ? 1 : 0;
        }
        const uint64_t kept = __ballot(lane < a.groups && rank < a.top_groups);
#pragma unroll
        for (int i = 0; i < VPL; i++) {
            const int e = lane + 64 * i;
            there[i] = there[i] && ((kept >> (e / width)) & 1);
        }
    }
    id = -1;
    double share = 0.0;
    for (int j = 0; j < a.top_k; j++) {
        double top = NEG;
#pragma unroll
        for (int i = 0; i < VPL; i++) top = __builtin_fmax(top, there[i] ? key[i] : NEG);
        top = wave_max_f64(top);
        bool found = false;
#pragma unroll
        for (int i = 0; i < VPL; i++) {
            const uint64_t b = __ballot(there[i] && key[i] == top);
            if (!found && b) {
                const int from = __builtin_ctzll(b);
                const double w = __shfl(p[i], from, 64);
                if (lane == j) id = from + 64 * i, share = w;
                if (lane == from) there[i] = false;
                found = true;
            }
        }
        if (!found) break;
    }
    if (a.renormalize) {
        const double sum = wave_sum_f64(share);
        share = sum > 0.0 ? share / sum : 0.0;
    }
    weight = (float)(share * (double)a.scale);
}

// Experts and weights of a run of tokens, and how many rows each expert gets of it.
template <bool F32, int VPL>
__global__ __launch_bounds__(RT_THREADS) void route_tokens(RouteArgs a, int chunk) {
    __shared__ int count[RT_MAX_EXPERTS];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    for (int e = tid; e < a.experts; e += RT_THREADS) count[e] = 0;
    __syncthreads();
    const int64_t first = (int64_t)blockIdx.x * chunk;
    for (int u = wave; u < chunk && first + u < a.tokens; u += RT_WAVES) {
        const int64_t t = first + u;
        int id;
        float w;
        route_token<F32, VPL>(a, t, id, w);
        if (lane < a.top_k) {
            a.ids[t * a.top_k + lane] = id;
            a.weights[t * a.top_k + lane] = w;
            if (id >= 0) atomicAdd(&count[id], 1);
        }
    }
    __syncthreads();
    for (int e = tid; e < a.experts; e += RT_THREADS) a.workspace[(int64_t)blockIdx.x * a.experts + e] = count[e];
}

// Counts of each run -> rows of the runs before it, expert by expert, and the totals.
__global__ __launch_bounds__(RT_THREADS) void route_counts(RouteArgs a, int blocks) {
    const int lane = threadIdx.x & 63, e = (int)blockIdx.x * RT_WAVES + (threadIdx.x >> 6);
    if (e >= a.experts) return;
    int before = 0;
    for (int b0 = 0; b0 < blocks; b0 += 64) {
        const int b = b0 + lane;
        const int own = b < blocks ? a.workspace[(int64_t)b * a.experts + e] : 0;
        int sum = own;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const int v = __shfl_up(sum, off, 64);
            if (lane >= off) sum += v;
        }
        if (b < blocks) a.workspace[(int64_t)b * a.experts + e] = before + sum - own;
        before += __shfl(sum, 63, 64);
    }
    if (lane == 0) a.workspace[(int64_t)blocks * a.experts + e] = before;
}

// A run's rows to their slots.
__global__ __launch_bounds__(RT_THREADS) void route_place(RouteArgs a, int chunk, int blocks) {
    __shared__ int base[RT_MAX_EXPERTS + 1];              // an expert's first slot, then this run's
    __shared__ int part[RT_THREADS];
    __shared__ int ids[RT_ENTRIES];
    const int tid = threadIdx.x, E = a.experts;
    constexpr int PER = RT_MAX_EXPERTS / RT_THREADS;
    int own[PER], sum = 0;
#pragma unroll
    for (int i = 0; i < PER; i++) {
        const int e = tid * PER + i;
        own[i] = e < E ? a.workspace[(int64_t)blocks * E + e] : 0;
        sum += own[i];
    }
    part[tid] = sum;
    __syncthreads();
    for (int off = 1; off < RT_THREADS; off <<= 1) {
        const int v = tid >= off ? part[tid - off] : 0;
        __syncthreads();
        part[tid] += v;
        __syncthreads();
    }
    int at = part[tid] - sum;
#pragma unroll
    for (int i = 0; i < PER; i++) {
        const int e = tid * PER + i;
        if (e < E) {
            base[e] = at;
            if (blockIdx.x == 0) a.expert_start[e] = at;
        }
        at += own[i];
    }
    const int total = part[RT_THREADS - 1];
    if (blockIdx.x == 0 && tid == 0) a.expert_start[E] = total;
    if (blocks == 0) return;                              // no token at all
    const int64_t first = (int64_t)blockIdx.x * chunk * a.top_k;
    const int entries = (int)min((int64_t)chunk * a.top_k, (int64_t)a.tokens * a.top_k - first);
    for (int i = tid; i < entries; i += RT_THREADS) ids[i] = a.ids[first + i];
    __syncthreads();
    for (int e = tid; e < E; e += RT_THREADS) base[e] += a.workspace[(int64_t)blockIdx.x * E + e];
    __syncthreads();
    for (int i = tid; i < entries; i += RT_THREADS) {
        const int id = ids[i];
        int slot = -1;
        if (id >= 0) {
            int rank = 0;
            for (int j = 0; j < i; j++) rank += ids[j] == id ? 1 : 0;
            slot = base[id] + rank;
            a.rows[slot] = (int)((first + i) / a.top_k);
        }
        a.slots[first + i] = slot;
        if (first + i >= total) a.rows[first + i] = -1;   // behind the last expert's
    }
}

int64_t moe_route_bytes(const RouteArgs& a) { return ((int64_t)route_plan(a).blocks + 1) * a.experts * 4; }

template <bool F32>
static void queue_tokens(const RouteArgs& a, const RoutePlan& p, hipStream_t stream) {
    const dim3 grid((unsigned)p.blocks), threads(RT_THREADS);
    if (a.experts <= 64) route_tokens<F32, 1><<<grid, threads, 0, stream>>>(a, p.chunk);
    else if (a.experts <= 128) route_tokens<F32, 2><<<grid, threads, 0, stream>>>(a, p.chunk);
    else if (a.experts <= 256) route_tokens<F32, 4><<<grid, threads, 0, stream>>>(a, p.chunk);
    else if (a.experts <= 512) route_tokens<F32, 8><<<grid, threads, 0, stream>>>(a, p.chunk);
    else route_tokens<F32, 16><<<grid, threads, 0, stream>>>(a, p.chunk);
}

hipError_t launch_moe_route(const RouteArgs& a, int f32, hipStream_t stream) {
    const RoutePlan p = route_plan(a);
    if (p.blocks > 0) {
        if (f32) queue_tokens<true>(a, p, stream);
        else queue_tokens<false>(a, p, stream);
    }
    route_counts<<<dim3((unsigned)((a.experts + RT_WAVES - 1) / RT_WAVES)), dim3(RT_THREADS), 0, stream>>>(a, p.blocks);
    route_place<<<dim3((unsigned)(p.blocks ? p.blocks : 1)), dim3(RT_THREADS), 0, stream>>>(a, p.chunk, p.blocks);
    return hipGetLastError();
}

}  // namespace fp8g
