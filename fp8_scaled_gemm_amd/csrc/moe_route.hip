// moe_route: the experts of every token, and the routed rows sorted by expert.
//
//   p = softmax or sigmoid of the logits, choice = p + bias; groups by the sum
//   of their largest choices; the top_k of the kept groups' experts
//
// A wave scores a token: lane L holds the experts L VPL .. L VPL + VPL - 1, and
// each of the top_k rounds takes the wave's largest choice, among equals the
// lowest expert.  Choices are defined in fp64, so that the ids do not hang on
// the rounding of an exponential or a sum.  They are looked at in fp32 first: the
// logits themselves are exact there, and where a choice is p + bias, or groups
// are compared, every decision of the token is checked to be wider than the fp32
// error (RT_MARGIN); a token with a closer one (about one in a thousand) is gone
// through again in fp64.  Weights always come from fp64.
//
// Bound by the vector instructions of a token (680 of them, most in the rounds, each
// of which waits for the one before), not by its bytes; a run of tokens has 16
// waves, four on a SIMD.  16384 tokens, 8 of 256 experts in 8 groups, sigmoid with
// bias: 34 us, and 10 us for the order; without groups 27 us in all; one token 4.3 us.
//
// The rows are sorted by counting, stably and with no result that hangs on an
// order: a run of at most 64 tokens sets bit t of its experts' 64-bit masks in
// LDS for its token t, so a mask's bits are the run's rows of the expert, in
// order, and a row's rank is the number of bits below its own.  The runs' counts
// are summed expert by expert, and each run places its rows behind those of the
// runs before it.  Up to RT_SMALL tokens one workgroup does all of it in one launch.

#include "launch_ffn.h"
#include "wave_ops.h"

namespace fp8g {

// waves of a run's workgroup: 16, and 8 where a lane holds more experts than 128
// registers do
constexpr int rt_waves(int vpl) { return vpl <= 4 ? 16 : 8; }
constexpr int RT_PLACE = 256;            // threads that place a run's rows
constexpr int RT_MAX_EXPERTS = 1024;
constexpr int RT_RUN = 64;               // tokens of a run, at most: bits of a mask
// one workgroup for all: 24 tokens of 256 experts in groups, 12.2 us against 13.2 us
// in two launches; 32 tokens 15.8 against 13.1, and of 64 experts 8.2 against 8.9
constexpr int RT_SMALL = 24;
constexpr int RT_SUM_RUNS = 64;          // runs whose counts the placing workgroups sum by themselves
// fp32 choices: p from the hardware's exponential and reciprocal (one ulp each, the
// argument's rounding times an exponent of at most 88 p) and a sum of 1024
// terms is within 2^-20 of p's range [0, 1]; the bias adds half an ulp of the
// choice, a group's sum twice all of that, by the size of its terms: biases of both
// signs may leave a small sum of large ones.
constexpr float RT_MARGIN = 1.0f / (1 << 18);

__device__ __forceinline__ float exp_of(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504f); }
__device__ __forceinline__ double exp_of(double x) { return exp(x); }
__device__ __forceinline__ float inverse(float x) { return __builtin_amdgcn_rcpf(x); }
__device__ __forceinline__ double inverse(double x) { return 1.0 / x; }

// A lane's experts in falling order (VPL <= 4), among equals the lowest first;
// byte i of `order` is the place of the i-th.
template <class R, int VPL>
__device__ __forceinline__ void sort_lane(R (&key)[VPL], uint32_t& order) {
    order = 0x03020100u;
    auto step = [&](int i, int j) __attribute__((always_inline)) {      // i < j
        const uint32_t a = (order >> (8 * i)) & 0xFFu, b = (order >> (8 * j)) & 0xFFu;
        const bool turn = key[j] > key[i] || (key[j] == key[i] && b < a);
        const R u = key[i], v = key[j];
        key[i] = turn ? v : u, key[j] = turn ? u : v;
        const uint32_t both = (a ^ b) << (8 * i) | (a ^ b) << (8 * j);
        order = turn ? order ^ both : order;
    };
    if constexpr (VPL == 2) {
        step(0, 1);
    } else if constexpr (VPL == 4) {
        step(0, 1), step(2, 3), step(0, 2), step(1, 3), step(1, 2);
    }
}

// The token's experts: in lane at + j, j < top_k, the j-th; lanes keep what ids
// holds where there is none.  False: two of them, or two groups, are too close for
// R = float to tell.  x, bias: the lane's experts (-inf behind the last one).
template <class R, int VPL>
__device__ __forceinline__ bool choose(const RouteArgs& a, const float (&x)[VPL], const float (&bias)[VPL], int to, int& ids) {
    const int lane = threadIdx.x & 63, E = a.experts;
    const R NEG = -(R)__builtin_inff();
    const bool exact = sizeof(R) == 8;
    R p[VPL], key[VPL];                                   // NEG: not available
    const bool scored = a.bias != nullptr || a.groups > 1;
#pragma unroll
    for (int i = 0; i < VPL; i++) {
        key[i] = x[i] > -__builtin_inff() ? (R)x[i] + (R)0 : NEG;      // NaN: not there; -0 as +0
        p[i] = (R)0;
    }
    if (scored) {
        if (a.sigmoid) {
#pragma unroll
            for (int i = 0; i < VPL; i++) p[i] = inverse((R)1 + exp_of(-key[i]));
        } else {
            R most = NEG, sum = (R)0;
#pragma unroll
            for (int i = 0; i < VPL; i++) most = larger(most, key[i]);
            most = wave_most(most);
#pragma unroll
            for (int i = 0; i < VPL; i++) {
                // the largest itself without a difference, which is NaN between infinities
                p[i] = key[i] == NEG ? (R)0 : key[i] == most ? (R)1 : exp_of(key[i] - most);
                sum += p[i];
            }
            sum = wave_total(sum);
            const R part = sum > (R)0 ? (R)1 / sum : (R)0;
#pragma unroll
            for (int i = 0; i < VPL; i++) p[i] = exact ? (sum > (R)0 ? p[i] / sum : (R)0) : p[i] * part;
        }
    }
    if (a.bias) {
#pragma unroll
        for (int i = 0; i < VPL; i++) {
            const R c = p[i] + (R)bias[i];
            key[i] = key[i] > NEG && c > NEG ? c : NEG;   // a bias of -inf or NaN: not there
        }
    }
    bool clear = true;                                    // every decision so far is wider than the error
    if (a.groups > 1) {
        const int width = E / a.groups, lanes = width / VPL;
        R mine = NEG;                                     // lane q: group q's value
        R size = (R)1;                                    // of the values' largest term (p is at most 1)
        const auto term = [&](R v) __attribute__((always_inline)) { return v > NEG ? larger(v, -v) : (R)0; };
        if (width % VPL == 0 && (lanes & (lanes - 1)) == 0) {
            // a group is `lanes` neighbouring lanes: all groups at once
            R top = NEG, second = NEG;
#pragma unroll
            for (int i = 0; i < VPL; i++) {
                const R v = key[i] > NEG ? (a.bias ? key[i] : p[i]) : NEG;
                second = larger(second, v < top ? v : top);
                top = larger(top, v);
            }
            for (int off = 1; off < lanes; off <<= 1) {
                const R t = __shfl_xor(top, off, 64), u = __shfl_xor(second, off, 64);
                second = larger(larger(second, u), t < top ? t : top);
                top = larger(top, t);
            }
            // behind all others without a second one, whatever the first (+inf - inf is NaN)
            const R value = a.group_top == 1 ? top : second > NEG ? top + second : NEG;
            if (!exact && a.bias) size = wave_most(larger(term(top), a.group_top == 2 ? term(second) : (R)0));
            mine = __shfl(value, lane * lanes & 63, 64);
            if (lane >= a.groups) mine = NEG;
        } else {
            for (int q = 0; q < a.groups; q++) {
                R top = NEG, v[VPL];
#pragma unroll
                for (int i = 0; i < VPL; i++) {
                    const int e = lane * VPL + i;
                    v[i] = key[i] > NEG && e / width == q ? (a.bias ? key[i] : p[i]) : NEG;
                    top = larger(top, v[i]);
                }
                const R best = wave_most(top);
                R value = best;
                if (a.group_top == 2) {
                    // one of the largest taken out: the lowest lane's first
                    const uint64_t b = __ballot(top == best);
                    bool gone = lane != __builtin_ctzll(b);
                    R second = NEG;
#pragma unroll
                    for (int i = 0; i < VPL; i++) {
                        const bool out = !gone && v[i] == best;
                        second = larger(second, out ? NEG : v[i]);
                        gone = gone || out;
                    }
                    second = wave_most(second);
                    value = second > NEG ? best + second : NEG;
                    size = larger(size, term(second));
                }
                size = larger(size, term(best));
                if (lane == q) mine = value;
            }
        }
        int rank = 0;
        for (int q = 0; q < a.groups; q++) {
            const R other = from_lane(mine, q);
            rank += other > mine || (other == mine && q < lane) ? 1 : 0;
        }
        const bool in = lane < a.groups && rank < a.top_groups;
        const uint64_t kept = __ballot(in);
        if (!exact && a.top_groups < a.groups) {
            const R last = -wave_most(in ? -mine : NEG), next = wave_most(lane < a.groups && !in ? mine : NEG);
            // groups without enough experts (NEG) are behind all others for sure
            clear = next == NEG || last - next > (R)RT_MARGIN * ((R)1 + size);
        }
#pragma unroll
        for (int i = 0; i < VPL; i++) {
            const int e = lane * VPL + i;
            if (e >= E || !((kept >> (e / width)) & 1)) key[i] = NEG;
        }
    }
    const int rounds = !exact && a.bias ? a.top_k + 1 : a.top_k;       // one more: the gap behind the last
    R tops = NEG;                                         // lane j: the j-th choice
    uint32_t order;
    if constexpr (VPL <= 4) sort_lane<R, VPL>(key, order);
    for (int j = 0; j < rounds; j++) {
        R own = key[0];
        if constexpr (VPL > 4) {
#pragma unroll
            for (int i = 1; i < VPL; i++) own = larger(own, key[i]);
        }
        const R top = wave_most(own);
        if (!(top > NEG)) break;
        const int from = __builtin_ctzll(__ballot(own == top));
        int at = 0;
        if constexpr (VPL <= 4) {
            at = __builtin_amdgcn_readlane((int)order, from) & 0xFF;
            if (lane == from) {
#pragma unroll
                for (int i = 0; i + 1 < VPL; i++) key[i] = key[i + 1];
                key[VPL - 1] = NEG;
                order >>= 8;
            }
        } else {
            bool gone = lane != from;
#pragma unroll
            for (int i = 0; i < VPL; i++) {
                const bool out = !gone && key[i] == top;
                key[i] = out ? NEG : key[i];
                at = out ? i : at;
                gone = gone || out;
            }
            at = __builtin_amdgcn_readlane(at, from);
        }
        if (j < a.top_k) ids = lane == to + j ? from * VPL + at : ids;
        if (!exact && a.bias) tops = lane == j ? top : tops;
    }
    if (!exact && a.bias) {
        const R next = __shfl_down(tops, 1, 64);
        const bool close = next > NEG && !(tops - next > (R)RT_MARGIN * ((R)1 + larger(tops, -tops)));
        clear = clear && __ballot(lane < a.top_k && close) == 0;
    }
    return clear;
}

template <bool F32>
__device__ __forceinline__ float logit_at(const RouteArgs& a, int64_t i) {
    if constexpr (F32) return static_cast<const float*>(a.logits)[i];
    else return __builtin_bit_cast(float, (uint32_t)static_cast<const uint16_t*>(a.logits)[i] << 16);
}

// What a lane reads of a token's row: its VPL experts' logits, all loads at once.
template <bool F32, int VPL>
__device__ __forceinline__ void load_logits(const RouteArgs& a, int64_t t, float (&x)[VPL]) {
    const int lane = threadIdx.x & 63, E = a.experts;
#pragma unroll
    for (int i = 0; i < VPL; i++) x[i] = logit_at<F32>(a, t * E + min(lane * VPL + i, E - 1));
}
template <int VPL>
__device__ __forceinline__ void load_bias(const RouteArgs& a, float (&bias)[VPL]) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < VPL; i++) bias[i] = a.bias ? a.bias[min(lane * VPL + i, a.experts - 1)] : 0.0f;
}

// Over aligned groups of `width` lanes (a power of two), in every lane.
__device__ __forceinline__ double group_most(double v, int width) {
    for (int off = 1; off < width; off <<= 1) v = larger(v, __shfl_xor(v, off, 64));
    return v;
}
__device__ __forceinline__ double group_total(double v, int width) {
    for (int off = 1; off < width; off <<= 1) v += __shfl_xor(v, off, 64);
    return v;
}

// Tokens first + wave, first + wave + WAVES, ... below `end` of this workgroup's
// run.  The next one's logits are on their way while one is worked out.  The
// weights, in fp64, are worked out for as many tokens at once as fit a wave, a
// token in `wide` lanes, the power of two that holds top_k.
template <bool F32, int VPL>
__device__ __forceinline__ void route_run(const RouteArgs& a, int64_t first, int end, int wide, unsigned long long* mask) {
    constexpr int WAVES = rt_waves(VPL);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const double NEG = -__builtin_inf();
    if (wave >= end) return;
    float bias[VPL], next[VPL];
    load_bias<VPL>(a, bias);
    load_logits<F32, VPL>(a, first + wave, next);
    for (int u0 = wave; u0 < end; u0 += WAVES * (64 / wide)) {
        int id = -1;
        float logit = 0.0f;
        double most = NEG, total = 0.0;                   // of the softmax over all experts, where it is needed
        for (int at = 0; at < 64; at += wide) {
            const int u = u0 + WAVES * (at / wide);
            if (u >= end) break;
            float x[VPL];
#pragma unroll
            for (int i = 0; i < VPL; i++) x[i] = lane * VPL + i < a.experts ? next[i] : -__builtin_inff();
            load_logits<F32, VPL>(a, first + min(u + WAVES, end - 1), next);
            const bool here = lane >= at && lane < at + wide;
            if (!choose<float, VPL>(a, x, bias, at, id)) {
                id = here ? -1 : id;                      // fp64 may find fewer experts than fp32 did
                choose<double, VPL>(a, x, bias, at, id);
            }
#pragma unroll
            for (int i = 0; i < VPL; i++) {
                const float v = __shfl(x[i], id >= 0 ? id / VPL : 0, 64);
                logit = here && id >= 0 && id % VPL == i ? v : logit;
            }
            if (!a.sigmoid && !a.renormalize) {
                double m = NEG, sum = 0.0;
#pragma unroll
                for (int i = 0; i < VPL; i++) m = larger(m, x[i] > -__builtin_inff() ? (double)x[i] : NEG);
                m = wave_most(m);
#pragma unroll
                for (int i = 0; i < VPL; i++)
                    if (x[i] > -__builtin_inff()) sum += (double)x[i] == m ? 1.0 : exp((double)x[i] - m);
                sum = wave_total(sum);
                most = here ? m : most, total = here ? sum : total;
            }
        }
        const double own = id >= 0 ? (double)logit : NEG;
        double share;
        if (a.sigmoid) {
            share = id >= 0 ? 1.0 / (1.0 + exp(-own)) : 0.0;
        } else {
            if (a.renormalize) most = group_most(own, wide);
            // the largest itself without a difference, which is NaN between infinities
            share = id < 0 ? 0.0 : own == most ? 1.0 : exp(own - most);
        }
        if (a.renormalize) total = group_total(share, wide);
        if (a.renormalize || !a.sigmoid) share = total > 0.0 ? share / total : 0.0;
        const int u = u0 + WAVES * (lane / wide), j = lane & (wide - 1);
        if (u < end && j < a.top_k) {
            const int64_t i = (first + u) * a.top_k + j;
            a.ids[i] = id;
            a.weights[i] = (float)(share * (double)a.scale);
            if (id >= 0) atomicOr(&mask[id], 1ull << u);
        }
    }
}

// Sums over the threads before, of `threads` threads; part: one word a thread.
template <int THREADS>
__device__ __forceinline__ int before_threads(int own, int* part, int& total) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int sum = own;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const int v = __shfl_up(sum, off, 64);
        if (lane >= off) sum += v;
    }
    if (lane == 63) part[wave] = sum;
    __syncthreads();
    int ahead = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 64; w++) {
        if (w < wave) ahead += part[w];
        total += part[w];
    }
    return ahead + sum - own;
}

// A run's row i (of token i / top_k) to its slot; base: the experts' first slots for this run.
__device__ __forceinline__ void place(const RouteArgs& a, int64_t first, int i, int id, const int* base,
                                      const unsigned long long* mask, int total) {
    int slot = -1;
    if (id >= 0) {
        const int t = i / a.top_k;
        slot = base[id] + __popcll(mask[id] & ((1ull << t) - 1));
        a.rows[slot] = (int)((first + i) / a.top_k);
    }
    a.slots[first + i] = slot;
    if (first + i >= total) a.rows[first + i] = -1;       // behind the last expert's
}

// Experts and weights of a run of tokens, and how many rows each expert gets of it.
template <bool F32, int VPL>
__global__ __launch_bounds__(64 * rt_waves(VPL)) void route_tokens(RouteArgs a, int run, int wide) {
    constexpr int THREADS = 64 * rt_waves(VPL);
    __shared__ unsigned long long mask[RT_MAX_EXPERTS];
    const int tid = threadIdx.x;
    for (int e = tid; e < a.experts; e += THREADS) mask[e] = 0;
    __syncthreads();
    const int64_t first = (int64_t)blockIdx.x * run;
    route_run<F32, VPL>(a, first, (int)min((int64_t)run, a.tokens - first), wide, mask);
    __syncthreads();
    for (int e = tid; e < a.experts; e += THREADS) a.workspace[(int64_t)blockIdx.x * a.experts + e] = __popcll(mask[e]);
}

// Counts of each run -> rows of the runs before it, expert by expert, and the totals.
__global__ __launch_bounds__(RT_PLACE) void route_counts(RouteArgs a, int runs) {
    const int lane = threadIdx.x & 63, e = (int)blockIdx.x * (RT_PLACE / 64) + (threadIdx.x >> 6);
    if (e >= a.experts) return;
    int before = 0;
    for (int b0 = 0; b0 < runs; b0 += 64) {
        const int b = b0 + lane;
        const int own = b < runs ? a.workspace[(int64_t)b * a.experts + e] : 0;
        int sum = own;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const int v = __shfl_up(sum, off, 64);
            if (lane >= off) sum += v;
        }
        if (b < runs) a.workspace[(int64_t)b * a.experts + e] = before + sum - own;
        before += __shfl(sum, 63, 64);
    }
    if (lane == 0) a.workspace[(int64_t)runs * a.experts + e] = before;
}

// A run's rows to their slots.  SUM: the counts of few runs are summed here, by every
// workgroup for itself, instead of by a launch before it.
template <bool SUM>
__global__ __launch_bounds__(RT_PLACE) void route_place(RouteArgs a, int run, int runs) {
    __shared__ int base[RT_MAX_EXPERTS];                  // an expert's first slot for this run
    __shared__ int whole[SUM ? RT_MAX_EXPERTS : 1];       // its rows of all runs
    __shared__ int part[RT_PLACE / 64];
    __shared__ unsigned long long mask[RT_MAX_EXPERTS];
    const int tid = threadIdx.x, E = a.experts;
    constexpr int PER = RT_MAX_EXPERTS / RT_PLACE;
    int own[PER], ahead[PER], sum = 0;
    if constexpr (SUM) {
        for (int e = tid; e < E; e += RT_PLACE) {
            int all = 0, before = 0;
            for (int b0 = 0; b0 < runs; b0 += 16) {       // 16 loads at once
                int c[16];
#pragma unroll
                for (int i = 0; i < 16; i++) c[i] = a.workspace[min(b0 + i, runs - 1) * E + e];
#pragma unroll
                for (int i = 0; i < 16; i++) {
                    all += b0 + i < runs ? c[i] : 0;
                    before += b0 + i < (int)blockIdx.x ? c[i] : 0;
                }
            }
            base[e] = before, whole[e] = all;
        }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < PER; i++) {
        const int e = tid * PER + i;
        own[i] = e >= E ? 0 : SUM ? whole[e] : a.workspace[(int64_t)runs * E + e];
        ahead[i] = e >= E ? 0 : SUM ? base[e] : a.workspace[(int64_t)blockIdx.x * E + e];
        sum += own[i];
        if (e < E) mask[e] = 0;
    }
    int total;
    int at = before_threads<RT_PLACE>(sum, part, total);
#pragma unroll
    for (int i = 0; i < PER; i++) {
        const int e = tid * PER + i;
        if (e < E) {
            base[e] = at + ahead[i];
            if (blockIdx.x == 0) a.expert_start[e] = at;
        }
        at += own[i];
    }
    if (blockIdx.x == 0 && tid == 0) a.expert_start[E] = total;
    __syncthreads();
    const int64_t first = (int64_t)blockIdx.x * run * a.top_k;
    const int entries = (int)min((int64_t)run * a.top_k, (int64_t)a.tokens * a.top_k - first);
    for (int i = tid; i < entries; i += RT_PLACE) {
        const int id = a.ids[first + i];
        if (id >= 0) atomicOr(&mask[id], 1ull << (i / a.top_k));
    }
    __syncthreads();
    for (int i = tid; i < entries; i += RT_PLACE) place(a, first, i, a.ids[first + i], base, mask, total);
}

// Up to RT_SMALL tokens: everything in one workgroup.
template <bool F32, int VPL>
__global__ __launch_bounds__(64 * rt_waves(VPL)) void route_small(RouteArgs a, int wide) {
    constexpr int THREADS = 64 * rt_waves(VPL), PER = RT_MAX_EXPERTS / THREADS;
    __shared__ int base[RT_MAX_EXPERTS];
    __shared__ int part[rt_waves(VPL)];
    __shared__ unsigned long long mask[RT_MAX_EXPERTS];
    const int tid = threadIdx.x, E = a.experts;
    for (int e = tid; e < E; e += THREADS) mask[e] = 0;
    __syncthreads();
    route_run<F32, VPL>(a, 0, a.tokens, wide, mask);
    __syncthreads();
    int own[PER], sum = 0, total;
#pragma unroll
    for (int i = 0; i < PER; i++) {
        const int e = tid * PER + i;
        own[i] = e < E ? __popcll(mask[e]) : 0;
        sum += own[i];
    }
    int at = before_threads<THREADS>(sum, part, total);
#pragma unroll
    for (int i = 0; i < PER; i++) {
        const int e = tid * PER + i;
        if (e < E) base[e] = a.expert_start[e] = at;
        at += own[i];
    }
    if (tid == 0) a.expert_start[E] = total;
    __syncthreads();
    const int entries = a.tokens * a.top_k;
    // ids from this workgroup's own stores (ordered by the barriers)
    for (int i = tid; i < entries; i += THREADS) place(a, 0, i, a.ids[i], base, mask, total);
}

struct RoutePlan {
    int run, runs;                       // tokens of a run; runs (0: one workgroup for all)
};
static RoutePlan route_plan(const RouteArgs& a) {
    if (a.tokens <= RT_SMALL) return {RT_RUN, 0};
    int run = 16;                        // a token a wave, until the card is full of runs
    while (run < RT_RUN && (int64_t)run * 256 < a.tokens) run *= 2;
    return {run, (a.tokens + run - 1) / run};
}

// A run's workgroup has up to 1024 threads; the other launches have fewer.
bool moe_route_fits(const RouteArgs& a) { return route_plan(a).runs < ((int64_t)1 << 32) / 1024; }

int64_t moe_route_bytes(const RouteArgs& a) {
    const RoutePlan p = route_plan(a);
    return p.runs ? ((int64_t)p.runs + 1) * a.experts * 4 : 0;
}

template <bool F32, int VPL>
static hipError_t queue_route(const RouteArgs& a, hipStream_t stream) {
    const RoutePlan p = route_plan(a);
    int wide = 1;
    while (wide < a.top_k) wide *= 2;
    if (p.runs == 0) {
        route_small<F32, VPL><<<dim3(1), dim3(64 * rt_waves(VPL)), 0, stream>>>(a, wide);
        return hipGetLastError();
    }
    route_tokens<F32, VPL><<<dim3((unsigned)p.runs), dim3(64 * rt_waves(VPL)), 0, stream>>>(a, p.run, wide);
    if (p.runs <= RT_SUM_RUNS) {
        route_place<true><<<dim3((unsigned)p.runs), dim3(RT_PLACE), 0, stream>>>(a, p.run, p.runs);
        return hipGetLastError();
    }
    route_counts<<<dim3((unsigned)((a.experts + RT_PLACE / 64 - 1) / (RT_PLACE / 64))), dim3(RT_PLACE), 0, stream>>>(a, p.runs);
    route_place<false><<<dim3((unsigned)p.runs), dim3(RT_PLACE), 0, stream>>>(a, p.run, p.runs);
    return hipGetLastError();
}

template <bool F32>
static hipError_t launch_route(const RouteArgs& a, hipStream_t stream) {
    if (a.experts <= 64) return queue_route<F32, 1>(a, stream);
    if (a.experts <= 128) return queue_route<F32, 2>(a, stream);
    if (a.experts <= 256) return queue_route<F32, 4>(a, stream);
    if (a.experts <= 512) return queue_route<F32, 8>(a, stream);
    return queue_route<F32, 16>(a, stream);
}

hipError_t launch_moe_route(const RouteArgs& a, int f32, hipStream_t stream) {
    return f32 ? launch_route<true>(a, stream) : launch_route<false>(a, stream);
}

}  // namespace fp8g
