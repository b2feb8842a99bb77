// add_rms_norm_quantize: residual addition, RMS norm and quantization to FP8 in
// one pass over the rows.
//
//   s = round(x + r);  y = s w rstd,  rstd = 1 / sqrt(mean s^2 + eps)
//   per row:  scale = max|y| / MAX,  q = RNE(y / scale) = RNE(s w MAX / max|s w|)
//   MX:       e of each 32 elements, q = RNE(y 2^-e)
//
// HBM-bound: x and r are read once, s and the codes written once; the row stays
// in registers in between.  A workgroup of 256 threads holds a row, 16 bytes of it
// a load; rows longer than 16384 elements are read twice, the second time from the
// cache.  rstd cancels in a row's quotient, so the sum of squares and the largest
// |s w| are found together, behind one barrier.  With MX the amax is that of 32
// neighbouring elements, held by 4 (bf16) or 8 (fp32) lanes.
// 16384 rows of 8192 bf16 with a residual, 940 MB: 167 us (5.6 TB/s); one row 2.9 us.
//
// Everything behind s is fp64, whose vector instructions run at the fp32 ones'
// rate here: products of two fp32 values are exact, so a code is the
// definition's but for ties 2^-50 apart, where in fp32 the roundings of y, scale
// and quotient moved one code in a million to its neighbour.

#include "launch_ffn.h"
#include "row_div.h"
#include "rows16.h"
#include "wave_ops.h"

namespace fp8g {

constexpr int NORM_THREADS = 256;

// A vector of floats that is aligned as one float is.
typedef float v4f_a4 __attribute__((ext_vector_type(4), aligned(4)));
typedef unsigned int v2u __attribute__((ext_vector_type(2)));

__device__ __forceinline__ double lane_xor(double v, int off) { return __shfl_xor(v, off, 64); }

// p * by to fp32 by rounding to odd: truncated to 20 bits of the significand,
// with the last bit set where any were lost, so that the rounding to FP8 behind
// it sees on which side of a tie the product lies.  by > 0, |p by| < 2^127; 2^-120
// of p's sign is added, which no product that FP8 tells from zero notices, so
// that the exponent is never below fp32's and the sign of a zero is kept.
__device__ __forceinline__ float to_odd(double p, double by) {
    const uint32_t sign = (uint32_t)(__builtin_bit_cast(uint64_t, p) >> 32) & 0x80000000u;
    const double little = __builtin_bit_cast(double, (uint64_t)(sign | 0x38700000u) << 32);
    const uint64_t u = __builtin_bit_cast(uint64_t, __builtin_fma(p, by, little));
    const uint32_t hi = (uint32_t)(u >> 32), lo = (uint32_t)u;
    // the exponent rebiased by 127 - 1023, modulo 2^32
    const uint32_t t = ((hi << 3) + 0x40000000u) | min(lo, 1u);
    return __builtin_bit_cast(float, (t & 0x7FFFFFFFu) | (hi & 0x80000000u));
}

// Four quotients, none above the format's largest value by more than a rounding
// of fp64, as codes: no clamp is needed (464 would be the first to overflow E4M3,
// 61440 E5M2).
__device__ __forceinline__ uint32_t pack_odd(OutE4M3, float a, float b, float c, float d) {
    const int r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, r, true);
}
__device__ __forceinline__ uint32_t pack_odd(OutE5M2, float a, float b, float c, float d) {
    const int r = __builtin_amdgcn_cvt_pk_bf8_f32(a, b, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_bf8_f32(c, d, r, true);
}

// 1 / sqrt(v), v > 0: the hardware's root to 2^-26 or so, and one Newton step.
__device__ __forceinline__ double inverse_root(double v) {
    const double r = __builtin_amdgcn_rsq(v);
    return r * (1.5 - 0.5 * v * r * r);
}

// Waves of a SIMD that the registers of a row are to allow.
constexpr int norm_waves(int vpl, int vec) { return vpl * vec > 32 ? 2 : 4; }

template <bool F32, int VPL, bool MX, class O>
__global__ __launch_bounds__(NORM_THREADS, norm_waves(VPL, Row16<F32>::VEC)) void norm_rows(NormArgs a) {
    using R = Row16<F32>;
    constexpr int VEC = R::VEC, NV = VPL > 0 ? VPL : 1;
    __shared__ double red[2][NORM_THREADS / 64];
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.x, cols = a.cols;
    const int nv = a.cols / VEC;
    const v4u* x = reinterpret_cast<const v4u*>(a.x) + row * (a.x_stride / VEC);
    const v4u* res = a.residual ? reinterpret_cast<const v4u*>(a.residual) + row * (a.residual_stride / VEC) : nullptr;
    v4u* sum = a.sum ? reinterpret_cast<v4u*>(a.sum) + row * nv : nullptr;
    v4u* norm = a.norm ? reinterpret_cast<v4u*>(a.norm) + row * nv : nullptr;
    uint8_t* q = a.q + row * cols;

    // the s of a vector; `out`: as it is stored
    auto add = [&](v4u vx, v4u vr, float* f, v4u& out) __attribute__((always_inline)) {
        R::unpack(vx, f);
        out = vx;
        if (res) {
            float g[VEC];
            R::unpack(vr, g);
#pragma unroll
            for (int i = 0; i < VEC; i++) f[i] += g[i];
            out = R::pack(f);
            R::unpack(out, f);
        }
    };
    // the weights of vector idx
    auto weights = [&](int idx, float* w) __attribute__((always_inline)) {
        if (a.weight) {
            const v4f_a4* p = reinterpret_cast<const v4f_a4*>(a.weight + idx * VEC);
#pragma unroll
            for (int j = 0; j < VEC / 4; j++) {
                const v4f w4 = p[j];
#pragma unroll
                for (int t = 0; t < 4; t++) w[4 * j + t] = w4[t];
            }
        } else {
#pragma unroll
            for (int j = 0; j < VEC; j++) w[j] = 1.0f;
        }
    };
    // p = s w of a vector, exact, and its part of the row's two reductions (with MX
    // only of the squares)
    double ss = 0.0, most = 0.0;
    auto product = [&](const float* f, const float* w, double* p) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < VEC; j++) {
            const double s = (double)f[j];
            ss = __builtin_fma(s, s, ss);
            p[j] = s * (double)w[j];
            if constexpr (!MX) most = __builtin_fmax(most, __builtin_fabs(p[j]));
        }
    };
    double p[NV][VEC];
    if constexpr (VPL > 0) {
        v4u vx[NV], vr[NV];
#pragma unroll
        for (int i = 0; i < VPL; i++) {
            const int idx = tid + NORM_THREADS * i;
            vx[i] = vr[i] = (v4u){0, 0, 0, 0};
            if (idx < nv) {
                vx[i] = x[idx];
                if (res) vr[i] = res[idx];
            }
        }
#pragma unroll
        for (int i = 0; i < VPL; i++) {
            const int idx = tid + NORM_THREADS * i;
            v4u out;
            float f[VEC], w[VEC] = {};
            add(vx[i], vr[i], f, out);
            if (idx < nv) {
                if (sum) sum[idx] = out;
                weights(idx, w);
            }
            product(f, w, p[i]);
        }
    } else {
        for (int idx = tid; idx < nv; idx += NORM_THREADS) {
            v4u out;
            float f[VEC], w[VEC];
            add(x[idx], res ? res[idx] : (v4u){0, 0, 0, 0}, f, out);
            if (sum) sum[idx] = out;
            weights(idx, w);
            product(f, w, p[0]);
        }
    }
    ss = wave_total(ss);
    if constexpr (!MX) most = wave_most(most);
    if ((tid & 63) == 0) red[0][tid >> 6] = ss, red[1][tid >> 6] = most;
    __syncthreads();
    ss = (red[0][0] + red[0][1]) + (red[0][2] + red[0][3]);
    // a sum that is no finite number, or a mean + eps with no root (a row of zeros and
    // eps = 0): the row's scale says so
    const double mean = ss * a.inv_cols + (double)a.eps;
    const bool bad = !(ss <= 1.7976931348623157e308) || !(mean > 0.0);
    const double rstd = bad ? __builtin_nan("") : inverse_root(mean);

    auto store = [&](int idx, const float* y) __attribute__((always_inline)) {
        if constexpr (VEC == 8)
            reinterpret_cast<v2u*>(q)[idx] = bad ? (v2u){0, 0} : (v2u){pack_odd(O{}, y[0], y[1], y[2], y[3]), pack_odd(O{}, y[4], y[5], y[6], y[7])};
        else
            reinterpret_cast<uint32_t*>(q)[idx] = bad ? 0u : pack_odd(O{}, y[0], y[1], y[2], y[3]);
    };
    auto store_norm = [&](int idx, const double* v) __attribute__((always_inline)) {
        float y[VEC];
#pragma unroll
        for (int j = 0; j < VEC; j++) y[j] = (float)(v[j] * rstd);
        norm[idx] = R::pack(y);
    };
    // each(idx, p of vector idx, in the row) over the thread's vectors; whole waves go
    // together, a block's lanes with them
    auto vectors = [&](auto each) __attribute__((always_inline)) {
        if constexpr (VPL > 0) {
#pragma unroll
            for (int i = 0; i < VPL; i++) each(tid + NORM_THREADS * i, p[i], tid + NORM_THREADS * i < nv);
        } else {
            // the row again: what was written, or the addition
            for (int base = tid - (tid & 63); base < nv; base += NORM_THREADS) {
                const int idx = base + (tid & 63);
                float f[VEC] = {}, w[VEC] = {};
                if (idx < nv) {
                    v4u out;
                    if (sum) R::unpack(sum[idx], f);
                    else add(x[idx], res ? res[idx] : (v4u){0, 0, 0, 0}, f, out);
                    weights(idx, w);
                }
#pragma unroll
                for (int j = 0; j < VEC; j++) p[0][j] = (double)f[j] * (double)w[j];
                each(idx, p[0], idx < nv);
            }
        }
    };
    if constexpr (MX) {
        constexpr int LANES = 32 / VEC;          // of a block
        uint8_t* sc = reinterpret_cast<uint8_t*>(a.scale) + row * (cols / 32);
        vectors([&](int idx, const double* v, bool in) __attribute__((always_inline)) {
            double y[VEC], m = 0.0;
#pragma unroll
            for (int j = 0; j < VEC; j++) {
                y[j] = bad ? 0.0 : v[j] * rstd;
                m = __builtin_fmax(m, __builtin_fabs(y[j]));
            }
#pragma unroll
            for (int off = 1; off < LANES; off <<= 1) m = __builtin_fmax(m, lane_xor(m, off));
            if (!in) return;
            // e from m's own bits: m = c 2^k, 1 <= c < 2, and 448 = 1.75 * 2^8
            const uint64_t u = __builtin_bit_cast(uint64_t, m);
            int e = (int)(u >> 52) - 1023 - 8 + ((u & 0xFFFFFFFFFFFFFull) > 0xC000000000000ull ? 1 : 0);
            const bool over = e > 127;                     // past every scale (a weight near 2^127)
            e = min(max(e, -127), 127);
            if ((idx & (LANES - 1)) == 0) sc[idx / LANES] = bad || over ? 255 : (uint8_t)(e + 127);
            const double by = over ? 0x1p-300 : __builtin_bit_cast(double, (uint64_t)(1023 - e) << 52);
            float t[VEC];
#pragma unroll
            for (int j = 0; j < VEC; j++) t[j] = to_odd(y[j], by);
            store(idx, t);
            if (norm) store_norm(idx, v);
        });
    } else {
        most = __builtin_fmax(__builtin_fmax(red[1][0], red[1][1]), __builtin_fmax(red[1][2], red[1][3]));
        const float scale = bad ? __builtin_nanf("") : (float)(most * rstd / (double)O::MAX);
        if (tid == 0) reinterpret_cast<float*>(a.scale)[row] = scale;
        // a row whose scale is 0: signed zeros, by a factor below all codes
        const double by = scale > 0.0f ? (double)O::MAX / most : 0x1p-300;
        vectors([&](int idx, const double* v, bool in) __attribute__((always_inline)) {
            if (!in) return;
            float t[VEC];
#pragma unroll
            for (int j = 0; j < VEC; j++) t[j] = to_odd(v[j], by);
            store(idx, t);
            if (norm) store_norm(idx, v);
        });
    }
}

template <bool F32, bool MX, class O>
static hipError_t launch_norm(const NormArgs& a, hipStream_t stream) {
    constexpr int VEC = Row16<F32>::VEC;
    const int per = NORM_THREADS * VEC;
    auto go = [&](auto kernel) {
        kernel<<<dim3((unsigned)a.rows), dim3(NORM_THREADS), 0, stream>>>(a);
        return hipGetLastError();
    };
    if (a.cols <= per) return go(norm_rows<F32, 1, MX, O>);
    if (a.cols <= 2 * per) return go(norm_rows<F32, 2, MX, O>);
    if (a.cols <= 4 * per) return go(norm_rows<F32, 4, MX, O>);
    if (a.cols <= 8 * per) return go(norm_rows<F32, 8, MX, O>);
    if constexpr (F32)
        if (a.cols <= 16 * per) return go(norm_rows<F32, 16, MX, O>);
    return go(norm_rows<F32, 0, MX, O>);
}

hipError_t launch_add_rms_norm(const NormArgs& a, int f32, int mx, int e5m2, hipStream_t stream) {
    if (mx) return f32 ? launch_norm<true, true, OutE4M3>(a, stream) : launch_norm<false, true, OutE4M3>(a, stream);
    if (e5m2) return f32 ? launch_norm<true, false, OutE5M2>(a, stream) : launch_norm<false, false, OutE5M2>(a, stream);
    return f32 ? launch_norm<true, false, OutE4M3>(a, stream) : launch_norm<false, false, OutE4M3>(a, stream);
}

}  // namespace fp8g
