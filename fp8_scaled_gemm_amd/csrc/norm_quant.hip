// add_rms_norm_quantize: residual addition, RMS norm and quantization to FP8 in
// one pass over the rows.
//
//   s = round(x + r);  y = (s * rstd) * w,  rstd = 1 / sqrt(mean s^2 + eps)
//   per row:  scale = max|y| / MAX,  q = RNE(y / scale)
//   MX:       e of each 32 elements, q = RNE(y 2^-e)
//
// HBM-bound: x and r are read once, s and the codes written once; the row stays
// in registers between its two reductions (the sum of squares, and the amax of
// y, which needs rstd).  A workgroup of 256 threads holds a row, 16 bytes of
// it a load; rows longer than 16384 elements are read three times, the second
// and third time from the cache.  With MX the second reduction is that of 32
// neighbouring elements, held by 4 (bf16) or 8 (fp32) lanes.
//
// The squares are summed in fp32: a thread's in order, then over lanes and
// waves.  s is rounded to the input's type before the norm, since it is what
// the next layers read; y is not rounded before it is quantized.

#include "launch_ffn.h"
#include "row_div.h"
#include "rows16.h"

namespace fp8g {

constexpr int NORM_THREADS = 256;

// A vector of floats that is aligned as one float is.
typedef float v4f_a4 __attribute__((ext_vector_type(4), aligned(4)));
typedef unsigned int v2u __attribute__((ext_vector_type(2)));

template <class F>
__device__ __forceinline__ float over_waves(float v, float* red, F f) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    return f(f(red[0], red[1]), f(red[2], red[3]));
}

template <bool F32, int VPL, bool MX, class O>
__global__ __launch_bounds__(NORM_THREADS) void norm_rows(NormArgs a) {
    using R = Row16<F32>;
    constexpr int VEC = R::VEC, NV = VPL > 0 ? VPL : 1;
    __shared__ float red[8];
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.x, cols = a.cols;
    const int nv = a.cols / VEC;
    const v4u* x = reinterpret_cast<const v4u*>(a.x) + row * (a.x_stride / VEC);
    const v4u* res = a.residual ? reinterpret_cast<const v4u*>(a.residual) + row * (a.residual_stride / VEC) : nullptr;
    v4u* sum = a.sum ? reinterpret_cast<v4u*>(a.sum) + row * nv : nullptr;
    v4u* norm = a.norm ? reinterpret_cast<v4u*>(a.norm) + row * nv : nullptr;
    uint8_t* q = a.q + row * cols;

    // the s of vector idx, as loaded or added; `out`: its rounded form
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
    float f[NV][VEC], ss = 0.0f;
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
            add(vx[i], vr[i], f[i], out);
            if (sum && idx < nv) sum[idx] = out;
#pragma unroll
            for (int j = 0; j < VEC; j++) ss = __builtin_fmaf(f[i][j], f[i][j], ss);
        }
    } else {
        for (int idx = tid; idx < nv; idx += NORM_THREADS) {
            v4u out;
            add(x[idx], res ? res[idx] : (v4u){0, 0, 0, 0}, f[0], out);
            if (sum) sum[idx] = out;
#pragma unroll
            for (int j = 0; j < VEC; j++) ss = __builtin_fmaf(f[0][j], f[0][j], ss);
        }
    }
    ss = over_waves(wave_sum(ss), red, [](float u, float v) { return u + v; });
    // a sum that is no finite number: the row's scale says so
    const bool bad = !(ss <= 3.4028234e38f);
    const float rstd = bad ? __builtin_nanf("") : 1.0f / __builtin_sqrtf(ss / (float)a.cols + a.eps);

    // y of vector idx in place of its s
    auto normed = [&](int idx, float* v) __attribute__((always_inline)) {
        if (a.weight) {
            const v4f_a4* w = reinterpret_cast<const v4f_a4*>(a.weight + idx * VEC);
#pragma unroll
            for (int j = 0; j < VEC / 4; j++) {
                const v4f w4 = w[j];
#pragma unroll
                for (int t = 0; t < 4; t++) v[4 * j + t] = v[4 * j + t] * rstd * w4[t];
            }
        } else {
#pragma unroll
            for (int j = 0; j < VEC; j++) v[j] *= rstd;
        }
    };
    auto amax_of = [&](const float* v) __attribute__((always_inline)) {
        float m = 0.0f;
#pragma unroll
        for (int j = 0; j < VEC; j += 2) m = __builtin_fmaxf(m, amax2(v[j], v[j + 1]));
        return m;
    };
    // the s of vector idx once more (long rows): what was written, or the addition again
    auto again = [&](int idx, float* v) __attribute__((always_inline)) {
        v4u out;
        if (sum) R::unpack(sum[idx], v);
        else add(x[idx], res ? res[idx] : (v4u){0, 0, 0, 0}, v, out);
        normed(idx, v);
    };
    auto store = [&](int idx, const float* y) __attribute__((always_inline)) {
        if constexpr (VEC == 8)
            reinterpret_cast<v2u*>(q)[idx] = (v2u){O::pack4(y[0], y[1], y[2], y[3]), O::pack4(y[4], y[5], y[6], y[7])};
        else
            reinterpret_cast<uint32_t*>(q)[idx] = O::pack4(y[0], y[1], y[2], y[3]);
    };

    if constexpr (MX) {
        constexpr int LANES = 32 / VEC;          // of a block
        uint8_t* sc = reinterpret_cast<uint8_t*>(a.scale) + row * (cols / 32);
        auto block = [&](int idx, float* v) __attribute__((always_inline)) {
            if (norm && idx < nv) norm[idx] = R::pack(v);
            float m = bad ? 0.0f : amax_of(v);
#pragma unroll
            for (int off = 1; off < LANES; off <<= 1) m = __builtin_fmaxf(m, __shfl_xor(m, off, 64));
            const int e = mx_exponent(m);
            if (idx < nv) {
                if ((idx & (LANES - 1)) == 0) sc[idx / LANES] = bad ? 255 : (uint8_t)(e + 127);
#pragma unroll
                for (int j = 0; j < VEC; j++) v[j] = bad ? 0.0f : __builtin_amdgcn_ldexpf(v[j], -e);
                store(idx, v);
            }
        };
        if constexpr (VPL > 0) {
#pragma unroll
            for (int i = 0; i < VPL; i++) {
                const int idx = tid + NORM_THREADS * i;
                if (idx < nv) normed(idx, f[i]);
                block(idx, f[i]);
            }
        } else {
            // whole waves: a block's lanes stay together (nv is a multiple of LANES)
            for (int base = tid - (tid & 63); base < nv; base += NORM_THREADS) {
                const int idx = base + (tid & 63);
                float v[VEC] = {};
                if (idx < nv) again(idx, v);
                block(idx, v);
            }
        }
    } else {
        float m = 0.0f;
        if constexpr (VPL > 0) {
#pragma unroll
            for (int i = 0; i < VPL; i++) {
                const int idx = tid + NORM_THREADS * i;
                if (idx < nv) {
                    normed(idx, f[i]);
                    if (norm) norm[idx] = R::pack(f[i]);
                    m = __builtin_fmaxf(m, amax_of(f[i]));
                }
            }
        } else {
            for (int idx = tid; idx < nv; idx += NORM_THREADS) {
                again(idx, f[0]);
                if (norm) norm[idx] = R::pack(f[0]);
                m = __builtin_fmaxf(m, amax_of(f[0]));
            }
        }
        m = over_waves(wave_max(bad ? 0.0f : m), red + 4, [](float u, float v) { return __builtin_fmaxf(u, v); });
        const RowDiv d = row_div<O>(m);
        if (tid == 0) reinterpret_cast<float*>(a.scale)[row] = bad ? __builtin_nanf("") : d.s;
        by_path(d, [&](auto path) {
            constexpr int P = decltype(path)::value;
            auto quantize = [&](int idx, const float* v) __attribute__((always_inline)) {
                float y[VEC];
#pragma unroll
                for (int j = 0; j < VEC; j++) y[j] = bad ? 0.0f : quot<P>(v[j], d);
                store(idx, y);
            };
            if constexpr (VPL > 0) {
#pragma unroll
                for (int i = 0; i < VPL; i++) {
                    const int idx = tid + NORM_THREADS * i;
                    if (idx < nv) quantize(idx, f[i]);
                }
            } else {
                for (int idx = tid; idx < nv; idx += NORM_THREADS) {
                    again(idx, f[0]);
                    quantize(idx, f[0]);
                }
            }
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
