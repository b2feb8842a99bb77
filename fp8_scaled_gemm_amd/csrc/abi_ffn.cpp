// C ABI of the feed-forward half's operators (fp8g_ffn.h): host-side argument
// checks, then the launches on the caller's stream.  Every check runs before
// any HIP call, so a rejected call queues nothing and touches no device.

#include "fp8g_ffn.h"

#include <stdint.h>

#include "args.h"
#include "launch_ffn.h"

namespace {

using namespace fp8g;

bool valid_type(int t) { return t == 0 || t == 1; }
int hip_status(hipError_t e) { return e == hipSuccess ? FP8G_OK : FP8G_ERR_HIP; }

constexpr int64_t LIM22 = (int64_t)1 << 22, LIM23 = (int64_t)1 << 23, LIM28 = (int64_t)1 << 28, LIM31 = (int64_t)1 << 31;
constexpr int64_t MAX_EXPERTS = 1024;

// a * b fits 2^60 and so on: bytes of an array of a x b elements of `size`
int64_t bytes(int64_t a, int64_t b, int64_t size) { return mul3(a, b, size); }

// Sizes of a fused product that hold for both modes; `products`: experts, or 1.
int check_product(int64_t m, int64_t n, int64_t k, int64_t products, int act, int gated, int mx, int out_dtype) {
    if (m < 0 || n < 0 || k < 0 || products < 0) return FP8G_ERR_SHAPE;
    if (mx && k % 32 != 0) return FP8G_ERR_SHAPE;
    if (!valid_type(out_dtype) || act < FP8G_ACT_NONE || act > FP8G_ACT_GELU_TANH) return FP8G_ERR_DTYPE;
    const int64_t n_lim = out_dtype == FP8G_OUT_F32 ? LIM22 / 2 : LIM22;
    if (k % 16 != 0 || k >= LIM23 || m >= LIM31 || n >= n_lim || n * (gated ? 2 : 1) >= n_lim) return FP8G_ERR_UNSUPPORTED;
    return FP8G_OK;
}

int fused(int64_t m, int64_t n, int64_t k, int64_t experts, const uint8_t* A, int64_t a_rows, const int32_t* rows,
          const int32_t* start, const uint8_t* B, const void* sa, const void* sb, int mx, const float* bias, int act,
          int gated, const void* residual, void* D, int out_dtype, void* ws, int64_t ws_bytes, bool moe,
          hipStream_t stream) {
    const int64_t products = moe ? experts : 1, b_rows = gated ? 2 * n : n, esz = out_dtype == FP8G_OUT_F32 ? 4 : 2;
    const int st = check_product(m, n, k, products, act, gated, mx, out_dtype);
    if (st != FP8G_OK) return st;
    if (moe) {
        if (a_rows < 0 || (!rows && a_rows != m) || (a_rows == 0 && m > 0)) return FP8G_ERR_SHAPE;
        if (experts > MAX_EXPERTS || m >= LIM28 || a_rows >= LIM31) return FP8G_ERR_UNSUPPORTED;
        if (rows && (bytes(a_rows, k, 1) < 0 || bytes(a_rows, k, 1) >= LIM31)) return FP8G_ERR_UNSUPPORTED;
    }
    if (m == 0 || n == 0 || products == 0) return FP8G_OK;
    const int64_t scale = mx ? 1 : 4, per = mx ? k / 32 : 1;      // of scales: bytes, and how many a row
    const int64_t ab = bytes(a_rows, k, 1), bb = mul3(products, b_rows, k), db = bytes(m, n, esz);
    const int64_t sab = bytes(a_rows, per, scale), sbb = mul3(products * b_rows, per, scale);
    if (ab < 0 || bb < 0 || db < 0 || sab < 0 || sbb < 0) return FP8G_ERR_UNSUPPORTED;
    FusedArgs a = {A, B, sa, sb, bias, residual, D, rows, moe ? start : nullptr, ws, m, n, k, a_rows, products, act,
                   gated != 0, mx, out_dtype == FP8G_OUT_F32};
    const int64_t need = moe ? moe_gemm_bytes(a) : gemm_fused_bytes(a);
    if (ws_bytes < need || (moe && !moe_gemm_fits(a))) return FP8G_ERR_UNSUPPORTED;
    if ((ab > 0 && !A) || (bb > 0 && !B) || (sab > 0 && !sa) || (sbb > 0 && !sb) || !D || (moe && !start) ||
        (need > 0 && !ws))
        return FP8G_ERR_NULL;
    const uintptr_t scale_align = 16;
    if (!aligned16(A) || !aligned16(B) || !aligned(sa, scale_align) || !aligned(sb, scale_align) || !aligned16(D) ||
        !aligned16(residual) || !aligned(bias, 4) || !aligned(rows, 4) || !aligned(start, 4) || !aligned16(ws))
        return FP8G_ERR_ALIGN;
    const Rows in[] = {bytes_of(A, ab), bytes_of(B, bb), bytes_of(sa, sab), bytes_of(sb, sbb),
                       bytes_of(bias, bias ? products * b_rows * 4 : 0), bytes_of(rows, rows ? m * 4 : 0),
                       bytes_of(start, moe ? (experts + 1) * 4 : 0)};
    const Rows d = bytes_of(D, db), w = bytes_of(ws, need), r = bytes_of(residual, residual ? db : 0);
    for (const Rows& x : in)
        if (overlaps(d, x) || overlaps(w, x)) return FP8G_ERR_OVERLAP;
    if ((residual != D && overlaps(d, r)) || overlaps(d, w) || overlaps(w, r)) return FP8G_ERR_OVERLAP;
    return hip_status(launch_gemm_fused(a, stream));
}

RouteArgs route_sizes(int64_t tokens, int64_t experts, int64_t top_k) {
    RouteArgs a = {};
    a.tokens = (int32_t)tokens, a.experts = (int32_t)experts, a.top_k = (int32_t)top_k;
    return a;
}

int check_route_sizes(int64_t tokens, int64_t experts, int64_t top_k) {
    if (tokens < 0 || experts < 1 || top_k < 1 || top_k > experts) return FP8G_ERR_SHAPE;
    if (experts > MAX_EXPERTS || top_k > 32 || tokens >= LIM28 || tokens * top_k >= LIM28) return FP8G_ERR_UNSUPPORTED;
    if (!moe_route_fits(route_sizes(tokens, experts, top_k))) return FP8G_ERR_UNSUPPORTED;
    return FP8G_OK;
}

}  // namespace

extern "C" {

int add_rms_norm_quantize(const void* x, int64_t x_stride, const void* residual, int64_t residual_stride, int in_dtype,
                          int64_t rows, int64_t cols, const float* weight, float eps, int granularity, int out_fmt,
                          void* sum, void* norm, uint8_t* q, void* scale, hipStream_t stream) {
    if (rows < 0 || cols < 0) return FP8G_ERR_SHAPE;
    const bool mx = granularity == FP8G_SCALE_MX;
    if (!valid_type(in_dtype) || !valid_type(out_fmt) || (!mx && granularity != FP8G_SCALE_PER_ROW) ||
        (mx && out_fmt != FP8G_FMT_E4M3))
        return FP8G_ERR_DTYPE;
    if (mx && cols % 32 != 0) return FP8G_ERR_SHAPE;
    if (cols % 16 != 0 || cols >= LIM28 || rows >= ((int64_t)1 << 24)) return FP8G_ERR_UNSUPPORTED;
    if (rows == 0 || cols == 0) return FP8G_OK;
    const int64_t esz = in_dtype == FP8G_IN_F32 ? 4 : 2, to = 16 / esz;
    if (x_stride < cols || (residual && residual_stride < cols)) return FP8G_ERR_SHAPE;
    if (x_stride % to || (residual && residual_stride % to) || mul3(rows, x_stride, esz) < 0 ||
        (residual && mul3(rows, residual_stride, esz) < 0))
        return FP8G_ERR_UNSUPPORTED;
    if (!x || !q || !scale) return FP8G_ERR_NULL;
    if (!aligned16(x) || !aligned16(residual) || !aligned(weight, 4) || !aligned16(sum) || !aligned16(norm) || !aligned16(q) ||
        !aligned(scale, mx ? 1 : 4))
        return FP8G_ERR_ALIGN;
    const Rows in = rows_of(x, rows, cols * esz, x_stride * esz);
    const Rows res = rows_of(residual, residual ? rows : 0, cols * esz, residual_stride * esz);
    const Rows w = bytes_of(weight, weight ? cols * 4 : 0);
    const Rows out[] = {bytes_of(sum, sum ? rows * cols * esz : 0), bytes_of(norm, norm ? rows * cols * esz : 0),
                        bytes_of(q, rows * cols), bytes_of(scale, mx ? rows * (cols / 32) : rows * 4)};
    for (int i = 0; i < 4; i++) {
        const bool x_here = i == 0 && sum == x && x_stride == cols, r_here = i == 0 && sum == residual && residual_stride == cols;
        if ((!x_here && overlaps(out[i], in)) || (!r_here && overlaps(out[i], res)) || overlaps(out[i], w)) return FP8G_ERR_OVERLAP;
        for (int j = 0; j < i; j++)
            if (overlaps(out[i], out[j])) return FP8G_ERR_OVERLAP;
    }
    const NormArgs a = {x, residual, weight, sum, norm, q, scale, x_stride, residual_stride, (int32_t)rows, (int32_t)cols, eps, 1.0 / (double)cols};
    return hip_status(launch_add_rms_norm(a, in_dtype == FP8G_IN_F32, mx, out_fmt == FP8G_FMT_E5M2, stream));
}

int fp8_gemm_fused(int64_t m, int64_t n, int64_t k, const uint8_t* A, const uint8_t* B, const float* scale_a,
                   const float* scale_b, const float* bias, int act, int gated, const void* residual, void* D,
                   int out_dtype, void* workspace, int64_t workspace_bytes, hipStream_t stream) {
    return fused(m, n, k, 1, A, m, nullptr, nullptr, B, scale_a, scale_b, 0, bias, act, gated, residual, D, out_dtype,
                 workspace, workspace_bytes, false, stream);
}

int mxfp8_gemm_fused(int64_t m, int64_t n, int64_t k, const uint8_t* A, const uint8_t* B, const uint8_t* scale_a,
                     const uint8_t* scale_b, const float* bias, int act, int gated, const void* residual, void* D,
                     int out_dtype, void* workspace, int64_t workspace_bytes, hipStream_t stream) {
    return fused(m, n, k, 1, A, m, nullptr, nullptr, B, scale_a, scale_b, 1, bias, act, gated, residual, D, out_dtype,
                 workspace, workspace_bytes, false, stream);
}

int64_t gemm_fused_workspace(int64_t m, int64_t n, int64_t k, int gated, int mx) {
    if (check_product(m, n, k, 1, FP8G_ACT_NONE, gated, mx, FP8G_OUT_BF16) != FP8G_OK) return -1;
    FusedArgs a = {};
    a.m = m, a.n = n, a.k = k, a.experts = 1, a.gated = gated != 0, a.mx = mx != 0;
    return m && n ? gemm_fused_bytes(a) : 0;
}

int64_t moe_gemm_workspace(int64_t slots, int64_t n, int64_t k, int64_t experts, int gathered, int gated, int mx) {
    if (check_product(slots, n, k, experts, FP8G_ACT_NONE, gated, mx, FP8G_OUT_BF16) != FP8G_OK || experts > MAX_EXPERTS ||
        slots >= LIM28)
        return -1;
    FusedArgs a = {};
    static const int32_t some = 0;
    a.m = slots, a.n = n, a.k = k, a.experts = experts, a.gated = gated != 0, a.mx = mx != 0;
    a.rows = gathered ? &some : nullptr;
    a.expert_start = &some;
    if (!slots || !n || !experts) return 0;
    return moe_gemm_fits(a) ? moe_gemm_bytes(a) : -1;
}

int fp8_moe_gemm(int64_t slots, int64_t n, int64_t k, int64_t experts, const uint8_t* A, int64_t a_rows,
                 const int32_t* rows, const int32_t* expert_start, const uint8_t* B, const float* scale_a,
                 const float* scale_b, const float* bias, int act, int gated, void* D, int out_dtype, void* workspace,
                 int64_t workspace_bytes, hipStream_t stream) {
    return fused(slots, n, k, experts, A, a_rows, rows, expert_start, B, scale_a, scale_b, 0, bias, act, gated, nullptr, D,
                 out_dtype, workspace, workspace_bytes, true, stream);
}

int mxfp8_moe_gemm(int64_t slots, int64_t n, int64_t k, int64_t experts, const uint8_t* A, int64_t a_rows,
                   const int32_t* rows, const int32_t* expert_start, const uint8_t* B, const uint8_t* scale_a,
                   const uint8_t* scale_b, const float* bias, int act, int gated, void* D, int out_dtype,
                   void* workspace, int64_t workspace_bytes, hipStream_t stream) {
    return fused(slots, n, k, experts, A, a_rows, rows, expert_start, B, scale_a, scale_b, 1, bias, act, gated, nullptr, D,
                 out_dtype, workspace, workspace_bytes, true, stream);
}

int64_t moe_route_workspace(int64_t tokens, int64_t experts, int64_t top_k) {
    if (check_route_sizes(tokens, experts, top_k) != FP8G_OK) return -1;
    return moe_route_bytes(route_sizes(tokens, experts, top_k));
}

int moe_route(const void* logits, int in_dtype, int64_t tokens, int64_t experts, int64_t top_k, const float* bias,
              int score, int64_t groups, int64_t top_groups, int64_t group_top, int renormalize, float scale,
              int32_t* ids, float* weights, int32_t* expert_start, int32_t* rows, int32_t* slots, void* workspace,
              int64_t workspace_bytes, hipStream_t stream) {
    const int st = check_route_sizes(tokens, experts, top_k);
    if (st == FP8G_ERR_SHAPE || groups < 1 || (experts > 0 && experts % groups != 0) || top_groups < 1 ||
        top_groups > groups || group_top < 1 || group_top > 2 || group_top > experts / groups)
        return FP8G_ERR_SHAPE;
    if (!valid_type(in_dtype) || score < FP8G_SCORE_SOFTMAX || score > FP8G_SCORE_SIGMOID) return FP8G_ERR_DTYPE;
    if (st != FP8G_OK || groups > 64) return FP8G_ERR_UNSUPPORTED;
    RouteArgs a = route_sizes(tokens, experts, top_k);
    const int64_t need = moe_route_bytes(a);
    if (workspace_bytes < need) return FP8G_ERR_UNSUPPORTED;
    const int64_t slots_n = tokens * top_k, esz = in_dtype == FP8G_IN_F32 ? 4 : 2;
    if (!expert_start || (need > 0 && !workspace) || (tokens > 0 && (!logits || !ids || !weights || !rows || !slots)))
        return FP8G_ERR_NULL;
    if (!aligned16(logits) || !aligned(bias, 4) || !aligned(ids, 4) || !aligned(weights, 4) || !aligned(expert_start, 4) ||
        !aligned(rows, 4) || !aligned(slots, 4) || !aligned16(workspace))
        return FP8G_ERR_ALIGN;
    const Rows in[] = {bytes_of(logits, tokens * experts * esz), bytes_of(bias, bias ? experts * 4 : 0)};
    const Rows out[] = {bytes_of(ids, slots_n * 4), bytes_of(weights, slots_n * 4), bytes_of(expert_start, (experts + 1) * 4),
                        bytes_of(rows, slots_n * 4), bytes_of(slots, slots_n * 4), bytes_of(workspace, need)};
    for (int i = 0; i < 6; i++) {
        for (const Rows& r : in)
            if (overlaps(out[i], r)) return FP8G_ERR_OVERLAP;
        for (int j = 0; j < i; j++)
            if (overlaps(out[i], out[j])) return FP8G_ERR_OVERLAP;
    }
    a.logits = logits, a.bias = bias, a.ids = ids, a.weights = weights, a.expert_start = expert_start, a.rows = rows;
    a.slots = slots, a.workspace = static_cast<int32_t*>(workspace);
    a.groups = (int32_t)groups, a.top_groups = (int32_t)top_groups, a.group_top = (int32_t)group_top;
    a.sigmoid = score == FP8G_SCORE_SIGMOID, a.renormalize = renormalize != 0, a.scale = scale;
    return hip_status(launch_moe_route(a, in_dtype == FP8G_IN_F32, stream));
}

int moe_combine(const void* y, int64_t y_rows, const int32_t* slots, const float* weights, const void* residual,
                int dtype, int64_t tokens, int64_t top_k, int64_t width, void* out, hipStream_t stream) {
    if (y_rows < 0 || tokens < 0 || top_k < 0 || width < 0) return FP8G_ERR_SHAPE;
    if (!valid_type(dtype)) return FP8G_ERR_DTYPE;
    const int64_t esz = dtype == FP8G_OUT_F32 ? 4 : 2;
    if (width * esz % 16 != 0 || width >= LIM28 || tokens >= LIM28 || top_k >= LIM28 || y_rows >= LIM28) return FP8G_ERR_UNSUPPORTED;
    if (tokens == 0 || width == 0) return FP8G_OK;
    const int64_t yb = mul3(y_rows, width, esz), ob = mul3(tokens, width, esz), sb = mul3(tokens, top_k, 4);
    if (yb < 0 || ob < 0 || sb < 0) return FP8G_ERR_UNSUPPORTED;
    const CombineArgs a = {y, residual, slots, weights, out, (int32_t)y_rows, (int32_t)tokens, (int32_t)top_k, (int32_t)width};
    if (!moe_combine_fits(a, dtype == FP8G_OUT_F32)) return FP8G_ERR_UNSUPPORTED;
    if ((yb > 0 && sb > 0 && !y) || (sb > 0 && (!slots || !weights)) || !out) return FP8G_ERR_NULL;
    if (!aligned16(y) || !aligned16(residual) || !aligned16(out) || !aligned(slots, 4) || !aligned(weights, 4)) return FP8G_ERR_ALIGN;
    const Rows o = bytes_of(out, ob);
    if (overlaps(o, bytes_of(y, yb)) || overlaps(o, bytes_of(slots, sb)) || overlaps(o, bytes_of(weights, sb)) ||
        (residual != out && overlaps(o, bytes_of(residual, residual ? ob : 0))))
        return FP8G_ERR_OVERLAP;
    return hip_status(launch_moe_combine(a, dtype == FP8G_OUT_F32, stream));
}

}  // extern "C"
