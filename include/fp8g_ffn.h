/*
 * fp8g_ffn -- the feed-forward half's operators around the FP8 products, for
 * AMD Instinct MI355X (gfx950).  Same library, status codes and conventions as
 * fp8g.h (plain C ABI, device pointers, a HIP stream; arguments checked on the
 * host before any HIP call; nothing allocated, nothing synchronized).
 *
 * Operations (definitions in each entry point's comment):
 *   add_rms_norm_quantize   residual addition, RMS norm and quantization to FP8
 *   fp8_gemm_fused,         the scaled products with bias, activation (plain
 *   mxfp8_gemm_fused        or gated) and residual in their epilogue
 *   moe_route               the experts of every token, their weights, and the
 *                           routed rows sorted by expert
 *   fp8_moe_gemm,           the experts' products over the routed rows, with
 *   mxfp8_moe_gemm          the same epilogue
 *   moe_combine             the weighted sum of every token's routed rows
 *
 * Device-side indices (rows, slots, expert starts) are not known to the host
 * and cannot be refused by status.  The kernels clamp or skip what lies
 * outside the arrays, as stated at each call, so a wrong index gives wrong
 * results there and never an access out of range.
 *
 * Index and statistics arrays (int32, and the fp32 arrays weight, bias, scale,
 * weights) need the alignment of their element only; all others 16 bytes.
 *
 * A launch has fewer than 2^32 threads.  Sizes that would need more are
 * ERR_UNSUPPORTED, too.
 *
 * Workspaces belong to the caller: <call>_workspace gives the bytes that the
 * same sizes need (0: none; the pointer may then be NULL).  Contents are
 * undefined before and after the call; calls that may overlap need their own.
 */
#ifndef FP8G_FFN_H
#define FP8G_FFN_H

#include "fp8g.h"

#ifdef __cplusplus
extern "C" {
#endif

/* a granularity of add_rms_norm_quantize beside FP8G_SCALE_PER_ROW */
enum { FP8G_SCALE_MX = 2 /* one UE8M0 code per 32 elements: scale [rows, cols / 32] */ };

typedef enum {
    FP8G_ACT_NONE = 0,      /* v */
    FP8G_ACT_SILU = 1,      /* v / (1 + exp(-v)) */
    FP8G_ACT_GELU_TANH = 2  /* v / (1 + exp(-2 u)), u = sqrt(2 / pi) (v + 0.044715 v^3) */
} fp8g_act_t;

typedef enum {
    FP8G_SCORE_SOFTMAX = 0, /* over the experts of a token */
    FP8G_SCORE_SIGMOID = 1
} fp8g_score_t;

/*
 * add_rms_norm_quantize -- what stands between a residual stream and the FP8
 * product that reads it.
 *
 *   s = round_in_dtype(x + residual)        (s = x where residual is NULL)
 *   y = s / sqrt(mean_c s_c^2 + eps) * weight_c
 *   per row (FP8G_SCALE_PER_ROW): scale[r] = fp32(max_c |y| / MAX), q = RNE_SAT(y * MAX / max_c |y|),
 *       MAX and RNE_SAT as in fp8_quantize_ex for out_fmt
 *   MX (FP8G_SCALE_MX): q and scale codes of y as in mxfp8_quantize (E4M3 only)
 * with everything behind s in fp64 (within 2^-48) and one rounding each to
 * scale, norm and codes.  A scale of 0 gives
 * signed zeros.
 * A row whose sum of squares is no finite number (it holds a NaN or an
 * infinity), or whose mean square + eps is not above 0 (zeros with eps = 0), has
 * codes 0 with the scale NaN (MX: codes 255), and NaN in norm; the others are not
 * touched by it.
 *
 * x        device, [rows, cols] of in_dtype (fp8g_in_t), rows x_stride elements apart
 * residual device, the same type, rows residual_stride elements apart, or NULL
 * weight   device, fp32 [cols], finite, or NULL: all ones
 * sum      device, [rows, cols] of in_dtype, dense, written with s, or NULL;
 *          may be x or residual itself, where that is dense
 * norm     device, [rows, cols] of in_dtype, dense, written with round(y), or NULL
 * q        device, codes of out_fmt [rows, cols], written
 * scale    device, written: fp32 [rows] or UE8M0 codes [rows, cols / 32]
 * rows == 0 or cols == 0: no-op.
 * Limits (ERR_UNSUPPORTED): cols % 16 != 0 (MX: cols % 32 != 0 is ERR_SHAPE);
 * strides not a multiple of 16 bytes; rows * 256 >= 2^32; cols >= 2^28.
 * Errors: ERR_NULL, ERR_SHAPE (negative extent, a stride below the row),
 * ERR_ALIGN, ERR_DTYPE (in_dtype, granularity, out_fmt; E5M2 with MX),
 * ERR_OVERLAP, ERR_UNSUPPORTED, ERR_HIP.
 */
int add_rms_norm_quantize(const void* x, int64_t x_stride, const void* residual, int64_t residual_stride,
                          int in_dtype, int64_t rows, int64_t cols, const float* weight, float eps, int granularity,
                          int out_fmt, void* sum, void* norm, uint8_t* q, void* scale, hipStream_t stream);

/*
 * fp8_gemm_fused, mxfp8_gemm_fused -- the products of fp8_gemm_scaled and
 * mxfp8_gemm (both operands E4M3) with the work behind them in the epilogue.
 *
 *   z[m, j] = scaled product of A's row m and B's row j, + bias[j]
 *   v[m, n] = act(z[m, n])                       not gated: B has n rows
 *           = act(z[m, n]) * z[m, N + n]         gated: B has 2 N rows, the
 *             gate projection's N first, then the up projection's
 *   D[m, n] = out( v[m, n] + residual[m, n] )
 * All of it in fp32, one rounding at the end.  Accuracy of z as there; the
 * activation adds (4 + |p|) 2^-22 of |v|, p = z (SILU) or 2 u (GELU_TANH): its
 * exponential and reciprocal are the hardware's, one ulp each, and p's own
 * rounding passes through the exponential.  Where 1 + exp(-p) passes 2^126, the
 * activation (below 2^-126 |z| in size) may be 0.  Of +inf it is +inf, of -inf and
 * NaN it is NaN.
 *
 * A        device, E4M3 codes [m, k]      B  device, E4M3 codes [n or 2 n, k]
 * scale_a, scale_b   fp32 [m], [n or 2 n];  mxfp8: UE8M0 codes [.., k / 32]
 * bias     device, fp32 [n or 2 n], or NULL
 * act      fp8g_act_t
 * residual device, [m, n] of out_dtype, or NULL; may be D itself
 * D        device, [m, n] of out_dtype (fp8g_out_t), written
 * workspace  device, gemm_fused_workspace bytes: the partial sums of products
 *          whose K is split (few tiles and a long K; at most 16 MB), and with
 *          block scales and k % 128 != 0 also copies of both operands' scale rows
 *          in whole dwords, (m + rows of B) * 4 * ceil(k / 128) bytes
 * m == 0 or n == 0: no-op.  k == 0: the product is 0.
 * Limits and contract as fp8_gemm_scaled / mxfp8_gemm, with n or 2 n rows of B
 * below 2^22 (bf16 output) / 2^21 (fp32); a workspace smaller than
 * gemm_fused_workspace is ERR_UNSUPPORTED.
 * Errors: ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_DTYPE (out_dtype, act),
 * ERR_OVERLAP, ERR_UNSUPPORTED, ERR_HIP.
 */
int fp8_gemm_fused(int64_t m, int64_t n, int64_t k, const uint8_t* A, const uint8_t* B, const float* scale_a,
                   const float* scale_b, const float* bias, int act, int gated, const void* residual, void* D,
                   int out_dtype, void* workspace, int64_t workspace_bytes, hipStream_t stream);
int mxfp8_gemm_fused(int64_t m, int64_t n, int64_t k, const uint8_t* A, const uint8_t* B, const uint8_t* scale_a,
                     const uint8_t* scale_b, const float* bias, int act, int gated, const void* residual, void* D,
                     int out_dtype, void* workspace, int64_t workspace_bytes, hipStream_t stream);

/* Bytes of workspace the fused products need (mx: of mxfp8_gemm_fused); -1 for
 * sizes they refuse. */
int64_t gemm_fused_workspace(int64_t m, int64_t n, int64_t k, int gated, int mx);

/*
 * moe_route -- the experts of every token.
 *
 *   p = softmax(logits) over the experts, or sigmoid(logits)
 *   choice = p + bias where there is a bias, else the logit itself (p grows with it)
 *   groups > 1: the experts form `groups` runs of experts / groups; a group's
 *       value is the sum of the group_top largest p (+ bias) of its available
 *       experts, and only the top_groups groups of the largest value stay
 *   ids: the top_k available experts of the largest choice, in falling order;
 *       ties go to the lowest index, of experts and of groups
 *   weights: p of those experts; renormalize: divided by their sum (0 where
 *       that is 0); times scale
 * An expert whose logit or bias is -inf or NaN is not available; a token with fewer
 * than top_k available experts has -1 and weight 0 in the last places (a token
 * whose logits are all -inf, a padded one, goes nowhere).  A group that lacks
 * group_top available experts is behind all that have them.  Logits of +inf share the
 * softmax among themselves.  p, choice and the sums are worked out in fp64, so
 * that the ids do not hang on an fp32 rounding.
 *
 * The routed rows, sorted by expert and within an expert by token:
 *   expert_start[e] .. expert_start[e + 1] - 1   the slots of expert e
 *   rows[slot]      the token of a slot; -1 from expert_start[experts] on
 *   slots[t, j]     the slot of token t's j-th expert; -1 where ids is
 *
 * logits   device, [tokens, experts] of in_dtype (fp8g_in_t)
 * bias     device, fp32 [experts], or NULL
 * ids      device, int32 [tokens, top_k]         weights  device, fp32 [tokens, top_k]
 * expert_start  device, int32 [experts + 1]      rows     device, int32 [tokens * top_k]
 * slots    device, int32 [tokens, top_k]
 * tokens == 0: expert_start is all 0.
 * Limits (ERR_UNSUPPORTED): experts > 1024; top_k > 32; groups > 64; tokens *
 * top_k >= 2^28; a workspace smaller than moe_route_workspace.
 * Errors: ERR_NULL, ERR_SHAPE (negative extent; experts < 1; top_k < 1 or >
 * experts; groups < 1 or not a divisor of experts; top_groups < 1 or > groups;
 * group_top < 1 or > 2 or > experts / groups), ERR_ALIGN, ERR_DTYPE (in_dtype, score),
 * ERR_OVERLAP, ERR_UNSUPPORTED, ERR_HIP.
 */
int moe_route(const void* logits, int in_dtype, int64_t tokens, int64_t experts, int64_t top_k, const float* bias,
              int score, int64_t groups, int64_t top_groups, int64_t group_top, int renormalize, float scale,
              int32_t* ids, float* weights, int32_t* expert_start, int32_t* rows, int32_t* slots, void* workspace,
              int64_t workspace_bytes, hipStream_t stream);

/* Bytes of workspace moe_route needs; -1 for sizes it refuses. */
int64_t moe_route_workspace(int64_t tokens, int64_t experts, int64_t top_k);

/*
 * fp8_moe_gemm, mxfp8_moe_gemm -- the experts' products.
 *
 *   D[s, :] = the epilogue of fp8_gemm_fused / mxfp8_gemm_fused (no residual)
 *             over A's row rows[s] (rows NULL: row s) and expert e's B, scale
 *             and bias, for the slots s of expert_start[e] .. expert_start[e + 1] - 1
 *
 * slots    the rows of D
 * A        device, E4M3 codes [a_rows, k] (a_rows == slots where rows is NULL)
 * rows     device, int32 [slots], or NULL; a row outside [0, a_rows) stands
 *          for some row inside
 * expert_start  device, int32 [experts + 1], ascending; values are clamped to [0,
 *          slots], and an expert's end to its start.  Where they are not ascending,
 *          slots that several experts claim hold the row of any of them, or none
 * B        device, E4M3 codes [experts, n or 2 n, k]
 * scale_a  fp32 [a_rows] or UE8M0 codes [a_rows, k / 32];  scale_b  [experts, n or 2 n] or [.., k / 32]
 * bias     device, fp32 [experts, n or 2 n], or NULL
 * D        device, [slots, n] of out_dtype, written; rows of no expert are not
 * slots == 0, experts == 0 or n == 0: no-op.  k == 0: the product is 0.
 * Limits (ERR_UNSUPPORTED) as fp8_gemm_fused; also experts > 1024; slots >=
 * 2^28; a_rows * k >= 2^31 where rows is given; a workspace smaller than
 * moe_gemm_workspace.
 * Errors: ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_DTYPE, ERR_OVERLAP,
 * ERR_UNSUPPORTED, ERR_HIP.
 */
int fp8_moe_gemm(int64_t slots, int64_t n, int64_t k, int64_t experts, const uint8_t* A, int64_t a_rows,
                 const int32_t* rows, const int32_t* expert_start, const uint8_t* B, const float* scale_a,
                 const float* scale_b, const float* bias, int act, int gated, void* D, int out_dtype, void* workspace,
                 int64_t workspace_bytes, hipStream_t stream);
int mxfp8_moe_gemm(int64_t slots, int64_t n, int64_t k, int64_t experts, const uint8_t* A, int64_t a_rows,
                   const int32_t* rows, const int32_t* expert_start, const uint8_t* B, const uint8_t* scale_a,
                   const uint8_t* scale_b, const float* bias, int act, int gated, void* D, int out_dtype,
                   void* workspace, int64_t workspace_bytes, hipStream_t stream);

/* Bytes of workspace the experts' products need (mx: of mxfp8_moe_gemm;
 * gathered: with rows); -1 for sizes they refuse. */
int64_t moe_gemm_workspace(int64_t slots, int64_t n, int64_t k, int64_t experts, int gathered, int gated, int mx);

/*
 * moe_combine -- the routed rows back to their tokens.
 *
 *   out[t, :] = round( residual[t, :] + sum_j weights[t, j] * y[slots[t, j], :] )
 * summed in fp32 in the order of j; slots outside [0, y_rows) add nothing.
 *
 * y        device, [y_rows, width] of dtype (fp8g_out_t)
 * slots    device, int32 [tokens, top_k]    weights  device, fp32 [tokens, top_k]
 * residual device, [tokens, width] of dtype, or NULL; may be out itself
 * out      device, [tokens, width] of dtype, written
 * tokens == 0 or width == 0: no-op.  top_k == 0: out = residual, or 0.
 * Limits (ERR_UNSUPPORTED): width not a multiple of 16 bytes; width >= 2^28;
 * tokens, top_k or y_rows >= 2^28; launches of 2^32 threads and more.
 * Errors: ERR_NULL, ERR_SHAPE (negative extent), ERR_ALIGN, ERR_DTYPE,
 * ERR_OVERLAP, ERR_UNSUPPORTED, ERR_HIP.
 */
int moe_combine(const void* y, int64_t y_rows, const int32_t* slots, const float* weights, const void* residual,
                int dtype, int64_t tokens, int64_t top_k, int64_t width, void* out, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* FP8G_FFN_H */
