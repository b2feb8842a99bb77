/*
 * fp8g_block -- the attention block's operators around the FP8 projections, for
 * AMD Instinct MI355X (gfx950).  Same library, status codes and conventions as
 * fp8g.h (plain C ABI, device pointers, a HIP stream; arguments checked on the
 * host before any HIP call; nothing allocated, nothing synchronized).
 *
 * Operations (definitions in each entry point's comment):
 *   lora_add        out = base + scale[a] * B[a] (A[a] x), the adapter a by request
 *   qk_norm_rope    per-head RMS norm of queries and keys, and the position
 *                   rotation, in one pass
 *   kv4_append      key / value rows -> a paged MXFP4 cache
 *   kv4_gather      rows of that cache -> bf16 or float32
 *   kv4_attention   attention over that cache: decode and chunked prefill
 *
 * Device-side indices (slots, page tables, segment starts, lengths, positions)
 * are not known to the host and cannot be refused by status.  The kernels
 * clamp or skip what lies outside the arrays, as stated at each call, so a
 * wrong index gives wrong results there and never an access out of range.
 *
 * Index and statistics arrays (int32, int64, and the fp32 arrays scale, weight,
 * cos_sin, lse) need the alignment of their element only; all others 16 bytes.
 *
 * A launch has fewer than 2^32 threads.  Sizes that would need more
 * (hundreds of millions of rows) are ERR_UNSUPPORTED, too.
 *
 * Workspaces belong to the caller: <call>_workspace gives the bytes that the
 * same sizes need (0: none; the pointer may then be NULL).  Contents are
 * undefined before and after the call; calls that may overlap need their own.
 */
#ifndef FP8G_BLOCK_H
#define FP8G_BLOCK_H

#include "fp8g.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * lora_add -- low-rank adapters of many requests beside a shared projection.
 *
 *   out[t,:] = round( base[t,:] + scale[a] * B[a] (A[a] x[t,:]) ),
 *   a = seg_adapter[s] for seg_start[s] <= t < seg_start[s + 1]
 * with both products accumulated in fp32 and one rounding to `dtype` at the
 * end.  Tokens of a segment whose adapter is negative or >= adapters, and
 * tokens in no segment, keep base.  base is the projection's own output (for
 * example fp8_gemm_scaled's D).
 *
 * base     device, [tokens, n] of dtype (fp8g_out_t), read only unless out == base
 * x        device, bf16 [tokens, k], the projection's input
 * A        device, bf16 [adapters, rank, k]
 * B        device, bf16 [adapters, n, rank]
 * scale    device, fp32 [adapters]
 * seg_start    device, int32 [segments + 1], ascending; values are clamped to
 *              [0, tokens].  seg_adapter  device, int32 [segments]
 * out      device, [tokens, n] of dtype, written; may be base itself
 * Limits (ERR_UNSUPPORTED): rank % 8 != 0 or rank > 256; k % 8 != 0; tokens,
 * n, k or adapters >= 2^28; segments > 2^20.  tokens == 0 or n == 0: no-op.  k == 0
 * or rank == 0: out = base.
 * Accuracy: |out - exact| <= 1 ulp of dtype + 2^-16 (bf16) or 2^-22 (f32) of
 * |scale| sum |B| |A x| + the fp32 rounding of the sums.
 * Errors: ERR_NULL, ERR_SHAPE (negative extent), ERR_ALIGN, ERR_DTYPE,
 * ERR_OVERLAP (out or the workspace overlaps an input), ERR_UNSUPPORTED (also
 * a workspace smaller than lora_add_workspace), ERR_HIP.
 */
int lora_add(const void* base, const void* x, const void* A, const void* B, const float* scale,
             const int32_t* seg_start, const int32_t* seg_adapter, int64_t tokens, int64_t n, int64_t k,
             int64_t rank, int64_t adapters, int64_t segments, int dtype, void* out, void* workspace,
             int64_t workspace_bytes, hipStream_t stream);

/* Bytes of workspace lora_add needs; -1 for sizes it refuses. */
int64_t lora_add_workspace(int64_t tokens, int64_t n, int64_t k, int64_t rank, int64_t adapters, int64_t segments);

/*
 * qk_norm_rope -- RMS norm of every query and key head, then the rotation.
 *
 *   y = x / sqrt(mean_d x_d^2 + eps) * weight        (fp32, over head_dim)
 *   for every pair i < rotary_dim / 2, with p = positions[axis[i], t],
 *   c = cos_sin[p, i], s = cos_sin[p, rotary_dim / 2 + i]:
 *     (y_a, y_b) -> (y_a c - y_b s, y_b c + y_a s)
 *   a, b = i, i + rotary_dim / 2, or 2i, 2i + 1 where interleaved != 0;
 *   dimensions from rotary_dim on are normed only.  One rounding at the end.
 *
 * q        device, [tokens, q_heads, head_dim] of dtype (fp8g_out_t); rows of
 *          one token are dense, tokens are q_stride elements apart
 * k        device, [tokens, k_heads, head_dim], tokens k_stride apart
 * q_weight, k_weight  device, fp32 [head_dim]; NULL: all ones
 * positions  device, int32 [axes, tokens], clamped to [0, max_position)
 * axis     device, int32 [rotary_dim / 2], the axis of each pair, clamped to
 *          [0, axes); may be NULL when axes == 1
 * cos_sin  device, fp32 [max_position, rotary_dim]: cosines, then sines
 * q_out, k_out  device, written, strides as above; q_out may be q itself with
 *          its stride, and k_out may be k
 * Limits (ERR_UNSUPPORTED): head_dim % 8 != 0 or > 256; rotary_dim % 16 != 0;
 * strides not a multiple of 16 bytes; tokens >= 2^31; tokens * heads >= 2^31.
 * tokens == 0: no-op.  q_heads or k_heads may be 0.
 * Errors: ERR_NULL, ERR_SHAPE (negative extent, rotary_dim > head_dim or < 16,
 * axes < 1, axes > 1 without axis, max_position < 1, a stride below the row),
 * ERR_ALIGN, ERR_DTYPE, ERR_OVERLAP, ERR_UNSUPPORTED, ERR_HIP.
 */
int qk_norm_rope(const void* q, int64_t q_stride, const void* k, int64_t k_stride, int dtype, int64_t tokens,
                 int64_t q_heads, int64_t k_heads, int64_t head_dim, const float* q_weight, const float* k_weight,
                 float eps, const int32_t* positions, int64_t axes, const int32_t* axis, const float* cos_sin,
                 int64_t max_position, int64_t rotary_dim, int interleaved, void* q_out, int64_t q_out_stride,
                 void* k_out, int64_t k_out_stride, hipStream_t stream);

/*
 * The MXFP4 cache.  For keys and for values:
 *   codes   device, E2M1 [pages, heads, page_size, dim / 2], element 2i in the
 *           low nibble of byte i
 *   scales  device, UE8M0 [pages, heads, dim / 32, page_size]: code c stands
 *           for 2^(c - 127), one for each 32 elements of a row; the rows of a
 *           page lie side by side, so that attention reads 4 or 16 rows'
 *           scales at once
 * dim is dk for keys and dv for values; (dk, dv) one of (64, 64), (128, 128),
 * (192, 128).  page_size: a multiple of 16.  A slot is page * page_size + row.
 * The E2M1 magnitudes are 0, 0.5, 1, 1.5, 2, 3, 4, 6.
 */

/*
 * kv4_append -- quantize rows and write them to their slots.  For each block
 * of 32 elements of a row:
 *   e = the smallest integer with amax <= 6 * 2^e, in [-127, 127]; -127 for a
 *       block of zeros;  scale code e + 127
 *   code = E2M1_RNE(x * 2^-e)    (never above 6; the sign of zero is kept)
 * Bit-exact with this definition.
 *
 * k        device, [tokens, heads, dk] of in_dtype (fp8g_in_t), rows of one
 *          token dense, tokens k_stride elements apart;  v the same with dv
 * slots    device, int64 [tokens]; a negative slot or one >= pages *
 *          page_size is skipped; no two tokens may share one
 * NaN/Inf in k or v are outside the contract; magnitudes of 2^127 and more may
 * read back as infinity.
 * Limits (ERR_UNSUPPORTED): other dims; page_size % 16 != 0; strides not a
 * multiple of 16 bytes; tokens >= 2^31; heads > 2^16; size overflow.
 * tokens == 0 or heads == 0: no-op.
 * Errors: ERR_NULL, ERR_SHAPE (negative extent, page_size < 1, a stride below
 * the row), ERR_ALIGN, ERR_DTYPE, ERR_OVERLAP, ERR_UNSUPPORTED, ERR_HIP.
 */
int kv4_append(const void* k, int64_t k_stride, const void* v, int64_t v_stride, int in_dtype, int64_t tokens,
               int64_t heads, int64_t dk, int64_t dv, const int64_t* slots, int64_t pages, int64_t page_size,
               uint8_t* k_codes, uint8_t* k_scales, uint8_t* v_codes, uint8_t* v_scales, hipStream_t stream);

/*
 * kv4_gather -- read rows of the cache back as values (exact in bf16 and
 * float32): k_out [tokens, heads, dk], v_out [tokens, heads, dv] of out_dtype
 * (fp8g_out_t), dense.  Rows of a slot that kv4_append would skip are zero.
 * Limits and errors as kv4_append.
 */
int kv4_gather(const uint8_t* k_codes, const uint8_t* k_scales, const uint8_t* v_codes, const uint8_t* v_scales,
               int64_t pages, int64_t page_size, int64_t heads, int64_t dk, int64_t dv, const int64_t* slots,
               int64_t tokens, int out_dtype, void* k_out, void* v_out, hipStream_t stream);

/*
 * kv4_attention -- attention over the cache.
 *
 * Sequence b has the queries q_start[b] .. q_start[b + 1] - 1, n_b of them,
 * and the keys 0 .. kv_len[b] - 1; key j lies in page page_table[b, j /
 * page_size].  Its query i stands at position p = kv_len[b] - n_b + i and sees
 *   key j  if  j < kv_len[b]  and (not causal or j <= p)
 *              and (window == 0 or j > p - window).
 *   s_j = scale * q . k_j;  out = sum_j softmax(s)_j v_j;  lse = log sum_j exp s_j
 * over the keys it sees; a query that sees none has out = 0, lse = -inf, one
 * with a score of NaN or +inf NaN in both.
 * Query head h reads key head h / (q_heads / kv_heads).
 * Products on the bf16 matrix cores (keys and values are exact in bf16, the
 * softmax weights are rounded to bf16), sums and statistics in fp32.
 *
 * q        device, bf16 [queries, q_heads, dk], rows of one query dense,
 *          queries q_stride elements apart
 * page_table  device, int32 [batch, max_pages], entries clamped to [0, pages);
 *          entries of pages that no query sees are not used
 * q_start  device, int32 [batch + 1], ascending, clamped to [0, queries]
 * kv_len   device, int32 [batch], clamped to [0, max_pages * page_size]
 * window   > 0 needs causal != 0
 * out      device, bf16 [queries, q_heads, dv], dense; rows of no sequence are
 *          not written
 * lse      device, fp32 [queries, q_heads], or NULL
 * Bytes of a page beyond kv_len, and in front of the window, may hold anything.
 * A value that is no finite number (scale codes from 254 on) may also give NaN
 * to queries of its sequence that do not see it but whose neighbours do.
 * Limits (ERR_UNSUPPORTED): other dims; page_size % 16 != 0; q_heads not a
 * multiple of kv_heads; max_pages * page_size > 2^30; queries * q_heads >=
 * 2^31; batch > 2^20; strides not a multiple of 16 bytes; a workspace smaller
 * than kv4_attention_workspace.  queries == 0, batch == 0 or q_heads == 0:
 * no-op.
 * Errors: ERR_NULL, ERR_SHAPE (negative extent, a window without causal,
 * page_size < 1, a stride below the row), ERR_ALIGN, ERR_OVERLAP,
 * ERR_UNSUPPORTED, ERR_HIP.
 */
int kv4_attention(const void* q, int64_t q_stride, int64_t queries, int64_t q_heads, const uint8_t* k_codes,
                  const uint8_t* k_scales, const uint8_t* v_codes, const uint8_t* v_scales, int64_t pages,
                  int64_t page_size, int64_t kv_heads, int64_t dk, int64_t dv, const int32_t* page_table,
                  int64_t batch, int64_t max_pages, const int32_t* q_start, const int32_t* kv_len, float scale,
                  int causal, int64_t window, void* out, float* lse, void* workspace, int64_t workspace_bytes,
                  hipStream_t stream);

/* Bytes of workspace kv4_attention needs; -1 for sizes it refuses.  At most 69
 * MB, however long the table's rows are. */
int64_t kv4_attention_workspace(int64_t queries, int64_t q_heads, int64_t kv_heads, int64_t dk, int64_t dv,
                                int64_t batch, int64_t max_pages, int64_t page_size, int64_t window);

#ifdef __cplusplus
}
#endif

#endif /* FP8G_BLOCK_H */
