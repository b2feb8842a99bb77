// C ABI of the attention block's operators (fp8g_block.h): host-side argument
// checks, then the launches on the caller's stream.  Every check runs before
// any HIP call, so a rejected call queues nothing and touches no device.

#include "fp8g_block.h"

#include <stdint.h>

#include "args.h"
#include "launch_block.h"

namespace {

using namespace fp8g;

bool valid_type(int t) { return t == 0 || t == 1; }
int hip_status(hipError_t e) { return e == hipSuccess ? FP8G_OK : FP8G_ERR_HIP; }

constexpr int64_t LIM28 = (int64_t)1 << 28, LIM31 = (int64_t)1 << 31;

fp8g::LoraArgs lora_sizes(int64_t tokens, int64_t n, int64_t k, int64_t rank, int64_t adapters, int64_t segments) {
    fp8g::LoraArgs a = {};
    a.tokens = (int32_t)tokens, a.n = (int32_t)n, a.k = (int32_t)k, a.rank = (int32_t)rank;
    a.adapters = (int32_t)adapters, a.segments = (int32_t)segments;
    return a;
}

int check_lora_sizes(int64_t tokens, int64_t n, int64_t k, int64_t rank, int64_t adapters, int64_t segments) {
    if (tokens < 0 || n < 0 || k < 0 || rank < 0 || adapters < 0 || segments < 0) return FP8G_ERR_SHAPE;
    if (rank % 8 != 0 || rank > 256 || k % 8 != 0 || tokens >= LIM28 || n >= LIM28 || k >= LIM28 ||
        adapters >= LIM28 || segments > ((int64_t)1 << 20))
        return FP8G_ERR_UNSUPPORTED;
    return fp8g::lora_add_fits(lora_sizes(tokens, n, k, rank, adapters, segments)) ? FP8G_OK : FP8G_ERR_UNSUPPORTED;
}

bool dims_ok(int64_t dk, int64_t dv) {
    return (dk == 64 && dv == 64) || (dk == 128 && dv == 128) || (dk == 192 && dv == 128);
}

bool rows_fit(int64_t tokens, int64_t heads, int64_t dk, int64_t dv) {
    fp8g::Kv4RowsArgs a = {};
    a.side[0].dim = (int32_t)dk, a.side[1].dim = (int32_t)dv;
    a.tokens = (int32_t)tokens, a.heads = (int32_t)heads, a.page_size = 16;
    return fp8g::kv4_rows_fit(a);
}

// The cache's arrays, as ranges; a status below 0: go on.
struct Cache {
    Rows r[4];
};
int check_cache(const void* kc, const void* ks, const void* vc, const void* vs, int64_t pages, int64_t page_size,
                int64_t heads, int64_t dk, int64_t dv, Cache& c) {
    const int64_t cells = mul3(pages, heads, page_size);
    if (cells < 0 || mul3(cells, dk, 1) < 0) return FP8G_ERR_UNSUPPORTED;
    if (cells > 0 && (!kc || !ks || !vc || !vs)) return FP8G_ERR_NULL;
    if (!aligned16(kc) || !aligned16(ks) || !aligned16(vc) || !aligned16(vs)) return FP8G_ERR_ALIGN;
    c.r[0] = bytes_of(kc, cells * (dk / 2));
    c.r[1] = bytes_of(ks, cells * (dk / 32));
    c.r[2] = bytes_of(vc, cells * (dv / 2));
    c.r[3] = bytes_of(vs, cells * (dv / 32));
    return -1;
}

// a window that reaches behind every key is none
int32_t window_of(int64_t window) { return (int32_t)(window < LIM28 * 4 ? window : 0); }

fp8g::Kv4AttnArgs attn_sizes(int64_t queries, int64_t q_heads, int64_t kv_heads, int64_t dk, int64_t dv, int64_t batch,
                             int64_t max_pages, int64_t page_size, int64_t window) {
    fp8g::Kv4AttnArgs a = {};
    a.queries = (int32_t)queries, a.q_heads = (int32_t)q_heads, a.kv_heads = (int32_t)kv_heads;
    a.dk = (int32_t)dk, a.dv = (int32_t)dv, a.batch = (int32_t)batch, a.max_pages = (int32_t)max_pages;
    a.page_size = (int32_t)page_size, a.window = window_of(window);
    return a;
}

int check_attn_sizes(int64_t queries, int64_t q_heads, int64_t kv_heads, int64_t dk, int64_t dv, int64_t batch,
                     int64_t max_pages, int64_t page_size, int64_t window) {
    if (queries < 0 || q_heads < 0 || kv_heads < 0 || dk < 0 || dv < 0 || batch < 0 || max_pages < 0 ||
        page_size < 1 || window < 0 || (kv_heads == 0 && q_heads > 0))
        return FP8G_ERR_SHAPE;
    if (!dims_ok(dk, dv) || page_size % 16 != 0 || (kv_heads > 0 && q_heads % kv_heads != 0) ||
        batch > ((int64_t)1 << 20))
        return FP8G_ERR_UNSUPPORTED;
    const int64_t keys = mul3(max_pages, page_size, 1), rows = mul3(queries, q_heads, 1), blocks = mul3(batch, q_heads, 1);
    if (keys < 0 || keys > ((int64_t)1 << 30) || page_size > ((int64_t)1 << 30) || rows < 0 || rows >= LIM31 ||
        queries >= LIM31 || blocks < 0 || blocks >= LIM28)
        return FP8G_ERR_UNSUPPORTED;
    return fp8g::kv4_attention_fits(attn_sizes(queries, q_heads, kv_heads, dk, dv, batch, max_pages, page_size, window))
               ? FP8G_OK : FP8G_ERR_UNSUPPORTED;
}

}  // namespace

extern "C" {

int64_t lora_add_workspace(int64_t tokens, int64_t n, int64_t k, int64_t rank, int64_t adapters, int64_t segments) {
    if (check_lora_sizes(tokens, n, k, rank, adapters, segments) != FP8G_OK) return -1;
    return fp8g::lora_add_bytes(lora_sizes(tokens, n, k, rank, adapters, segments));
}

int lora_add(const void* base, const void* x, const void* A, const void* B, const float* scale,
             const int32_t* seg_start, const int32_t* seg_adapter, int64_t tokens, int64_t n, int64_t k, int64_t rank,
             int64_t adapters, int64_t segments, int dtype, void* out, void* workspace, int64_t workspace_bytes,
             hipStream_t stream) {
    const int st = check_lora_sizes(tokens, n, k, rank, adapters, segments);
    if (st == FP8G_ERR_SHAPE) return st;
    if (!valid_type(dtype)) return FP8G_ERR_DTYPE;
    if (st != FP8G_OK) return st;
    if (tokens == 0 || n == 0) return FP8G_OK;
    const int64_t esz = dtype == FP8G_OUT_F32 ? 4 : 2;
    const int64_t o_bytes = mul3(tokens, n, esz), x_bytes = mul3(tokens, k, 2);
    const int64_t a_bytes = mul3(adapters, rank * k, 2), b_bytes = mul3(adapters, rank * n, 2);
    if (o_bytes < 0 || x_bytes < 0 || a_bytes < 0 || b_bytes < 0) return FP8G_ERR_UNSUPPORTED;
    if (!base || !out || !seg_start || (segments > 0 && !seg_adapter) || (x_bytes > 0 && !x) || (a_bytes > 0 && !A) ||
        (b_bytes > 0 && !B) || (adapters > 0 && !scale))
        return FP8G_ERR_NULL;
    if (!aligned16(base) || !aligned16(out) || !aligned16(x) || !aligned16(A) || !aligned16(B) || !aligned(scale, 4) ||
        !aligned(seg_start, 4) || !aligned(seg_adapter, 4) || !aligned16(workspace))
        return FP8G_ERR_ALIGN;
    fp8g::LoraArgs a = {base, x, A, B, scale, seg_start, seg_adapter, out, static_cast<float*>(workspace),
                        (int32_t)tokens, (int32_t)n, (int32_t)k, (int32_t)rank, (int32_t)adapters, (int32_t)segments};
    const int64_t need = adapters > 0 && segments > 0 ? fp8g::lora_add_bytes(a) : 0;
    if (workspace_bytes < need) return FP8G_ERR_UNSUPPORTED;
    if (need > 0 && !workspace) return FP8G_ERR_NULL;
    const Rows in[] = {bytes_of(x, x_bytes), bytes_of(A, a_bytes), bytes_of(B, b_bytes), bytes_of(scale, adapters * 4),
                       bytes_of(seg_start, (segments + 1) * 4), bytes_of(seg_adapter, segments * 4)};
    const Rows o = bytes_of(out, o_bytes), bs = bytes_of(base, o_bytes), ws = bytes_of(workspace, need);
    for (const Rows& r : in)
        if (overlaps(o, r) || overlaps(ws, r)) return FP8G_ERR_OVERLAP;
    if ((out != base && overlaps(o, bs)) || overlaps(ws, o) || overlaps(ws, bs)) return FP8G_ERR_OVERLAP;
    return hip_status(fp8g::launch_lora_add(a, dtype == FP8G_OUT_F32, stream));
}

int qk_norm_rope(const void* q, int64_t q_stride, const void* k, int64_t k_stride, int dtype, int64_t tokens,
                 int64_t q_heads, int64_t k_heads, int64_t head_dim, const float* q_weight, const float* k_weight,
                 float eps, const int32_t* positions, int64_t axes, const int32_t* axis, const float* cos_sin,
                 int64_t max_position, int64_t rotary_dim, int interleaved, void* q_out, int64_t q_out_stride,
                 void* k_out, int64_t k_out_stride, hipStream_t stream) {
    if (tokens < 0 || q_heads < 0 || k_heads < 0 || head_dim < 0) return FP8G_ERR_SHAPE;
    if (!valid_type(dtype)) return FP8G_ERR_DTYPE;
    if (tokens == 0 || q_heads + k_heads == 0 || head_dim == 0) return FP8G_OK;
    if (rotary_dim < 16 || rotary_dim > head_dim || axes < 1 || max_position < 1) return FP8G_ERR_SHAPE;
    if (head_dim % 8 != 0 || head_dim > 256 || rotary_dim % 16 != 0 || q_heads >= LIM28 || k_heads >= LIM28 ||
        tokens >= LIM31 || axes >= LIM28 || max_position >= LIM31 || mul3(tokens, q_heads + k_heads, 1) < 0 ||
        mul3(tokens, q_heads + k_heads, 1) >= LIM31)
        return FP8G_ERR_UNSUPPORTED;
    const int64_t esz = dtype == FP8G_OUT_F32 ? 4 : 2, to = 16 / esz;
    const int64_t q_row = q_heads * head_dim, k_row = k_heads * head_dim;
    if ((q_heads > 0 && (q_stride < q_row || q_out_stride < q_row)) ||
        (k_heads > 0 && (k_stride < k_row || k_out_stride < k_row)) || (axes > 1 && !axis))
        return FP8G_ERR_SHAPE;
    fp8g::QkArgs sizes = {};
    sizes.tokens = (int32_t)tokens, sizes.q_heads = (int32_t)q_heads, sizes.k_heads = (int32_t)k_heads;
    sizes.head_dim = (int32_t)head_dim;
    if (!fp8g::qk_norm_rope_fits(sizes, dtype == FP8G_OUT_F32)) return FP8G_ERR_UNSUPPORTED;
    if ((q_heads > 0 && (q_stride % to || q_out_stride % to)) || (k_heads > 0 && (k_stride % to || k_out_stride % to)))
        return FP8G_ERR_UNSUPPORTED;
    if ((q_heads > 0 && (mul3(tokens, q_stride, esz) < 0 || mul3(tokens, q_out_stride, esz) < 0)) ||
        (k_heads > 0 && (mul3(tokens, k_stride, esz) < 0 || mul3(tokens, k_out_stride, esz) < 0)))
        return FP8G_ERR_UNSUPPORTED;
    if ((q_heads > 0 && (!q || !q_out)) || (k_heads > 0 && (!k || !k_out)) || !positions || !cos_sin) return FP8G_ERR_NULL;
    if ((q_heads > 0 && (!aligned16(q) || !aligned16(q_out))) || (k_heads > 0 && (!aligned16(k) || !aligned16(k_out))) ||
        !aligned(q_weight, 4) || !aligned(k_weight, 4) || !aligned(positions, 4) || !aligned(axis, 4) || !aligned(cos_sin, 4))
        return FP8G_ERR_ALIGN;
    const Rows qi = rows_of(q, tokens, q_row * esz, q_stride * esz), ki = rows_of(k, tokens, k_row * esz, k_stride * esz);
    const Rows qo = rows_of(q_out, tokens, q_row * esz, q_out_stride * esz);
    const Rows ko = rows_of(k_out, tokens, k_row * esz, k_out_stride * esz);
    const bool q_here = q_out == q && q_out_stride == q_stride, k_here = k_out == k && k_out_stride == k_stride;
    if ((!q_here && overlaps(qo, qi)) || (!k_here && overlaps(ko, ki)) || overlaps(qo, ki) || overlaps(ko, qi) ||
        overlaps(qo, ko))
        return FP8G_ERR_OVERLAP;
    const Rows read[] = {bytes_of(q_weight, q_weight ? head_dim * 4 : 0), bytes_of(k_weight, k_weight ? head_dim * 4 : 0),
                         bytes_of(positions, axes * tokens * 4), bytes_of(axis, axis ? rotary_dim * 2 : 0),
                         bytes_of(cos_sin, max_position * rotary_dim * 4)};
    for (const Rows& r : read)
        if (overlaps(qo, r) || overlaps(ko, r)) return FP8G_ERR_OVERLAP;
    const fp8g::QkArgs a = {q, k, q_out, k_out, q_weight, k_weight, cos_sin, positions, axis, q_stride, k_stride,
                            q_out_stride, k_out_stride, (int32_t)tokens, (int32_t)q_heads, (int32_t)k_heads,
                            (int32_t)head_dim, (int32_t)rotary_dim, (int32_t)axes, (int32_t)max_position,
                            interleaved != 0, eps};
    return hip_status(fp8g::launch_qk_norm_rope(a, dtype == FP8G_OUT_F32, stream));
}

int kv4_append(const void* k, int64_t k_stride, const void* v, int64_t v_stride, int in_dtype, int64_t tokens,
               int64_t heads, int64_t dk, int64_t dv, const int64_t* slots, int64_t pages, int64_t page_size,
               uint8_t* k_codes, uint8_t* k_scales, uint8_t* v_codes, uint8_t* v_scales, hipStream_t stream) {
    if (tokens < 0 || heads < 0 || dk < 0 || dv < 0 || pages < 0 || page_size < 1) return FP8G_ERR_SHAPE;
    if (!valid_type(in_dtype)) return FP8G_ERR_DTYPE;
    if (!dims_ok(dk, dv) || page_size % 16 != 0 || page_size > ((int64_t)1 << 30) || heads > 65536 || tokens >= LIM31)
        return FP8G_ERR_UNSUPPORTED;
    if (tokens == 0 || heads == 0) return FP8G_OK;
    if (!rows_fit(tokens, heads, dk, dv)) return FP8G_ERR_UNSUPPORTED;
    const int64_t esz = in_dtype == FP8G_IN_BF16 ? 2 : 4, to = 16 / esz;
    if (k_stride < heads * dk || v_stride < heads * dv) return FP8G_ERR_SHAPE;
    if (k_stride % to || v_stride % to || mul3(tokens, k_stride, esz) < 0 || mul3(tokens, v_stride, esz) < 0)
        return FP8G_ERR_UNSUPPORTED;
    if (!k || !v || !slots) return FP8G_ERR_NULL;
    if (!aligned16(k) || !aligned16(v) || !aligned(slots, 8)) return FP8G_ERR_ALIGN;
    Cache c;
    const int st = check_cache(k_codes, k_scales, v_codes, v_scales, pages, page_size, heads, dk, dv, c);
    if (st >= 0) return st;
    const Rows in[] = {rows_of(k, tokens, heads * dk * esz, k_stride * esz),
                       rows_of(v, tokens, heads * dv * esz, v_stride * esz), bytes_of(slots, tokens * 8)};
    for (int i = 0; i < 4; i++) {
        for (const Rows& r : in)
            if (overlaps(c.r[i], r)) return FP8G_ERR_OVERLAP;
        for (int j = 0; j < i; j++)
            if (overlaps(c.r[i], c.r[j])) return FP8G_ERR_OVERLAP;
    }
    fp8g::Kv4RowsArgs a = {};
    a.side[0] = {k_codes, k_scales, (int32_t)dk};
    a.side[1] = {v_codes, v_scales, (int32_t)dv};
    a.in[0] = k, a.in[1] = v;
    a.stride[0] = k_stride, a.stride[1] = v_stride;
    a.slots = slots, a.slot_end = pages * page_size;
    a.tokens = (int32_t)tokens, a.heads = (int32_t)heads, a.page_size = (int32_t)page_size;
    return hip_status(fp8g::launch_kv4_append(a, in_dtype == FP8G_IN_BF16, stream));
}

int kv4_gather(const uint8_t* k_codes, const uint8_t* k_scales, const uint8_t* v_codes, const uint8_t* v_scales,
               int64_t pages, int64_t page_size, int64_t heads, int64_t dk, int64_t dv, const int64_t* slots,
               int64_t tokens, int out_dtype, void* k_out, void* v_out, hipStream_t stream) {
    if (tokens < 0 || heads < 0 || dk < 0 || dv < 0 || pages < 0 || page_size < 1) return FP8G_ERR_SHAPE;
    if (!valid_type(out_dtype)) return FP8G_ERR_DTYPE;
    if (!dims_ok(dk, dv) || page_size % 16 != 0 || page_size > ((int64_t)1 << 30) || heads > 65536 || tokens >= LIM31)
        return FP8G_ERR_UNSUPPORTED;
    if (tokens == 0 || heads == 0) return FP8G_OK;
    if (!rows_fit(tokens, heads, dk, dv)) return FP8G_ERR_UNSUPPORTED;
    const int64_t esz = out_dtype == FP8G_OUT_F32 ? 4 : 2;
    const int64_t kb = mul3(tokens, heads, dk * esz), vb = mul3(tokens, heads, dv * esz);
    if (kb < 0 || vb < 0) return FP8G_ERR_UNSUPPORTED;
    if (!k_out || !v_out || !slots) return FP8G_ERR_NULL;
    if (!aligned16(k_out) || !aligned16(v_out) || !aligned(slots, 8)) return FP8G_ERR_ALIGN;
    Cache c;
    const int st = check_cache(k_codes, k_scales, v_codes, v_scales, pages, page_size, heads, dk, dv, c);
    if (st >= 0) return st;
    const Rows ko = bytes_of(k_out, kb), vo = bytes_of(v_out, vb), sl = bytes_of(slots, tokens * 8);
    if (overlaps(ko, vo) || overlaps(ko, sl) || overlaps(vo, sl)) return FP8G_ERR_OVERLAP;
    for (const Rows& r : c.r)
        if (overlaps(ko, r) || overlaps(vo, r)) return FP8G_ERR_OVERLAP;
    fp8g::Kv4RowsArgs a = {};
    a.side[0] = {const_cast<uint8_t*>(k_codes), const_cast<uint8_t*>(k_scales), (int32_t)dk};
    a.side[1] = {const_cast<uint8_t*>(v_codes), const_cast<uint8_t*>(v_scales), (int32_t)dv};
    a.out[0] = k_out, a.out[1] = v_out;
    a.slots = slots, a.slot_end = pages * page_size;
    a.tokens = (int32_t)tokens, a.heads = (int32_t)heads, a.page_size = (int32_t)page_size;
    return hip_status(fp8g::launch_kv4_gather(a, out_dtype == FP8G_OUT_F32, stream));
}

int64_t kv4_attention_workspace(int64_t queries, int64_t q_heads, int64_t kv_heads, int64_t dk, int64_t dv,
                                int64_t batch, int64_t max_pages, int64_t page_size, int64_t window) {
    if (check_attn_sizes(queries, q_heads, kv_heads, dk, dv, batch, max_pages, page_size, window) != FP8G_OK) return -1;
    return fp8g::kv4_attention_bytes(attn_sizes(queries, q_heads, kv_heads, dk, dv, batch, max_pages, page_size, window));
}

int kv4_attention(const void* q, int64_t q_stride, int64_t queries, int64_t q_heads, const uint8_t* k_codes,
                  const uint8_t* k_scales, const uint8_t* v_codes, const uint8_t* v_scales, int64_t pages,
                  int64_t page_size, int64_t kv_heads, int64_t dk, int64_t dv, const int32_t* page_table,
                  int64_t batch, int64_t max_pages, const int32_t* q_start, const int32_t* kv_len, float scale,
                  int causal, int64_t window, void* out, float* lse, void* workspace, int64_t workspace_bytes,
                  hipStream_t stream) {
    int st = check_attn_sizes(queries, q_heads, kv_heads, dk, dv, batch, max_pages, page_size, window);
    if (st != FP8G_OK) return st;
    if (pages < 0 || (window > 0 && !causal)) return FP8G_ERR_SHAPE;
    if (queries == 0 || batch == 0 || q_heads == 0) return FP8G_OK;
    if (q_stride < q_heads * dk) return FP8G_ERR_SHAPE;
    if (pages >= LIM31 || q_stride % 8 || mul3(queries, q_stride, 2) < 0) return FP8G_ERR_UNSUPPORTED;
    if (!q || !out || !q_start || !kv_len || (max_pages > 0 && !page_table)) return FP8G_ERR_NULL;
    if (!aligned16(q) || !aligned16(out) || !aligned16(workspace) || !aligned(q_start, 4) || !aligned(kv_len, 4) ||
        !aligned(page_table, 4) || !aligned(lse, 4))
        return FP8G_ERR_ALIGN;
    Cache c;
    st = check_cache(k_codes, k_scales, v_codes, v_scales, pages, page_size, kv_heads, dk, dv, c);
    if (st >= 0) return st;
    const fp8g::Kv4AttnArgs a = {q, k_codes, k_scales, v_codes, v_scales, page_table, q_start, kv_len, out, lse,
                                 static_cast<float*>(workspace), q_stride, (int32_t)queries, (int32_t)q_heads,
                                 (int32_t)kv_heads, (int32_t)dk, (int32_t)dv, (int32_t)pages, (int32_t)page_size,
                                 (int32_t)batch, (int32_t)max_pages, causal != 0,
                                 window_of(window), scale};
    const int64_t need = fp8g::kv4_attention_bytes(a);
    if (workspace_bytes < need) return FP8G_ERR_UNSUPPORTED;
    if (need > 0 && !workspace) return FP8G_ERR_NULL;
    const Rows o[] = {bytes_of(out, queries * q_heads * dv * 2), bytes_of(lse, lse ? queries * q_heads * 4 : 0),
                      bytes_of(workspace, need)};
    const Rows in[] = {rows_of(q, queries, q_heads * dk * 2, q_stride * 2), c.r[0], c.r[1], c.r[2], c.r[3],
                       bytes_of(page_table, batch * max_pages * 4), bytes_of(q_start, (batch + 1) * 4),
                       bytes_of(kv_len, batch * 4)};
    for (int i = 0; i < 3; i++) {
        for (const Rows& r : in)
            if (overlaps(o[i], r)) return FP8G_ERR_OVERLAP;
        for (int j = 0; j < i; j++)
            if (overlaps(o[i], o[j])) return FP8G_ERR_OVERLAP;
    }
    return hip_status(fp8g::launch_kv4_attention(a, stream));
}

}  // extern "C"
