// Internal launchers of the attention block's operators (fp8g_block.h), called
// by the C ABI after argument checks.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp8g {

// A launch has fewer than 2^32 threads along a dimension; the runtime refuses
// others.  <operator>_fits: whether the launches of these sizes are so (pointers
// unread), asked before anything is queued.
inline int64_t most_blocks(int threads) { return (((int64_t)1 << 32) - 1) / threads; }

struct QkArgs {
    const void *q, *k;
    void *q_out, *k_out;
    const float *q_weight, *k_weight, *cos_sin;
    const int32_t *positions, *axis;
    int64_t q_stride, k_stride, q_out_stride, k_out_stride;   // elements
    int32_t tokens, q_heads, k_heads, head_dim, rotary_dim, axes, max_position, interleaved;
    float eps;
};
bool qk_norm_rope_fits(const QkArgs& a, int f32);
hipError_t launch_qk_norm_rope(const QkArgs& a, int f32, hipStream_t stream);

// One side (keys or values) of the MXFP4 cache.
struct Kv4Side {
    uint8_t *codes, *scales;
    int32_t dim;
};

struct Kv4RowsArgs {
    Kv4Side side[2];
    const void* in[2];        // append: rows; gather: unused
    void* out[2];             // gather: rows; append: unused
    int64_t stride[2];        // elements between tokens
    const int64_t* slots;
    int64_t slot_end;         // pages * page_size
    int32_t tokens, heads, page_size;
};
bool kv4_rows_fit(const Kv4RowsArgs& a);
hipError_t launch_kv4_append(const Kv4RowsArgs& a, int bf16, hipStream_t stream);
hipError_t launch_kv4_gather(const Kv4RowsArgs& a, int f32, hipStream_t stream);

struct Kv4AttnArgs {
    const void* q;
    const uint8_t *k_codes, *k_scales, *v_codes, *v_scales;
    const int32_t *page_table, *q_start, *kv_len;
    void* out;
    float *lse, *workspace;
    int64_t q_stride;
    int32_t queries, q_heads, kv_heads, dk, dv, pages, page_size, batch, max_pages, causal, window;
    float scale;
};
// bytes of workspace for these sizes (pointers and lengths on the device unread)
int64_t kv4_attention_bytes(const Kv4AttnArgs& a);
bool kv4_attention_fits(const Kv4AttnArgs& a);
hipError_t launch_kv4_attention(const Kv4AttnArgs& a, hipStream_t stream);

struct LoraArgs {
    const void *base, *x, *A, *B;
    const float* scale;
    const int32_t *seg_start, *seg_adapter;
    void* out;
    float* workspace;
    int32_t tokens, n, k, rank, adapters, segments;
};
int64_t lora_add_bytes(const LoraArgs& a);
bool lora_add_fits(const LoraArgs& a);
hipError_t launch_lora_add(const LoraArgs& a, int f32, hipStream_t stream);

}  // namespace fp8g
