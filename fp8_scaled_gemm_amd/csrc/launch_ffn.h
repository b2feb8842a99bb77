// Internal launchers of the feed-forward half's operators (fp8g_ffn.h), called
// by the C ABI after argument checks.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp8g {

struct NormArgs {
    const void *x, *residual;
    const float* weight;
    void *sum, *norm;
    uint8_t* q;
    void* scale;
    int64_t x_stride, residual_stride;   // elements
    int32_t rows, cols;
    float eps;
    double inv_cols;
};
hipError_t launch_add_rms_norm(const NormArgs& a, int f32, int mx, int e5m2, hipStream_t stream);

// One product, or the experts' (expert_start given): D = act(z) or act(z_gate) z_up, + residual.
struct FusedArgs {
    const uint8_t *A, *B;
    const void *scale_a, *scale_b;       // fp32, or UE8M0 codes
    const float* bias;
    const void* residual;
    void* D;
    const int32_t *rows, *expert_start;
    void* workspace;
    int64_t m, n, k, a_rows, experts;    // m: rows of D; n: columns of D
    int32_t act, gated, mx, f32;
};
int64_t gemm_fused_bytes(const FusedArgs& a);
int64_t moe_gemm_bytes(const FusedArgs& a);
bool moe_gemm_fits(const FusedArgs& a);
hipError_t launch_gemm_fused(const FusedArgs& a, hipStream_t stream);
hipError_t launch_gemm_rows(const FusedArgs& a, hipStream_t stream);      // few rows, no workspace
bool gemm_rows_fits(const FusedArgs& a);

// A launch of the tile kernel; for the experts' products with its plan (gemm_tile.h).
struct TileLaunch {
    int tile, dev, cus;
    int64_t tile_rows;                   // of all experts, at most
    const int32_t* plan;
    const uint32_t* row_at;
    const void* scale_a;
    int32_t ranges, pitch, part_rows;    // K ranges' partial sums
};
struct RouteArgs {
    const void* logits;
    const float* bias;
    int32_t *ids, *expert_start, *rows, *slots, *workspace;
    float* weights;
    int32_t tokens, experts, top_k, groups, top_groups, group_top, sigmoid, renormalize;
    float scale;
};
bool moe_route_fits(const RouteArgs& a);
int64_t moe_route_bytes(const RouteArgs& a);
hipError_t launch_moe_route(const RouteArgs& a, int f32, hipStream_t stream);

struct CombineArgs {
    const void *y, *residual;
    const int32_t* slots;
    const float* weights;
    void* out;
    int32_t y_rows, tokens, top_k, width;
};
bool moe_combine_fits(const CombineArgs& a, int f32);
hipError_t launch_moe_combine(const CombineArgs& a, int f32, hipStream_t stream);

}  // namespace fp8g
