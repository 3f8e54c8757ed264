// moe_kernels.h -- host-side interface between the entry points of expert
// routing, 8-bit integer products and the gather of expert rows (moe_api.hip)
// and their kernel files.  Internal to the library; not installed.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/qmm.h"

namespace qmm {

// Sets the calling thread's qmm_last_error text and returns st (qmm_api.hip).
qmm_status report(qmm_status st, const char* fmt, ...);

struct RouteArgs {
    const void* logits;  // fp32 or fp16 rows
    const float* bias;   // or null
    const uint8_t* keep; // or null
    int32_t* ids;        // each output or null
    float* weights;
    int32_t* pair_row;
    int32_t* offsets;    // null: no grouping
    int32_t* pair_token;
    float* pair_weight;
    uint8_t* counts;     // workspace: rows of experts rounded up to 16
    int64_t stride, tokens;
    int experts, groups, top_groups, group_best, top_k;
    float scale;
    bool f16, sigmoid, renorm, vec;
};
size_t route_workspace(int64_t tokens, int experts);
hipError_t launch_route(const RouteArgs& a, hipStream_t st);

struct QuantizeArgs {
    const void* x;
    int8_t* codes;
    float* scales;
    int64_t stride, rows;
    int k;
    bool f16, vec, vec8;  // rows in runs of four values, of eight
};
hipError_t launch_quantize(const QuantizeArgs& a, hipStream_t st);

// Experts of one call at most.
constexpr int I8_EXPERTS = 1024;
struct GemmI8Args {
    const int8_t *w, *w2;        // [experts][n][k]; w2: the up stack of a gated product, or null
    const float *ws, *ws2;       // [experts][n]
    const int8_t* x;
    const float* xs;
    const int32_t* x_rows;       // or null
    const int32_t* offsets;      // [experts + 1], or null: one product over all rows
    void* y;
    int64_t x_rows_count, rows;  // activation rows, product rows
    int64_t n;
    int k, experts, cus;
    bool y16;
    bool past_caches;            // y is written past the caches
};
hipError_t launch_gemm_i8(const GemmI8Args& a, hipStream_t st);

struct GatherArgs {
    const void* rows;
    const int32_t* pair_row;
    const float* weights;
    const float* residual;  // or null
    float* y;
    int64_t tokens, p_rows, n;
    int top_k;
    bool f16, vec;
};
hipError_t launch_gather(const GatherArgs& a, hipStream_t st);

}  // namespace qmm
