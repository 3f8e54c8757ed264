// layer_kernels.h -- host-side interface between the entry points of the
// attention half of a decoder layer (layer_api.hip) and their kernel files.
// Internal to the library; not installed.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/qmm.h"

namespace qmm {

// Sets the calling thread's qmm_last_error text and returns st (qmm_api.hip).
qmm_status report(qmm_status st, const char* fmt, ...);

struct NormArgs {
    const void* y;        // block output, fp32 or fp16, or null
    const float* post;    // weight of the norm on y, or null (no norm)
    const float* gate;    // multiplies y, or null
    const float* res;     // residual, or null (zero)
    const float* pre;     // weight of the norm that x gets, or null (one)
    float* h;             // residual stream, or null
    void* x;              // fp16 input of the next product, or null
    int64_t y_stride, gate_stride;
    int64_t rows;
    int n;
    float scale, eps;
    bool y_fp16, vec;
};
hipError_t launch_norm(const NormArgs& a, hipStream_t st);

struct CacheView {
    void *k, *ks, *km, *v, *vs, *vm;
    int64_t pages;
    int kv_heads, head_dim, page_shift, bits, group;
};

struct AppendArgs {
    CacheView c;
    const void *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;
    const float *q_norm, *k_norm, *inv_freq;
    float eps;
    int rot;
    const int32_t* positions;
    const int64_t* slots;
    void *q_out, *k_out, *v_out;
    int64_t tokens;
    int q_heads, cus;
    bool in_fp16, interleaved, out_cached;
};
hipError_t launch_append(const AppendArgs& a, hipStream_t st);

// qmm_attn_cache's work is cut into units (sequence, kv head, tile of 16 query
// rows) and those into steps of CACHE_STEP cached rows.
constexpr int CACHE_STEP = 128;
// Work-groups of its kernel that one compute unit holds.
constexpr int cache_resident(int bits, int head_dim) {
    return head_dim == 64 ? 4 : bits == 4 ? 3 : 2;
}
struct CacheAttnArgs {
    CacheView c;
    const void* q;
    const int32_t *table, *lens;
    int64_t table_stride;
    void* out;
    int* count;   // [groups] runs handed in, zero between calls
    float* part;  // [groups][2] sums of runs, [16][head_dim + 2] each
    int64_t n_seqs;
    int max_len, q_len, q_heads;
    int group;      // query heads per kv head
    int row_tiles;  // units per kv head
    float scale;
    int64_t groups;  // work-groups
    bool share;      // they share all steps evenly; else one unit each
};
hipError_t launch_attn_cache(const CacheAttnArgs& a, hipStream_t st);

struct PromptArgs {
    const void *q, *k, *v;
    void* out;
    const int32_t* offsets;
    int64_t tokens, n_seqs, q_stride, k_stride, v_stride, out_stride;
    int q_heads, kv_heads, head_dim;
    float scale;
    int cus;
};
hipError_t launch_attn_prompt(const PromptArgs& a, hipStream_t st);

}  // namespace qmm
