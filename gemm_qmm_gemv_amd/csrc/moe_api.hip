// moe_api.hip -- entry points of expert routing, 8-bit integer products and
// the gather of expert rows: argument checks and launches.  Declarations and
// the contract are in include/qmm.h.  Everything is decided on the host from
// the arguments; no allocation, no synchronization, no state between calls.
#include <hip/hip_runtime.h>

#include <cmath>

#include "api_checks.h"
#include "moe_kernels.h"

using namespace qmm;

namespace {

constexpr int64_t FOUR_GIB = 1LL << 32;

qmm_status check_route(int64_t tokens, int n_experts, int top_k) {
    CHECK(tokens >= 0, QMM_ERR_INVALID_ARGUMENT, "tokens=%lld is negative", (long long)tokens);
    CHECK(tokens < (1LL << 24), QMM_ERR_UNSUPPORTED, "tokens=%lld is 2^24 or more", (long long)tokens);
    CHECK(n_experts >= 1, QMM_ERR_INVALID_ARGUMENT, "n_experts=%d must be positive", n_experts);
    CHECK(n_experts <= 1024, QMM_ERR_UNSUPPORTED, "n_experts=%d above 1024", n_experts);
    CHECK(top_k >= 1 && top_k <= n_experts, QMM_ERR_INVALID_ARGUMENT, "top_k=%d outside 1..n_experts=%d", top_k, n_experts);
    CHECK(top_k <= 64, QMM_ERR_UNSUPPORTED, "top_k=%d above 64", top_k);
    return QMM_OK;
}

// Rows and matrices of 8-bit codes.
qmm_status check_i8(int64_t x_rows_count, int64_t p_rows, int64_t n_experts, int64_t n, int64_t k) {
    CHECK(n >= 0 && p_rows >= 0 && x_rows_count >= 0, QMM_ERR_INVALID_ARGUMENT, "n=%lld, rows=%lld or %lld is negative",
          (long long)n, (long long)p_rows, (long long)x_rows_count);
    CHECK(n_experts >= 0, QMM_ERR_INVALID_ARGUMENT, "n_experts=%lld is negative", (long long)n_experts);
    CHECK(n_experts <= I8_EXPERTS, QMM_ERR_UNSUPPORTED, "n_experts=%lld above %d", (long long)n_experts, I8_EXPERTS);
    CHECK(k >= 32 && k % 32 == 0, QMM_ERR_INVALID_ARGUMENT, "k=%lld must be a positive multiple of 32", (long long)k);
    CHECK(k <= 32768, QMM_ERR_UNSUPPORTED, "k=%lld above 32768", (long long)k);
    CHECK(n < FOUR_GIB / k, QMM_ERR_UNSUPPORTED, "one matrix of %lld x %lld codes is 4 GiB or more", (long long)n, (long long)k);
    CHECK(x_rows_count < FOUR_GIB / k, QMM_ERR_UNSUPPORTED, "%lld rows of %lld codes are 4 GiB or more",
          (long long)x_rows_count, (long long)k);
    CHECK(p_rows < (1LL << 31), QMM_ERR_UNSUPPORTED, "%lld rows are 2^31 or more", (long long)p_rows);
    return QMM_OK;
}

qmm_status i8_product(const int8_t* w, const float* ws, const int8_t* w2, const float* ws2, bool gated, const int8_t* x,
                      const float* xs, const int32_t* x_rows, int64_t x_rows_count, const int32_t* offsets, void* y, bool y16,
                      int64_t p_rows, int64_t n_experts, int64_t n, int64_t k, void* stream, const char* what) {
    qmm_status st = check_i8(x_rows_count, p_rows, n_experts, n, k);
    if (st != QMM_OK) return st;
    CHECK(offsets || n_experts <= 1, QMM_ERR_INVALID_ARGUMENT, "%lld experts without expert_offsets", (long long)n_experts);
    if (n == 0 || p_rows == 0 || n_experts == 0) return report(QMM_OK, "");
    CHECK(w && ws && y && (!gated || (w2 && ws2)), QMM_ERR_INVALID_ARGUMENT, "NULL weights, scales or output");
    CHECK((x && xs) || x_rows_count == 0, QMM_ERR_INVALID_ARGUMENT, "NULL activations or their scales");
    CHECK(x_rows || x_rows_count >= p_rows, QMM_ERR_INVALID_ARGUMENT, "%lld activation rows for %lld rows",
          (long long)x_rows_count, (long long)p_rows);
    CHECK(aligned(w, 16) && aligned(w2, 16) && aligned(x, 16) && aligned(y, 16), QMM_ERR_MISALIGNED,
          "weights, activations or output not 16-byte aligned");
    CHECK(aligned(ws, 4) && aligned(ws2, 4) && aligned(xs, 4) && aligned(x_rows, 4) && aligned(offsets, 4), QMM_ERR_MISALIGNED,
          "scales, x_rows or expert_offsets not 4-byte aligned");
    GemmI8Args a{};
    a.w = w;
    a.w2 = gated ? w2 : nullptr;
    a.ws = ws;
    a.ws2 = ws2;
    a.x = x;
    a.xs = xs;
    a.x_rows = x_rows;
    a.offsets = offsets;
    a.y = y;
    a.x_rows_count = x_rows_count;
    a.rows = p_rows;
    a.n = n;
    a.k = (int)k;
    a.experts = (int)n_experts;
    a.y16 = y16;
    if ((st = current_cus(&a.cus)) != QMM_OK) return st;
    const hipError_t e = launch_gemm_i8(a, static_cast<hipStream_t>(stream));
    CHECK(e != hipErrorInvalidConfiguration, QMM_ERR_UNSUPPORTED, "%lld rows of %lld are more than one launch covers",
          (long long)p_rows, (long long)n);
    return launched(e, what);
}

}  // namespace

extern "C" {

size_t qmm_moe_route_workspace_bytes(int64_t tokens, int n_experts, int top_k) {
    if (check_route(tokens, n_experts, top_k) != QMM_OK) return 0;
    (void)report(QMM_OK, "");
    return route_workspace(tokens, n_experts);
}

qmm_status qmm_moe_route(const void* logits, int logits_fp16, int64_t logits_stride, const float* bias, int sigmoid,
                         int n_groups, int top_groups, int group_best, int top_k, int renormalize, float scale,
                         const uint8_t* keep, int32_t* expert_ids, float* weights, int32_t* pair_row,
                         int32_t* expert_offsets, int32_t* pair_token, float* pair_weight, void* workspace,
                         size_t workspace_bytes, int64_t tokens, int n_experts, void* stream) {
    qmm_status st = check_route(tokens, n_experts, top_k);
    if (st != QMM_OK) return st;
    CHECK(n_groups >= 1 && n_experts % n_groups == 0, QMM_ERR_INVALID_ARGUMENT, "n_experts=%d do not form n_groups=%d",
          n_experts, n_groups);
    CHECK(n_groups <= 64, QMM_ERR_UNSUPPORTED, "n_groups=%d above 64", n_groups);
    CHECK(top_groups >= 1 && top_groups <= n_groups, QMM_ERR_INVALID_ARGUMENT, "top_groups=%d outside 1..n_groups=%d",
          top_groups, n_groups);
    const int each = n_experts / n_groups;
    CHECK(group_best == 1 || group_best == 2, QMM_ERR_INVALID_ARGUMENT, "group_best=%d is neither 1 nor 2", group_best);
    CHECK(n_groups == 1 || group_best <= each, QMM_ERR_INVALID_ARGUMENT, "group_best=%d of groups of %d", group_best, each);
    CHECK(top_groups * each >= top_k, QMM_ERR_INVALID_ARGUMENT, "top_k=%d experts of %d groups of %d", top_k, top_groups, each);
    CHECK(std::isfinite(scale), QMM_ERR_INVALID_ARGUMENT, "scale is not finite");
    CHECK(workspace_bytes == 0 || workspace, QMM_ERR_INVALID_ARGUMENT, "workspace_bytes without a workspace");
    if (tokens == 0 && !expert_offsets) return report(QMM_OK, "");
    if (tokens > 0) {
        CHECK(logits && expert_ids && weights, QMM_ERR_INVALID_ARGUMENT, "NULL logits, expert_ids or weights");
        CHECK(logits_stride >= n_experts || tokens == 1, QMM_ERR_INVALID_ARGUMENT, "logits_stride=%lld is below n_experts=%d",
              (long long)logits_stride, n_experts);
        CHECK(logits_stride < (1LL << 36), QMM_ERR_INVALID_ARGUMENT, "logits_stride of 2^36 or more");
        CHECK(aligned(logits, logits_fp16 ? 2 : 4), QMM_ERR_MISALIGNED, "logits not aligned to their elements");
    }
    CHECK(aligned(bias, 4) && aligned(expert_ids, 4) && aligned(weights, 4) && aligned(pair_row, 4) && aligned(expert_offsets, 4) &&
              aligned(pair_token, 4) && aligned(pair_weight, 4),
          QMM_ERR_MISALIGNED, "bias or an output not 4-byte aligned");
    CHECK(aligned(workspace, 16), QMM_ERR_MISALIGNED, "workspace not 16-byte aligned");
    if (expert_offsets) {
        const size_t need = route_workspace(tokens, n_experts);
        CHECK(workspace_bytes >= need, QMM_ERR_INVALID_ARGUMENT, "workspace of %zu bytes, %zu needed", workspace_bytes, need);
    }
    RouteArgs a{};
    a.logits = logits;
    a.bias = bias;
    a.keep = keep;
    a.ids = expert_ids;
    a.weights = weights;
    a.pair_row = expert_offsets ? pair_row : nullptr;
    a.offsets = expert_offsets;
    a.pair_token = pair_token;
    a.pair_weight = pair_weight;
    a.counts = static_cast<uint8_t*>(workspace);
    a.stride = tokens > 1 ? logits_stride : 0;
    a.tokens = tokens;
    a.experts = n_experts;
    a.groups = n_groups;
    a.top_groups = top_groups;
    a.group_best = group_best;
    a.top_k = top_k;
    a.scale = scale;
    a.f16 = logits_fp16 != 0;
    a.sigmoid = sigmoid != 0;
    a.renorm = renormalize != 0;
    const int size = a.f16 ? 2 : 4;
    a.vec = n_experts % 4 == 0 && a.stride % 4 == 0 && aligned(logits, 4 * size);
    int cus = 0;
    if ((st = current_cus(&cus)) != QMM_OK) return st;
    return launched(launch_route(a, static_cast<hipStream_t>(stream)), "qmm_moe_route");
}

qmm_status qmm_quantize_rows(const void* x, int x_fp16, int64_t x_stride, int8_t* codes, float* scales, int64_t rows,
                             int64_t k, void* stream) {
    CHECK(rows >= 0, QMM_ERR_INVALID_ARGUMENT, "rows=%lld is negative", (long long)rows);
    CHECK(rows < (1LL << 22), QMM_ERR_UNSUPPORTED, "rows=%lld is 2^22 or more", (long long)rows);
    CHECK(k >= 32 && k % 32 == 0, QMM_ERR_INVALID_ARGUMENT, "k=%lld must be a positive multiple of 32", (long long)k);
    CHECK(k <= 32768, QMM_ERR_UNSUPPORTED, "k=%lld above 32768", (long long)k);
    if (rows == 0) return report(QMM_OK, "");
    CHECK(x && codes && scales, QMM_ERR_INVALID_ARGUMENT, "NULL x, codes or scales");
    CHECK(x_stride >= k || rows == 1, QMM_ERR_INVALID_ARGUMENT, "x_stride=%lld is below k=%lld", (long long)x_stride, (long long)k);
    CHECK(x_stride < (1LL << 40), QMM_ERR_INVALID_ARGUMENT, "x_stride of 2^40 or more");
    const int size = x_fp16 ? 2 : 4;
    CHECK(aligned(x, size) && aligned(scales, 4), QMM_ERR_MISALIGNED, "x or scales not aligned to its elements");
    CHECK(aligned(codes, 16), QMM_ERR_MISALIGNED, "codes not 16-byte aligned");
    QuantizeArgs a{};
    a.x = x;
    a.codes = codes;
    a.scales = scales;
    a.stride = rows == 1 ? 0 : x_stride;
    a.rows = rows;
    a.k = (int)k;
    a.f16 = x_fp16 != 0;
    a.vec = a.stride % 4 == 0 && aligned(x, 4 * size);
    a.vec8 = a.stride % 8 == 0 && aligned(x, 16);
    int cus = 0;
    qmm_status st = current_cus(&cus);
    if (st != QMM_OK) return st;
    return launched(launch_quantize(a, static_cast<hipStream_t>(stream)), "qmm_quantize_rows");
}

qmm_status qmm_gemm_i8(const int8_t* w, const float* w_scales, const int8_t* x, const float* x_scales, void* y, int y_fp16,
                       int64_t m, int64_t n, int64_t k, void* stream) {
    return i8_product(w, w_scales, nullptr, nullptr, false, x, x_scales, nullptr, m, nullptr, y, y_fp16 != 0, m, 1, n, k, stream,
                      "qmm_gemm_i8");
}

qmm_status qmm_moe_gemm_i8(const int8_t* w, const float* w_scales, const int8_t* x, const float* x_scales,
                           const int32_t* x_rows, int64_t x_rows_count, const int32_t* expert_offsets, void* y, int y_fp16,
                           int64_t p_rows, int64_t n_experts, int64_t n, int64_t k, void* stream) {
    return i8_product(w, w_scales, nullptr, nullptr, false, x, x_scales, x_rows, x_rows_count, expert_offsets, y, y_fp16 != 0, p_rows,
                      n_experts, n, k, stream, "qmm_moe_gemm_i8");
}

qmm_status qmm_moe_swiglu_i8(const int8_t* gate_w, const float* gate_scales, const int8_t* up_w, const float* up_scales,
                             const int8_t* x, const float* x_scales, const int32_t* x_rows, int64_t x_rows_count,
                             const int32_t* expert_offsets, void* h, int h_fp16, int64_t p_rows, int64_t n_experts,
                             int64_t n, int64_t k, void* stream) {
    return i8_product(gate_w, gate_scales, up_w, up_scales, true, x, x_scales, x_rows, x_rows_count, expert_offsets, h, h_fp16 != 0,
                      p_rows, n_experts, n, k, stream, "qmm_moe_swiglu_i8");
}

qmm_status qmm_moe_gather(const void* rows, int rows_fp16, const int32_t* pair_row, const float* weights,
                          const float* residual, float* y, int64_t tokens, int top_k, int64_t p_rows, int64_t n, void* stream) {
    CHECK(tokens >= 0 && n >= 0 && p_rows >= 0, QMM_ERR_INVALID_ARGUMENT, "tokens=%lld, p_rows=%lld or n=%lld is negative",
          (long long)tokens, (long long)p_rows, (long long)n);
    CHECK(top_k >= 0, QMM_ERR_INVALID_ARGUMENT, "top_k=%d is negative", top_k);
    CHECK(top_k <= 64, QMM_ERR_UNSUPPORTED, "top_k=%d above 64", top_k);
    CHECK(tokens < (1LL << 24), QMM_ERR_UNSUPPORTED, "tokens=%lld is 2^24 or more", (long long)tokens);
    CHECK(n < (1LL << 22), QMM_ERR_UNSUPPORTED, "n=%lld is 2^22 or more", (long long)n);
    CHECK(p_rows < (1LL << 31), QMM_ERR_UNSUPPORTED, "p_rows=%lld is 2^31 or more", (long long)p_rows);
    if (tokens == 0 || n == 0) return report(QMM_OK, "");
    CHECK(y && ((pair_row && weights) || top_k == 0), QMM_ERR_INVALID_ARGUMENT, "NULL y, pair_row or weights");
    CHECK(rows || p_rows == 0 || top_k == 0, QMM_ERR_INVALID_ARGUMENT, "NULL rows");
    CHECK(aligned(rows, rows_fp16 ? 2 : 4) && aligned(pair_row, 4) && aligned(weights, 4) && aligned(residual, 4) && aligned(y, 4),
          QMM_ERR_MISALIGNED, "an array is not aligned to its elements");
    GatherArgs a{};
    a.rows = rows;
    a.pair_row = pair_row;
    a.weights = weights;
    a.residual = residual;
    a.y = y;
    a.tokens = tokens;
    a.p_rows = p_rows;
    a.n = n;
    a.top_k = top_k;
    a.f16 = rows_fp16 != 0;
    a.vec = n % (rows_fp16 ? 8 : 4) == 0 && aligned(rows, 16) && aligned(residual, 16) && aligned(y, 16);
    int cus = 0;
    qmm_status st = current_cus(&cus);
    if (st != QMM_OK) return st;
    return launched(launch_gather(a, static_cast<hipStream_t>(stream)), "qmm_moe_gather");
}

}  // extern "C"
