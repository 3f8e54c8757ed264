// layer_api.hip -- entry points of the attention half of a decoder layer:
// argument checks, launch plans and launches.  Declarations and the contract
// are in include/qmm.h.  Everything is decided on the host from the arguments;
// no allocation, no synchronization, no state between calls.
#include <hip/hip_runtime.h>

#include <climits>
#include <cmath>
#include <cstring>

#include "api_checks.h"
#include "layer_kernels.h"

using namespace qmm;

namespace {

constexpr int64_t MAX_BLOCKS = (1LL << 24) - 1;  // of 256 threads: HIP counts a launch's threads in 32 bits

qmm_status check_head_dim(int d) {
    CHECK(d > 0, QMM_ERR_INVALID_ARGUMENT, "head_dim=%d must be positive", d);
    CHECK(d == 64 || d == 128, QMM_ERR_UNSUPPORTED, "head_dim=%d not built (64 and 128 are)", d);
    return QMM_OK;
}

qmm_status check_heads(int q_heads, int kv_heads, bool q_required) {
    CHECK(kv_heads >= 1 && kv_heads <= 4096, QMM_ERR_INVALID_ARGUMENT, "kv_heads=%d outside 1..4096", kv_heads);
    CHECK(q_heads >= (q_required ? 1 : 0) && q_heads <= 4096, QMM_ERR_INVALID_ARGUMENT, "q_heads=%d outside %d..4096",
          q_heads, q_required ? 1 : 0);
    return QMM_OK;
}

// The kernels form scale * log2(e), over a cache of codes 2^24 times that, and
// products with scores in fp32: far above any use, infinities would come out.
qmm_status check_scale(float scale) {
    CHECK(std::isfinite(scale), QMM_ERR_INVALID_ARGUMENT, "scale is not finite");
    CHECK(std::fabs(scale) <= 18446744073709551616.f, QMM_ERR_UNSUPPORTED, "scale=%g is beyond 2^64", (double)scale);
    return QMM_OK;
}

// The cache's shape; its arrays too if they are going to be used.
qmm_status check_cache(const qmm_kv_cache* c, bool arrays) {
    CHECK(c, QMM_ERR_INVALID_ARGUMENT, "NULL cache");
    qmm_status st = check_head_dim(c->head_dim);
    if (st != QMM_OK) return st;
    CHECK(c->kv_heads >= 1 && c->kv_heads <= 4096, QMM_ERR_INVALID_ARGUMENT, "kv_heads=%d outside 1..4096", c->kv_heads);
    const int b = c->bits;
    CHECK(b == 16 || (b >= 2 && b <= 8), QMM_ERR_INVALID_ARGUMENT, "bits=%d is neither 2..8 nor 16 (fp16)", b);
    CHECK(b == 4 || b == 8 || b == 16, QMM_ERR_UNSUPPORTED, "a cache of %d bits is not built (4, 8 and 16 are)", b);
    if (b != 16) {
        const int g = c->group_size;
        CHECK(g > 0 && g % 32 == 0 && c->head_dim % g == 0, QMM_ERR_INVALID_ARGUMENT,
              "group_size=%d must be a multiple of 32 that divides head_dim=%d", g, c->head_dim);
    }
    const int p = c->page_size;
    CHECK(p > 0, QMM_ERR_INVALID_ARGUMENT, "page_size=%d must be positive", p);
    CHECK(p >= 16 && p <= 65536 && (p & (p - 1)) == 0, QMM_ERR_UNSUPPORTED,
          "page_size=%d is not a power of two from 16 to 65536", p);
    CHECK(c->pages >= 0 && c->pages <= 0x7fffffff, QMM_ERR_INVALID_ARGUMENT, "pages=%lld outside 0..2^31-1",
          (long long)c->pages);
    CHECK((double)c->pages * c->kv_heads * p * c->head_dim * 2 < 4e18, QMM_ERR_INVALID_ARGUMENT,
          "a cache of %lld pages is beyond 64-bit offsets", (long long)c->pages);
    if (!arrays) return QMM_OK;
    CHECK(c->k && c->v, QMM_ERR_INVALID_ARGUMENT, "NULL cache rows");
    CHECK(aligned(c->k, 16) && aligned(c->v, 16), QMM_ERR_MISALIGNED, "cache rows not 16-byte aligned");
    if (b != 16) {
        CHECK(c->k_scales && c->k_mins && c->v_scales && c->v_mins, QMM_ERR_INVALID_ARGUMENT, "NULL cache scales or mins");
        CHECK(aligned(c->k_scales, 16) && aligned(c->k_mins, 16) && aligned(c->v_scales, 16) && aligned(c->v_mins, 16),
              QMM_ERR_MISALIGNED, "cache scales or mins not 16-byte aligned");
    }
    return QMM_OK;
}

CacheView view(const qmm_kv_cache* c) {
    int shift = 0;
    while ((1 << shift) < c->page_size) ++shift;
    return CacheView{c->k, c->k_scales, c->k_mins, c->v, c->v_scales, c->v_mins, c->pages, c->kv_heads, c->head_dim,
                     shift, c->bits, c->group_size};
}

// A block of token rows: pointer, stride and width in elements of `size` bytes.
qmm_status check_rows(const char* name, const void* p, int64_t stride, int64_t width, int size) {
    CHECK(p, QMM_ERR_INVALID_ARGUMENT, "NULL %s", name);
    CHECK(stride >= width && stride < (1LL << 40), QMM_ERR_INVALID_ARGUMENT, "%s stride %lld is below its width %lld",
          name, (long long)stride, (long long)width);
    CHECK(aligned(p, 16) && stride * size % 16 == 0, QMM_ERR_MISALIGNED, "%s rows not 16-byte aligned", name);
    return QMM_OK;
}

// How qmm_attn_cache is cut: as many work-groups as the device holds at once
// share all steps evenly.  The sums of runs that
// begin or end inside a unit need workspace; without enough of it every unit
// gets a work-group of its own.
constexpr int64_t COUNTERS = QMM_ATTN_COUNTER_BYTES / 4;

struct CachePlan {
    int64_t groups;
    bool share;
    int row_tiles;
    size_t bytes;  // of workspace, if shared
};

size_t share_bytes(int64_t groups, int head_dim) {
    return (size_t)(QMM_ATTN_COUNTER_BYTES + groups * 2 * 16 * (head_dim + 2) * 4);
}

CachePlan plan_attn_cache(const qmm_kv_cache* c, int64_t n_seqs, int q_len, int q_heads, int64_t max_len, int cus,
                          size_t ws_bytes) {
    CachePlan p;
    p.row_tiles = (q_len * (q_heads / c->kv_heads) + 15) / 16;
    const int64_t units = n_seqs * c->kv_heads * p.row_tiles;
    const int64_t steps = units * ((max_len + CACHE_STEP - 1) / CACHE_STEP);  // at most
    p.groups = (int64_t)cus * cache_resident(c->bits, c->head_dim);
    if (p.groups > COUNTERS) p.groups = COUNTERS;
    if (p.groups > steps) p.groups = steps;
    while (p.groups > 0 && share_bytes(p.groups, c->head_dim) > ws_bytes) p.groups = p.groups * 3 / 4;
    p.bytes = share_bytes(p.groups, c->head_dim);
    // One run per unit: units of one step, no workspace to speak of, or more
    // steps than 32 bits count.
    p.share = max_len > CACHE_STEP && p.groups > units / 8 + 1 && steps < (1 << 28);
    if (!p.share) p.groups = units;
    return p;
}

qmm_status check_attn_cache(const qmm_kv_cache* c, bool arrays, int64_t n_seqs, int q_len, int q_heads, int64_t max_len) {
    qmm_status st = check_cache(c, arrays);
    if (st != QMM_OK) return st;
    if ((st = check_heads(q_heads, c->kv_heads, true)) != QMM_OK) return st;
    CHECK(q_heads % c->kv_heads == 0, QMM_ERR_INVALID_ARGUMENT, "q_heads=%d is not a multiple of kv_heads=%d", q_heads,
          c->kv_heads);
    CHECK(q_len >= 1 && q_len <= 256, QMM_ERR_INVALID_ARGUMENT, "q_len=%d outside 1..256", q_len);
    CHECK(n_seqs >= 0, QMM_ERR_INVALID_ARGUMENT, "n_seqs=%lld is negative", (long long)n_seqs);
    CHECK(max_len >= 0 && max_len < (1LL << 30), QMM_ERR_INVALID_ARGUMENT, "max_kv_len=%lld outside 0..2^30-1",
          (long long)max_len);
    const int64_t tiles = (q_len * (q_heads / c->kv_heads) + 15) / 16;
    CHECK(n_seqs <= MAX_BLOCKS && (n_seqs * c->kv_heads + 7) * tiles <= MAX_BLOCKS && n_seqs * q_len * q_heads / 4 < MAX_BLOCKS,
          QMM_ERR_UNSUPPORTED, "%lld sequences of %d x %d query rows are more than one launch covers", (long long)n_seqs,
          q_len, q_heads);
    return QMM_OK;
}

// Arguments of qmm_call_words.
struct Words {
    int64_t w[24];
    // What no int holds becomes one that every check refuses.
    int i(int k) const { return w[k] > INT_MAX ? INT_MAX : w[k] < INT_MIN ? INT_MIN : (int)w[k]; }
    float f(int k) const {
        double d;
        std::memcpy(&d, &w[k], 8);
        return (float)d;
    }
    template <class T = void>
    T* p(int k) const {
        return reinterpret_cast<T*>(w[k]);
    }
};

}  // namespace

extern "C" {

qmm_status qmm_norm_residual(const void* y, int y_fp16, int64_t y_stride, const float* post_weight, const float* gate,
                             int64_t gate_stride, float scale, const float* residual, float* h, const float* pre_weight,
                             void* x, int64_t rows, int64_t n, float eps, void* stream) {
    CHECK(rows >= 0 && n >= 0, QMM_ERR_INVALID_ARGUMENT, "rows=%lld or n=%lld is negative", (long long)rows, (long long)n);
    CHECK(eps >= 0.f && std::isfinite(eps), QMM_ERR_INVALID_ARGUMENT, "eps must be finite and not negative");
    CHECK(n <= 32768, QMM_ERR_UNSUPPORTED, "n=%lld above 32768", (long long)n);
    CHECK(rows < (1LL << 22), QMM_ERR_UNSUPPORTED, "rows=%lld is 2^22 or more", (long long)rows);
    if (rows == 0 || n == 0) return report(QMM_OK, "");
    CHECK(y || residual, QMM_ERR_INVALID_ARGUMENT, "neither y nor residual");
    CHECK(y ? (h || x) : x != nullptr, QMM_ERR_INVALID_ARGUMENT, "no output");
    const int ysize = y_fp16 ? 2 : 4;
    if (y) {
        CHECK(y_stride >= n || rows == 1, QMM_ERR_INVALID_ARGUMENT, "y_stride=%lld is below n=%lld", (long long)y_stride,
              (long long)n);
        CHECK(!gate || gate_stride == 0 || gate_stride >= n || rows == 1, QMM_ERR_INVALID_ARGUMENT,
              "gate_stride=%lld is neither 0 nor at least n=%lld", (long long)gate_stride, (long long)n);
        CHECK(y_stride < (1LL << 40) && gate_stride < (1LL << 40), QMM_ERR_INVALID_ARGUMENT, "stride of 2^40 or more");
        CHECK(aligned(y, ysize), QMM_ERR_MISALIGNED, "y not aligned to its elements");
    }
    CHECK(aligned(post_weight, 4) && aligned(gate, 4) && aligned(residual, 4) && aligned(h, 4) && aligned(pre_weight, 4),
          QMM_ERR_MISALIGNED, "fp32 array not 4-byte aligned");
    CHECK(aligned(x, 2), QMM_ERR_MISALIGNED, "x not 2-byte aligned");
    NormArgs a{};
    a.y = y;
    a.post = y ? post_weight : nullptr;
    a.gate = y ? gate : nullptr;
    a.res = residual;
    a.pre = pre_weight;
    a.h = y ? h : nullptr;
    a.x = x;
    a.y_stride = rows == 1 ? 0 : y_stride;
    a.gate_stride = rows == 1 ? 0 : gate_stride;
    a.rows = rows;
    a.n = (int)n;
    a.scale = scale;
    a.eps = eps;
    a.y_fp16 = y_fp16 != 0;
    // Runs of four: every row of every array starts on a 16-byte boundary
    // (8 for fp16).
    a.vec = n % 4 == 0 && a.y_stride % 4 == 0 && a.gate_stride % 4 == 0 && aligned(y, 4 * ysize) && aligned(a.post, 16) &&
            aligned(a.gate, 16) && aligned(residual, 16) && aligned(a.h, 16) && aligned(pre_weight, 16) && aligned(x, 8);
    int cus = 0;
    qmm_status st = current_cus(&cus);
    if (st != QMM_OK) return st;
    return launched(launch_norm(a, static_cast<hipStream_t>(stream)), "qmm_norm_residual");
}

qmm_status qmm_kv_append(const qmm_kv_cache* cache, const void* q, const void* k, const void* v, int in_fp16,
                         int64_t q_stride, int64_t k_stride, int64_t v_stride, const float* q_norm, const float* k_norm,
                         float eps, const float* inv_freq, int rot_dim, int interleaved, const int32_t* positions,
                         const int64_t* slots, void* q_out, void* k_out, void* v_out, int out_cached, int64_t tokens,
                         int q_heads, void* stream) {
    qmm_status st = check_cache(cache, slots != nullptr && tokens > 0);
    if (st != QMM_OK) return st;
    if ((st = check_heads(q_heads, cache->kv_heads, false)) != QMM_OK) return st;
    const int d = cache->head_dim;
    CHECK(rot_dim >= 0 && rot_dim <= d && rot_dim % 16 == 0, QMM_ERR_INVALID_ARGUMENT,
          "rot_dim=%d must be a multiple of 16 within 0..head_dim=%d", rot_dim, d);
    CHECK(eps >= 0.f && std::isfinite(eps), QMM_ERR_INVALID_ARGUMENT, "eps must be finite and not negative");
    CHECK(tokens >= 0, QMM_ERR_INVALID_ARGUMENT, "tokens=%lld is negative", (long long)tokens);
    CHECK(tokens < (1LL << 24), QMM_ERR_UNSUPPORTED, "tokens=%lld is 2^24 or more", (long long)tokens);
    if (tokens == 0) return report(QMM_OK, "");
    const int size = in_fp16 ? 2 : 4;
    if (q_heads > 0) {
        if ((st = check_rows("q", q, q_stride, (int64_t)q_heads * d, size)) != QMM_OK) return st;
        CHECK(q_out, QMM_ERR_INVALID_ARGUMENT, "NULL q_out");
    }
    if ((st = check_rows("k", k, k_stride, (int64_t)cache->kv_heads * d, size)) != QMM_OK) return st;
    if ((st = check_rows("v", v, v_stride, (int64_t)cache->kv_heads * d, size)) != QMM_OK) return st;
    CHECK(aligned(q_out, 16) && aligned(k_out, 16) && aligned(v_out, 16), QMM_ERR_MISALIGNED,
          "q_out, k_out or v_out not 16-byte aligned");
    CHECK(rot_dim == 0 || (inv_freq && positions), QMM_ERR_INVALID_ARGUMENT, "NULL inv_freq or positions");
    CHECK(aligned(q_norm, 4) && aligned(k_norm, 4) && aligned(inv_freq, 4) && aligned(positions, 4) && aligned(slots, 8),
          QMM_ERR_MISALIGNED, "norm weights, inv_freq, positions or slots not aligned to their elements");
    AppendArgs a{};
    a.c = view(cache);
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.q_norm = q_norm;
    a.k_norm = k_norm;
    a.inv_freq = inv_freq;
    a.eps = eps;
    a.rot = rot_dim;
    a.positions = positions;
    a.slots = slots;
    a.q_out = q_out;
    a.k_out = k_out;
    a.v_out = v_out;
    a.tokens = tokens;
    a.q_heads = q_heads;
    a.in_fp16 = in_fp16 != 0;
    a.interleaved = interleaved != 0;
    a.out_cached = out_cached != 0;
    if ((st = current_cus(&a.cus)) != QMM_OK) return st;
    return launched(launch_append(a, static_cast<hipStream_t>(stream)), "qmm_kv_append");
}

size_t qmm_attn_cache_workspace_bytes(const qmm_kv_cache* cache, int64_t n_seqs, int q_len, int q_heads,
                                      int64_t max_kv_len) {
    if (check_attn_cache(cache, false, n_seqs, q_len, q_heads, max_kv_len) != QMM_OK || n_seqs == 0) return 0;
    int cus = 0;
    if (current_cus(&cus) != QMM_OK) cus = 256;
    (void)report(QMM_OK, "");
    const CachePlan plan = plan_attn_cache(cache, n_seqs, q_len, q_heads, max_kv_len, cus, SIZE_MAX);
    return plan.share ? plan.bytes : 0;
}

qmm_status qmm_attn_cache(const qmm_kv_cache* cache, const void* q, const int32_t* page_table, int64_t table_stride,
                          const int32_t* kv_lens, int64_t max_kv_len, void* out, int64_t n_seqs, int q_len, int q_heads,
                          float scale, void* workspace, size_t workspace_bytes, void* stream) {
    qmm_status st = check_attn_cache(cache, n_seqs > 0, n_seqs, q_len, q_heads, max_kv_len);
    if (st != QMM_OK) return st;
    if ((st = check_scale(scale)) != QMM_OK) return st;
    CHECK(workspace_bytes == 0 || workspace, QMM_ERR_INVALID_ARGUMENT, "workspace_bytes without a workspace");
    CHECK(aligned(workspace, 16), QMM_ERR_MISALIGNED, "workspace not 16-byte aligned");
    CHECK(table_stride >= 0 && table_stride < (1LL << 40), QMM_ERR_INVALID_ARGUMENT, "table_stride=%lld out of range",
          (long long)table_stride);
    CHECK((double)table_stride * cache->page_size >= (double)max_kv_len, QMM_ERR_INVALID_ARGUMENT,
          "%lld pages of %d rows cannot hold max_kv_len=%lld", (long long)table_stride, cache->page_size,
          (long long)max_kv_len);
    if (n_seqs == 0) return report(QMM_OK, "");
    CHECK(q && out && kv_lens && (page_table || max_kv_len == 0), QMM_ERR_INVALID_ARGUMENT,
          "NULL q, out, kv_lens or page_table");
    CHECK(cache->pages > 0 || max_kv_len == 0, QMM_ERR_INVALID_ARGUMENT, "a cache without pages");
    CHECK(aligned(q, 16) && aligned(out, 16), QMM_ERR_MISALIGNED, "q or out not 16-byte aligned");
    CHECK(aligned(page_table, 4) && aligned(kv_lens, 4), QMM_ERR_MISALIGNED, "page_table or kv_lens not 4-byte aligned");
    int cus = 0;
    if ((st = current_cus(&cus)) != QMM_OK) return st;
    CacheAttnArgs a{};
    a.c = view(cache);
    a.q = q;
    a.table = page_table;
    a.lens = kv_lens;
    a.table_stride = table_stride;
    a.out = out;
    a.count = static_cast<int*>(workspace);
    a.part = static_cast<float*>(workspace) + COUNTERS;
    a.n_seqs = n_seqs;
    a.max_len = (int)max_kv_len;
    a.q_len = q_len;
    a.q_heads = q_heads;
    a.scale = scale;
    const CachePlan plan = plan_attn_cache(cache, n_seqs, q_len, q_heads, max_kv_len, cus, workspace_bytes);
    a.group = q_heads / cache->kv_heads;
    a.row_tiles = plan.row_tiles;
    a.groups = plan.groups;
    a.share = plan.share;
    return launched(launch_attn_cache(a, static_cast<hipStream_t>(stream)), "qmm_attn_cache");
}

qmm_status qmm_attn_prompt(const void* q, const void* k, const void* v, const int32_t* seq_offsets, void* out,
                           int64_t tokens, int64_t n_seqs, int q_heads, int kv_heads, int head_dim, int64_t q_stride,
                           int64_t k_stride, int64_t v_stride, int64_t out_stride, float scale, void* stream) {
    qmm_status st = check_head_dim(head_dim);
    if (st != QMM_OK) return st;
    if ((st = check_heads(q_heads, kv_heads, true)) != QMM_OK) return st;
    CHECK(q_heads % kv_heads == 0, QMM_ERR_INVALID_ARGUMENT, "q_heads=%d is not a multiple of kv_heads=%d", q_heads,
          kv_heads);
    if ((st = check_scale(scale)) != QMM_OK) return st;
    CHECK(tokens >= 0 && n_seqs >= 0 && n_seqs < 0x7ffffffe, QMM_ERR_INVALID_ARGUMENT, "tokens=%lld or n_seqs=%lld out of range",
          (long long)tokens, (long long)n_seqs);
    CHECK(tokens <= 65535 * 128 && (tokens + 127) / 128 * q_heads <= MAX_BLOCKS, QMM_ERR_UNSUPPORTED,
          "tokens=%lld with %d heads are more than one launch covers", (long long)tokens, q_heads);
    if (tokens == 0 || n_seqs == 0) return report(QMM_OK, "");
    if ((st = check_rows("q", q, q_stride, (int64_t)q_heads * head_dim, 2)) != QMM_OK) return st;
    if ((st = check_rows("k", k, k_stride, (int64_t)kv_heads * head_dim, 2)) != QMM_OK) return st;
    if ((st = check_rows("v", v, v_stride, (int64_t)kv_heads * head_dim, 2)) != QMM_OK) return st;
    if ((st = check_rows("out", out, out_stride, (int64_t)q_heads * head_dim, 2)) != QMM_OK) return st;
    // The kernel addresses 64 rows of k and v at a time with 32-bit offsets.
    CHECK(k_stride < (1 << 23) && v_stride < (1 << 23), QMM_ERR_UNSUPPORTED, "k or v stride of 2^23 elements or more");
    CHECK(seq_offsets, QMM_ERR_INVALID_ARGUMENT, "NULL seq_offsets");
    CHECK(aligned(seq_offsets, 4), QMM_ERR_MISALIGNED, "seq_offsets not 4-byte aligned");
    int cus = 0;
    if ((st = current_cus(&cus)) != QMM_OK) return st;
    PromptArgs a{q, k, v, out, seq_offsets, tokens, n_seqs, q_stride, k_stride, v_stride, out_stride, q_heads, kv_heads,
                 head_dim, scale, cus};
    return launched(launch_attn_prompt(a, static_cast<hipStream_t>(stream)), "qmm_attn_prompt");
}

qmm_status qmm_call_words(int call, const void* words) {
    CHECK(words, QMM_ERR_INVALID_ARGUMENT, "NULL words");
    Words a;
    switch (call) {
        case QMM_CALL_NORM_RESIDUAL:
            std::memcpy(a.w, words, 15 * 8);
            return qmm_norm_residual(a.p(0), a.i(1), a.w[2], a.p<float>(3), a.p<float>(4), a.w[5], a.f(6), a.p<float>(7),
                                     a.p<float>(8), a.p<float>(9), a.p(10), a.w[11], a.w[12], a.f(13), a.p(14));
        case QMM_CALL_KV_APPEND:
            std::memcpy(a.w, words, 23 * 8);
            return qmm_kv_append(a.p<qmm_kv_cache>(0), a.p(1), a.p(2), a.p(3), a.i(4), a.w[5], a.w[6], a.w[7],
                                 a.p<float>(8), a.p<float>(9), a.f(10), a.p<float>(11), a.i(12), a.i(13),
                                 a.p<int32_t>(14), a.p<int64_t>(15), a.p(16), a.p(17), a.p(18), a.i(19), a.w[20],
                                 a.i(21), a.p(22));
        case QMM_CALL_ATTN_CACHE:
            std::memcpy(a.w, words, 14 * 8);
            return qmm_attn_cache(a.p<qmm_kv_cache>(0), a.p(1), a.p<int32_t>(2), a.w[3], a.p<int32_t>(4), a.w[5], a.p(6),
                                  a.w[7], a.i(8), a.i(9), a.f(10), a.p(11), (size_t)a.w[12], a.p(13));
        case QMM_CALL_ATTN_PROMPT:
            std::memcpy(a.w, words, 16 * 8);
            return qmm_attn_prompt(a.p(0), a.p(1), a.p(2), a.p<int32_t>(3), a.p(4), a.w[5], a.w[6], a.i(7), a.i(8), a.i(9),
                                   a.w[10], a.w[11], a.w[12], a.w[13], a.f(14), a.p(15));
        case QMM_CALL_MOE_ROUTE:
            std::memcpy(a.w, words, 23 * 8);
            return qmm_moe_route(a.p(0), a.i(1), a.w[2], a.p<float>(3), a.i(4), a.i(5), a.i(6), a.i(7), a.i(8), a.i(9),
                                 a.f(10), a.p<uint8_t>(11), a.p<int32_t>(12), a.p<float>(13), a.p<int32_t>(14),
                                 a.p<int32_t>(15), a.p<int32_t>(16), a.p<float>(17), a.p(18), (size_t)a.w[19], a.w[20],
                                 a.i(21), a.p(22));
        case QMM_CALL_QUANTIZE_ROWS:
            std::memcpy(a.w, words, 8 * 8);
            return qmm_quantize_rows(a.p(0), a.i(1), a.w[2], a.p<int8_t>(3), a.p<float>(4), a.w[5], a.w[6], a.p(7));
        case QMM_CALL_GEMM_I8:
            std::memcpy(a.w, words, 10 * 8);
            return qmm_gemm_i8(a.p<int8_t>(0), a.p<float>(1), a.p<int8_t>(2), a.p<float>(3), a.p(4), a.i(5), a.w[6], a.w[7],
                               a.w[8], a.p(9));
        case QMM_CALL_MOE_GEMM_I8:
            std::memcpy(a.w, words, 14 * 8);
            return qmm_moe_gemm_i8(a.p<int8_t>(0), a.p<float>(1), a.p<int8_t>(2), a.p<float>(3), a.p<int32_t>(4), a.w[5],
                                   a.p<int32_t>(6), a.p(7), a.i(8), a.w[9], a.w[10], a.w[11], a.w[12], a.p(13));
        case QMM_CALL_MOE_SWIGLU_I8:
            std::memcpy(a.w, words, 16 * 8);
            return qmm_moe_swiglu_i8(a.p<int8_t>(0), a.p<float>(1), a.p<int8_t>(2), a.p<float>(3), a.p<int8_t>(4),
                                     a.p<float>(5), a.p<int32_t>(6), a.w[7], a.p<int32_t>(8), a.p(9), a.i(10), a.w[11],
                                     a.w[12], a.w[13], a.w[14], a.p(15));
        case QMM_CALL_MOE_GATHER:
            std::memcpy(a.w, words, 11 * 8);
            return qmm_moe_gather(a.p(0), a.i(1), a.p<int32_t>(2), a.p<float>(3), a.p<float>(4), a.p<float>(5), a.w[6], a.i(7),
                                  a.w[8], a.w[9], a.p(10));
    }
    return report(QMM_ERR_INVALID_ARGUMENT, "call=%d is none of QMM_CALL_*", call);
}

}  // extern "C"
