/*
 * qmm.h -- quantized matrix products with inline dequantization, for AMD
 * Instinct MI355X (gfx950).  Plain C ABI: no HIP, torch or C++ types.
 *
 * The operation (from the pages):
 *   Weights are stored with affine quantization at 2 to 8 bits per weight
 *   ("Apple Silicon 로컬 LLM 추론의 새 기준 BaseRT" (thakicloud.com), section
 *   "BaseRT는 무엇인가").  Decode multiplies one activation row by the
 *   weights with a dedicated GEMV (M = 1) and prefill several rows with a
 *   GEMM (M > 1); dequantization happens inside the compute loop, so full
 *   precision weights never go to memory and memory traffic scales with the
 *   compressed size ("BaseRT claims fastest Apple Silicon inference"
 *   (thetesserapress.com), section "What BaseRT does differently"; "BaseRT:
 *   Best-in-Class LLM Inference on Apple Silicon via Native Metal"
 *   (gist.science summary), section "Metodologia", per-format GEMV/GEMM
 *   variants with dequantization in the inner loop).
 *
 * Format (the pages fix none of these details; this is the library's format):
 *   W is N x K (output rows x reduction).  Codes are unsigned b-bit integers,
 *   b in {2, 3, 4, 5, 6, 8}.  Row n is a little-endian bitstream of K*b bits held
 *   in K*b/32 uint32 words: code k occupies stream bits [k*b, k*b + b), and
 *   stream bit i is bit (i mod 32) of word floor(i / 32) of the row.  Rows are
 *   contiguous (row n starts at word n*K*b/32).
 *   Each run of `group_size` consecutive k of a row shares one fp16 scale s
 *   and one fp16 min m, stored as two arrays [N][K/group_size] row-major.
 *   The weight is w[n][k] = s[n][k/group_size] * q[n][k] + m[n][k/group_size].
 *   Activations x are fp16 [M][K] row-major; outputs y are fp32 [M][N]
 *   row-major:  y[i][n] = sum_k w[n][k] * x[i][k].
 *   bits = 16 is the unquantized format ("FP16"/"Q16" in the per-format
 *   kernel lists of the pages above): w_packed holds the fp16 weights
 *   themselves, K/2 words per row, word j holding k = 2j in its low 16 bits
 *   and k = 2j + 1 in its high 16 bits.  Scales and mins are not read and may
 *   be NULL; group_size is still checked as above.  qmm_unpack rejects it
 *   (QMM_ERR_UNSUPPORTED), and a batched launch covers K <= 4096 at 16 bits.
 *
 * Requirements checked on the host before anything is launched:
 *   bits in {2, 3, 4, 5, 6, 8, 16} (7 is QMM_ERR_UNSUPPORTED); group_size a
 *   positive multiple of 32;
 *   k >= 32 and k a multiple of group_size; n >= 0, m >= 0 (0 is a no-op);
 *   weight, activation and output pointers 16-byte aligned; scale and min
 *   pointers 2-byte aligned; non-NULL pointers wherever work is to be done.
 *   One packed matrix (one expert of a stack) and one activation block must
 *   each stay below 4 GiB, else QMM_ERR_UNSUPPORTED (the kernels address
 *   them with 32-bit offsets); so must one output block.
 *   A failed check returns a status, writes nothing and launches nothing;
 *   qmm_last_error() then holds a one-line explanation (thread-local).
 *
 * Memory and streams:
 *   Every pointer argument except those marked "host" is a device pointer,
 *   owned by the caller.  The library allocates no device memory, frees none
 *   and keeps no per-call state.  Calls are asynchronous on `stream`
 *   (a hipStream_t passed as void*; NULL means the null stream); a kernel
 *   fault shows up at the caller's next synchronization.  Results are
 *   deterministic -- every output element is summed in a fixed order that
 *   depends only on the shape and the launch plan -- except for
 *   qmm_moe_combine, whose float atomic adds into a token's row happen in
 *   no fixed order.  The one exception to "allocates nothing" is
 *   qmm_gemm_noalloc's fixed scratch array (see there).
 *   The launch plan (kernel variant, tiles, splits, grids) depends on the
 *   shape, the bit width and the device's compute-unit count, and on the
 *   overrides of qmm_set_override, which the library reads from the
 *   environment once, when it is loaded; no call reads the environment.
 *   QMM_ERR_DEVICE is returned when the HIP runtime reports an error at
 *   launch time, or when no GPU is present.
 */
#ifndef QMM_H
#define QMM_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define QMM_ABI_VERSION 3

#if defined(__GNUC__) || defined(__clang__)
#define QMM_API __attribute__((visibility("default")))
#else
#define QMM_API
#endif

typedef enum qmm_status {
    QMM_OK = 0,
    QMM_ERR_INVALID_ARGUMENT = 1, /* shape, size or NULL pointer problem      */
    QMM_ERR_UNSUPPORTED = 2,      /* valid request the library does not cover */
    QMM_ERR_MISALIGNED = 3,       /* pointer alignment below the requirement  */
    QMM_ERR_DEVICE = 4            /* HIP runtime error at launch / no device  */
} qmm_status;

/* Decode GEMV (M = 1): y[n] = sum_k (s*q + m)[n][k] * x[k].
 * Pages: "BaseRT claims fastest Apple Silicon inference", section "What
 * BaseRT does differently" (dedicated GEMV kernels for decode where M = 1,
 * dequantization inline in the compute loop).
 *   w_packed  uint32 [n][k*bits/32]      scales, mins  fp16 [n][k/group_size]
 *   x         fp16   [k]                 y             fp32 [n] (written)     */
QMM_API qmm_status qmm_gemv(const void *w_packed, const void *scales, const void *mins,
                    const void *x, float *y, int64_t n, int64_t k,
                    int bits, int group_size, void *stream);

/* Decode GEMV with the residual add fused into its epilogue:
 *   y[n] = residual[n] + sum_k (s*q + m)[n][k] * x[k].
 * Pages: "BaseRT claims fastest Apple Silicon inference", section "What
 * BaseRT does differently" (fusion removes a launch and a global-memory round
 * trip per fusion; residual buffers are part of the decode loop's state).
 *   residual fp32 [n], 4-byte aligned, non-NULL; it may be y itself (y +=
 *   W x: each row's residual is read before that row is written).  Other
 *   arguments as qmm_gemv.                                                  */
QMM_API qmm_status qmm_gemv_residual(const void *w_packed, const void *scales,
                                     const void *mins, const void *x, const float *residual,
                                     float *y, int64_t n, int64_t k, int bits, int group_size,
                                     void *stream);

/* Fused gate/up projection of a feed-forward block (decode, M = 1):
 *   h[n] = silu(g[n]) * u[n],  g = Wg x,  u = Wu x,  silu(v) = v / (1 + e^-v).
 * Pages: "BaseRT claims fastest Apple Silicon inference", section "What
 * BaseRT does differently" (kernel fusion removes a launch and a global
 * memory round trip per fusion); "BaseRT: Best-in-Class LLM Inference on
 * Apple Silicon via Native Metal", section "Metodologia" (operator sequences
 * of feed-forward blocks fused into one kernel).
 * Both matrices are n x k in the same format (bits, group_size) with their
 * own scale and min arrays; g and u stay in registers, only h is written.
 *   x fp16 [k]      h fp32 [n] (written)
 * k must fit one pass of the decode kernel (k <= 8192 codes for 64-multiple
 * groups, 4096 for 32-code groups and for fp16 weights), else
 * QMM_ERR_UNSUPPORTED.                                                      */
QMM_API qmm_status qmm_gemv_swiglu(const void *gate_w, const void *gate_scales,
                                   const void *gate_mins, const void *up_w,
                                   const void *up_scales, const void *up_mins,
                                   const void *x, float *h, int64_t n, int64_t k,
                                   int bits, int group_size, void *stream);

/* Prefill GEMM (M >= 1): y[i][n] = sum_k (s*q + m)[n][k] * x[i][k].
 * Pages: "BaseRT claims fastest Apple Silicon inference", section "What
 * BaseRT does differently" (GEMM kernels for prefill where M > 1); "BaseRT:
 * Best-in-Class LLM Inference on Apple Silicon via Native Metal", section
 * "Metodologia" (tiled prefill GEMM on the GPU's matrix units).
 * The weights are dequantized to fp16 tiles and multiplied on fp16 matrix
 * cores with fp32 accumulation.  Small m is routed to the bandwidth-bound
 * multi-row GEMV kernel.
 *   x  fp16 [m][k]      y  fp32 [m][n] (written)
 *   workspace: optional device scratch (may be NULL / 0 bytes), 16-byte
 *   aligned.  When the shape leaves the GPU under-filled, up to
 *   qmm_gemm_workspace_bytes() of it is used to split the K loop; with less,
 *   the split shrinks to what fits (no split with none).  Its first 4096
 *   bytes hold per-tile arrival counters: the workspace must be all zero before
 *   its first use (allocate it zeroed once), and every call leaves those
 *   counters zero again, so one workspace serves any sequence of calls on
 *   one stream.  Calls that overlap (other streams) need their own
 *   workspace.  The rest of its contents on return are unspecified.
 *   Two-way splits are summed inside the GEMM kernel: each work-group
 *   writes its partial sums with stores that go through every cache to
 *   memory (the system-coherent cache policy of gfx950 buffer stores),
 *   waits until they are acknowledged, then bumps its tile's counter with a
 *   relaxed device-scope atomic add; the work-group that arrives last reads
 *   the partial sums with loads that bypass the caches, writes y and resets
 *   the counter.  Correctness rests on those cache-policy bits and the
 *   store acknowledgement, not on release/acquire fences (a device-scope
 *   fence would write back and invalidate a whole L2 per wave).  Larger
 *   splits are summed by a second kernel on the same stream.               */
QMM_API qmm_status qmm_gemm(const void *w_packed, const void *scales, const void *mins,
                    const void *x, float *y, int64_t m, int64_t n, int64_t k,
                    int bits, int group_size, void *workspace,
                    size_t workspace_bytes, void *stream);

/* Prefill GEMM with fp16 output: y[i][n] as qmm_gemm, rounded once from the
 * fp32 sums to fp16 (nearest even; beyond the fp16 range +-inf).  Halves the
 * output bytes for long prefills ("BaseRT: Best-in-Class LLM Inference on
 * Apple Silicon via Native Metal", section "Resultados": prefill measured at
 * 2048 tokens).  Every m runs on the matrix-core kernel; workspace as for
 * qmm_gemm (split partial sums stay fp32; qmm_gemm_workspace_bytes gives the
 * preferred size for m > 2, none is needed below that).
 *   y  fp16 [m][n] (written), 16-byte aligned.                             */
QMM_API qmm_status qmm_gemm_f16out(const void *w_packed, const void *scales,
                                   const void *mins, const void *x, void *y, int64_t m,
                                   int64_t n, int64_t k, int bits, int group_size,
                                   void *workspace, size_t workspace_bytes, void *stream);

/* Prefill GEMM that allocates nothing, for callers that cannot call
 * hipMalloc or take a workspace: code under HIP graph capture, tight
 * serving loops, harnesses that forbid allocation.
 * Same arguments and result as qmm_gemm without the workspace: it runs the
 * plan qmm_gemm takes with its preferred workspace (qmm_gemm_workspace_bytes),
 * so y is bit-identical to that call's.  The K-split partial sums and
 * arrival counters live in a static device array of
 * QMM_NOALLOC_SCRATCH_BYTES inside the library, one per GPU, held until the
 * process ends; a shape that would need more (qmm_gemm_workspace_bytes
 * above that) returns QMM_ERR_UNSUPPORTED and launches nothing.  Each call
 * resets the counters it uses with a small kernel before the GEMM (no
 * memset, no allocation).  Every call on one GPU shares that GPU's array:
 * calls that overlap on one GPU (other streams, other host threads) race
 * and give wrong results; calls ordered on one stream are safe.           */
#define QMM_NOALLOC_SCRATCH_BYTES (32u * 1024u * 1024u)

QMM_API qmm_status qmm_gemm_noalloc(const void *w_packed, const void *scales, const void *mins,
                                    const void *x, float *y, int64_t m, int64_t n, int64_t k,
                                    int bits, int group_size, void *stream);

/* Grouped prefill GEMM: up to 4 weight matrices that share the activations
 * x [m][k] (the q, k and v projections of a layer, or gate and up), one
 * launch: y_i[r][j] = sum_k (s*q + m)_i[j][k] * x[r][k] for every member i.
 * Pages: "BaseRT claims fastest Apple Silicon inference", section "What
 * BaseRT does differently" (operations other runtimes dispatch separately
 * run as one fused dispatch; GEMM kernels for prefill).
 *   members (host array of count, 1..4): each member's packed weights,
 *     scales and mins in the qmm_gemm layout with its own n (n == 0: the
 *     member is skipped), and its output y fp32 [m][n], 16-byte aligned.
 *   x fp16 [m][k], 16-byte aligned; bits and group_size shared.
 *   workspace: as qmm_gemm (zero before its first use, counters left zero);
 *     qmm_gemm_grouped_workspace_bytes gives the preferred size (it reads
 *     the members' n only; sized for the current device, or for 256
 *     compute units where no device can be queried).
 * The library chooses between one launch and one launch per member (as
 * qmm_gemm would, same stream, same workspace) from the shapes: one launch
 * where the members underfill the GPU on their own, or where their tiles
 * together fill it without a K split; separate launches where each
 * member's own tile grid fills it.  Either way each y_i is member i's
 * product to qmm_gemm's accuracy.  A grouped launch sums any K split
 * inside the kernel, as described for two-way splits under qmm_gemm.      */
typedef struct {
    const void *w_packed;
    const void *scales;
    const void *mins;
    float *y;
    int64_t n;
} qmm_gemm_member;

QMM_API qmm_status qmm_gemm_grouped(const qmm_gemm_member *members, int count, const void *x,
                                    int64_t m, int64_t k, int bits, int group_size,
                                    void *workspace, size_t workspace_bytes, void *stream);
QMM_API size_t qmm_gemm_grouped_workspace_bytes(const qmm_gemm_member *members, int count,
                                                int64_t m, int64_t k, int bits, int group_size);

/* Many independent decode GEMVs in one launch.
 * Pages: "BaseRT claims fastest Apple Silicon inference", section "What
 * BaseRT does differently" (operations other runtimes dispatch separately
 * are combined, saving launches); "BaseRT: Best-in-Class LLM Inference on
 * Apple Silicon via Native Metal", section "Metodologia" (low-overhead
 * dispatch without per-operation scheduling).
 * Every descriptor is one qmm_gemv (same bits and group_size for all; each
 * k at most 8192 codes for 64-multiple groups, 4096 otherwise and at 16
 * bits, else QMM_ERR_UNSUPPORTED; the whole batch below 2^31 row batches,
 * likewise).  Launch start-up reads a 256-entry index of the work list from
 * the kernel arguments, so finding a wave's first descriptor costs one
 * dependent load of the device copy whatever the count.  first_item is owned by
 * the library: qmm_gemv_batch_prepare fills it in a host array, the caller
 * copies the array to device memory (once; it can be reused for every
 * later call with the same shapes and pointers) and passes both copies to
 * qmm_gemv_batched, which checks the host copy and launches one kernel that
 * reads the device copy.  The two copies must hold the same bytes.  Outputs
 * of different descriptors must not overlap.                                */
typedef struct qmm_gemv_desc {
    const void *w_packed;   /* uint32 [n][k*bits/32]                          */
    const void *scales;     /* fp16 [n][k/group_size]                         */
    const void *mins;       /* fp16 [n][k/group_size]                         */
    const void *x;          /* fp16 [k]                                       */
    float *y;               /* fp32 [n] (written)                             */
    int64_t n, k;
    int64_t first_item;     /* library-owned, see qmm_gemv_batch_prepare      */
} qmm_gemv_desc;

QMM_API qmm_status qmm_gemv_batch_prepare(qmm_gemv_desc *descs /* host */, int64_t count,
                                          int bits, int group_size);
QMM_API qmm_status qmm_gemv_batched(const qmm_gemv_desc *descs_device,
                                    const qmm_gemv_desc *descs_host, int64_t count,
                                    int bits, int group_size, void *stream);

/* Bytes of workspace that let qmm_gemm use its preferred K split for this
 * shape on the current device (0 when it would not split; sized for 256
 * compute units where no device can be queried).  Host only.              */
QMM_API size_t qmm_gemm_workspace_bytes(int64_t m, int64_t n, int64_t k, int bits,
                                int group_size);

/* Mixture-of-experts projection over rows grouped by expert.
 * Pages: "BaseRT claims fastest Apple Silicon inference", section "Where the
 * wins land, and where they don't" (MoE decode and prefill; routing handled
 * without branching in the hot path); "BaseRT: Best-in-Class LLM Inference on
 * Apple Silicon via Native Metal", section "Resultados" (MoE prefill).
 *   w_packed  uint32 [n_experts][n][k*bits/32]  (experts stacked)
 *   scales, mins fp16 [n_experts][n][k/group_size]
 *   expert_offsets int32 [n_experts + 1] (device): rows of expert e are
 *     p in [expert_offsets[e], expert_offsets[e+1]); non-decreasing, from 0
 *     to p_rows.
 *   x fp16 [x_rows_count][k]; x_rows int32 [p_rows] (device) or NULL:
 *     row p of the product reads activation row x_rows[p] (row p if NULL).
 *   y fp32 [p_rows][n] (written): y[p][j] = sum_k w_e[j][k] * x[row(p)][k].
 * Rows whose activation index is outside [0, x_rows_count) are written as
 * NaN (nothing is read out of bounds); output rows that no expert range
 * covers are left untouched.  Offsets are clamped to [0, p_rows].  Routing
 * weights are not applied.                                                 */
QMM_API qmm_status qmm_moe_gemm(const void *w_packed, const void *scales, const void *mins,
                        const void *x, const int32_t *x_rows, int64_t x_rows_count,
                        const int32_t *expert_offsets, float *y, int64_t p_rows,
                        int64_t n_experts, int64_t n, int64_t k, int bits,
                        int group_size, void *stream);

/* Fused gate/up projection of the selected experts:
 *   h[p][j] = silu(g[p][j]) * u[p][j], g and u as qmm_moe_gemm over the
 *   gate stack and the up stack, silu(v) = v / (1 + e^-v).
 * Pages: as qmm_gemv_swiglu (fusion of feed-forward operator sequences) and
 * as qmm_moe_gemm (expert rows).  Both stacks [n_experts][n][...] in one
 * format; the remaining arguments and the NaN rule are those of
 * qmm_moe_gemm.  k must fit one pass (as qmm_gemv_swiglu), else
 * QMM_ERR_UNSUPPORTED.                                                      */
QMM_API qmm_status qmm_moe_swiglu(const void *gate_w, const void *gate_scales,
                                  const void *gate_mins, const void *up_w,
                                  const void *up_scales, const void *up_mins, const void *x,
                                  const int32_t *x_rows, int64_t x_rows_count,
                                  const int32_t *expert_offsets, float *h, int64_t p_rows,
                                  int64_t n_experts, int64_t n, int64_t k, int bits,
                                  int group_size, void *stream);

/* Expert projection with the routing-weighted combine fused into its store:
 *   y[pair_token[p]][j] += pair_weight[p] * sum_k w_e[j][k] * x[row(p)][k]
 * for every row p of expert e, so each token's row of y receives the
 * weighted sum of its selected experts' outputs (the MoE down projection and
 * combine in one launch; y may hold the residual stream beforehand).
 * Pages: as qmm_moe_gemm (expert rows) and as qmm_gemv_swiglu (fusion of
 * operator sequences saves a launch and a round trip through memory).
 *   pair_token int32 [p_rows], pair_weight fp32 [p_rows] (device, 4-byte
 *     aligned): token and routing weight of row p.
 *   y fp32 [n_tokens][n], 16-byte aligned, read and written (accumulated).
 * Other arguments as qmm_moe_gemm.  The adds into one element of y happen in
 * no fixed order (float atomics), so results may differ in the last bits
 * from run to run.  Rows with an activation index out of range add NaN to
 * their token's row; rows whose token is outside [0, n_tokens) add nothing.
 * n_tokens == 0 or p_rows == 0 is a no-op.                                  */
QMM_API qmm_status qmm_moe_combine(const void *w_packed, const void *scales, const void *mins,
                                   const void *x, const int32_t *x_rows, int64_t x_rows_count,
                                   const int32_t *expert_offsets, const int32_t *pair_token,
                                   const float *pair_weight, float *y, int64_t n_tokens,
                                   int64_t p_rows, int64_t n_experts, int64_t n, int64_t k,
                                   int bits, int group_size, void *stream);

/* ---- The attention half of a decoder layer -----------------------------
 * What stands between a layer's products: qmm_norm_residual turns one
 * product's fp32 (or fp16) output into the residual stream and the fp16 input
 * of the next, qmm_kv_append takes the q, k and v products to rotated queries
 * and a paged cache, qmm_attn_prompt and qmm_attn_cache give the input of the
 * output projection.  The rules at the top of this file hold (host checks,
 * no allocation, asynchronous on `stream`, errors); results repeat bit for
 * bit for the same arguments and plan.
 *
 * Norm, gate and residual around a block, per row r of n elements:
 *   u = y[r]                                     (y fp32, or fp16 with y_fp16)
 *   u = u * rsqrt(mean(u^2) + eps) * post_weight (post_weight not NULL)
 *   u = u * gate[r]                              (gate not NULL)
 *   h[r] = residual[r] + scale * u               (residual NULL: scale * u)
 *   x[r] = fp16(h[r] * rsqrt(mean(h[r]^2) + eps) * pre_weight)
 *   y  [rows] rows y_stride elements apart; NULL: h is residual, nothing is
 *      written to the argument h (it may be NULL), and residual is required.
 *   post_weight, pre_weight fp32 [n] or NULL (no norm on y; weight one on x).
 *   gate fp32, rows gate_stride elements apart; 0: one row for all.
 *   residual, h fp32 [rows][n]; h may be residual itself, or NULL (not kept).
 *   x fp16 [rows][n] or NULL (not wanted).  h or x has to be given.
 * Sums are fp32 in a fixed order.  n at most 32768, rows below 2^22, else
 * QMM_ERR_UNSUPPORTED.  Pointers aligned to their elements; 16-byte aligned
 * rows (n and strides multiples of 4) are faster.  x must not overlap an
 * input; neither must h, but for residual.                                 */
QMM_API qmm_status qmm_norm_residual(const void *y, int y_fp16, int64_t y_stride,
                                     const float *post_weight, const float *gate,
                                     int64_t gate_stride, float scale, const float *residual,
                                     float *h, const float *pre_weight, void *x, int64_t rows,
                                     int64_t n, float eps, void *stream);

/* A paged key/value cache (host struct of device pointers; the caller owns
 * the memory).  Page p, kv head j and place i hold one row of head_dim values:
 *   k, v          [pages][kv_heads][page_size] rows of head_dim codes, the
 *                 row bitstream of the weights (head_dim * bits / 32 words);
 *                 bits 16: fp16 values
 *   *_scales, *_mins  fp16 [pages][kv_heads][head_dim / group_size][page_size]:
 *                 the row's value d is scale * code + min of its group
 *                 d / group_size.  NULL at bits 16.
 * A slot is page * page_size + place.
 * bits 4, 8 or 16 (2, 3, 5, 6: QMM_ERR_UNSUPPORTED); head_dim 64 or 128 (other
 * positive: QMM_ERR_UNSUPPORTED); group_size a multiple of 32 that divides
 * head_dim (not looked at with 16 bits); page_size a power of two from 16 to
 * 65536 (other positive: QMM_ERR_UNSUPPORTED); kv_heads 1 to 4096.  Arrays
 * 16-byte aligned.  Any size: rows are addressed with 64-bit offsets.      */
typedef struct qmm_kv_cache {
    void *k, *k_scales, *k_mins;
    void *v, *v_scales, *v_mins;
    int64_t pages;
    int32_t kv_heads, head_dim, page_size, bits, group_size, reserved;
} qmm_kv_cache;

/* New tokens' q, k and v rows (fp32, or fp16 with in_fp16; token rows
 * *_stride elements apart, so one fused product serves as well as three):
 *   q, k: optional per-head norm, x * rsqrt(mean(x^2) + eps) * weight (q_norm,
 *     k_norm fp32 [head_dim] or NULL), then the rotation of the first rot_dim
 *     elements by position: with t = positions[token] * inv_freq[i], elements
 *     (a, b) = (x[i], x[i + rot_dim / 2]), or (x[2i], x[2i + 1]) if
 *     interleaved, become (a cos t - b sin t, b cos t + a sin t).  The angle
 *     (below 2^50) is formed and reduced in 64 bits.
 *   q_out fp16 [tokens][q_heads][head_dim]
 *   k, v: into slot slots[token] of the cache.  Per group: min fp16(lowest),
 *     scale fp16((highest - lowest) / (2^bits - 1)), code
 *     round((x - min) / scale) within 0 .. 2^bits - 1 (0 where the scale is 0 or
 *     not finite).
 *   k_out, v_out fp16 [tokens][kv_heads][head_dim] or NULL: what prompt
 *     attention reads; with out_cached the values that the cache stands for
 *     (fp16(scale * code + min)), else the rows before quantization.
 *   positions int32 [tokens], slots int64 [tokens] (device).  A slot outside
 *     [0, pages * page_size) (-1 for padding) is not stored.  slots NULL:
 *     nothing is stored and the cache's arrays are not looked at.  The slots of
 *     one call have to differ: one that is given twice holds a mixture of both.
 *   inv_freq fp32 [rot_dim / 2]; rot_dim 0 (no rotation, positions and
 *     inv_freq may be NULL) to head_dim, a multiple of 16.
 * q_heads 0 (q and q_out may be NULL) to 4096; rows 16-byte aligned (pointers
 * and strides); tokens below 2^24.  A group with a value that is not finite, or
 * whose lowest value is beyond fp16, or whose spread is (over 2^bits - 1),
 * gets a scale that is not finite and reads back as NaN.  Where the highest
 * value alone is beyond fp16 the group is held as it is: exact as a key, as a
 * value (and in k_out and v_out) infinite where it leaves fp16.              */
QMM_API qmm_status qmm_kv_append(const qmm_kv_cache *cache /* host */, const void *q,
                                 const void *k, const void *v, int in_fp16, int64_t q_stride,
                                 int64_t k_stride, int64_t v_stride, const float *q_norm,
                                 const float *k_norm, float eps, const float *inv_freq,
                                 int rot_dim, int interleaved, const int32_t *positions,
                                 const int64_t *slots, void *q_out, void *k_out, void *v_out,
                                 int out_cached, int64_t tokens, int q_heads, void *stream);

/* Attention of the newest q_len tokens of n_seqs sequences over the cache.
 *   q, out fp16 [n_seqs][q_len][q_heads][head_dim], 16-byte aligned; query
 *     head j reads kv head j / (q_heads / kv_heads).
 *   page_table int32 [n_seqs] rows of table_stride entries (device): cached
 *     row t of sequence i is place t % page_size of page
 *     page_table[i][t / page_size].  Entries behind a sequence's last page are
 *     not read.  An entry outside [0, pages) makes the sequence's rows NaN.
 *   kv_lens int32 [n_seqs] (device): cached rows of a sequence, the q_len new
 *     ones included; values outside [0, max_kv_len] are clamped.
 *   Token i of q_len sees rows t < kv_len - q_len + 1 + i; one that sees no
 *     row gets zeros.  Rows behind kv_len may hold anything.  A value of v,
 *     fp16(scale * code + min), that is not finite, and a score that is NaN or
 *     +inf, reaches the tokens that see it and no others; a score of -inf
 *     leaves its row out.
 *   max_kv_len (host): at most table_stride * page_size and below 2^30.
 *   scale multiplies the scores (before the softmax); its magnitude is at most
 *     2^64, else QMM_ERR_UNSUPPORTED.
 *   workspace: device scratch, 16-byte aligned, for partial sums.  Its first
 *     QMM_ATTN_COUNTER_BYTES bytes hold arrival counters: they must be zero
 *     before its first use (allocate it zeroed once), and every call leaves
 *     them zero again, so one workspace serves any sequence of calls on one
 *     stream, whatever their shapes.  With less than
 *     qmm_attn_cache_workspace_bytes() long sequences are split less, with
 *     none not at all.  Calls that overlap need a workspace each.
 * q_len 1 to 256.  Roundings to fp16: the output's; over codes that of the
 * values of v, over fp16 rows that of the probabilities.  Sums are fp32.     */
#define QMM_ATTN_COUNTER_BYTES (64u * 1024u)

QMM_API qmm_status qmm_attn_cache(const qmm_kv_cache *cache /* host */, const void *q,
                                  const int32_t *page_table, int64_t table_stride,
                                  const int32_t *kv_lens, int64_t max_kv_len, void *out,
                                  int64_t n_seqs, int q_len, int q_heads, float scale,
                                  void *workspace, size_t workspace_bytes, void *stream);
QMM_API size_t qmm_attn_cache_workspace_bytes(const qmm_kv_cache *cache /* host */,
                                              int64_t n_seqs, int q_len, int q_heads,
                                              int64_t max_kv_len);

/* Causal attention over whole prompts packed behind each other.
 *   q, out fp16 [tokens] rows of [q_heads][head_dim], k, v fp16 [tokens] rows of
 *     [kv_heads][head_dim]; rows *_stride elements apart, 16-byte aligned
 *     (pointers and strides).  out must not overlap an input.
 *   seq_offsets int32 [n_seqs + 1] (device), non-decreasing: sequence i is
 *     rows seq_offsets[i] .. seq_offsets[i + 1] - 1, and row r of it sees rows
 *     seq_offsets[i] .. r.  Rows that no sequence covers are left as they were.
 *     Whatever the offsets hold, nothing outside the given rows is touched.
 *   A value of v that is not finite, and a score that is NaN or +inf, reaches
 *     the rows that see it and no others; a score of -inf leaves its key out.
 * head_dim 64 or 128; q_heads a multiple of kv_heads; k and v strides below
 * 2^23, scale's magnitude at most 2^64 (else QMM_ERR_UNSUPPORTED).  Probabilities are
 * rounded to fp16 for the second product; sums are fp32.                    */
QMM_API qmm_status qmm_attn_prompt(const void *q, const void *k, const void *v,
                                   const int32_t *seq_offsets, void *out, int64_t tokens,
                                   int64_t n_seqs, int q_heads, int kv_heads, int head_dim,
                                   int64_t q_stride, int64_t k_stride, int64_t v_stride,
                                   int64_t out_stride, float scale, void *stream);

/* ---- A mixture of experts' feed-forward block ---------------------------
 * What stands around the experts' products: qmm_moe_route turns the router's
 * scores into experts, weights and the rows grouped by expert that
 * qmm_moe_gemm, qmm_moe_swiglu and the 8-bit products below take (its
 * pair_token is their x_rows), and qmm_moe_gather adds the experts' rows up by
 * token.  The rules at the top of this file hold; results repeat bit for bit.
 *
 * Routing, per token of n_experts scores l (fp32, or fp16 with logits_fp16; rows
 * logits_stride elements apart):
 *   s = softmax(l), or sigmoid(l) if `sigmoid`;  c = s + bias (bias fp32
 *     [n_experts], or NULL: c = s)
 *   n_groups > 1: expert e is of group e / (n_experts / n_groups); a group's
 *     score is the sum of its group_best (1 or 2) highest c, and only experts of
 *     the top_groups groups of highest score can be chosen
 *   the top_k experts of highest c, in falling order of c
 *   w = s[chosen], divided by their sum if `renormalize`, times scale
 * Of equals the lower group and the lower expert come first.  Without a bias
 * the c are in the order of the logits, exactly; sums of them, and c with a
 * bias, are formed in 64 bits.
 *   A logit of -inf scores 0 (it is chosen only where nothing else is left); a
 *     token of nothing else gets weights of 0.  A NaN logit is placed as -inf and
 *     makes the token's weights NaN, and so does +inf under softmax (where the
 *     others' scores are then 0).  A c that is NaN is placed as -inf.
 *   keep uint8 [tokens] or NULL: a token of 0 (padding) gets experts -1, weights 0
 *     and no row.
 *   expert_ids int32, weights fp32 [tokens][top_k]
 *   expert_offsets int32 [n_experts + 1], or NULL: nothing is grouped, and what
 *     follows is not looked at.  The pairs (token, choice) are sorted by expert,
 *     within an expert by token; expert e's rows are expert_offsets[e] ..
 *     expert_offsets[e + 1] - 1.
 *   pair_row int32 [tokens][top_k] or NULL: row of each pair (-1: none)
 *   pair_token int32, pair_weight fp32 [tokens * top_k], or NULL: token and
 *     weight of each row; behind the last row they are left as they were.
 *   workspace: device scratch of qmm_moe_route_workspace_bytes(), 16-byte aligned,
 *     needed only to group (else QMM_ERR_INVALID_ARGUMENT); it may hold anything,
 *     and one for some tokens serves fewer.  Calls that overlap need a workspace each.
 * n_experts at most 1024, n_groups and top_k at most 64, tokens below 2^24, else
 * QMM_ERR_UNSUPPORTED.  tokens 0: the offsets are set to 0.  No output may
 * overlap an input or another output.                                       */
QMM_API qmm_status qmm_moe_route(const void *logits, int logits_fp16, int64_t logits_stride,
                                 const float *bias, int sigmoid, int n_groups, int top_groups,
                                 int group_best, int top_k, int renormalize, float scale,
                                 const uint8_t *keep, int32_t *expert_ids, float *weights,
                                 int32_t *pair_row, int32_t *expert_offsets, int32_t *pair_token,
                                 float *pair_weight, void *workspace, size_t workspace_bytes,
                                 int64_t tokens, int n_experts, void *stream);
QMM_API size_t qmm_moe_route_workspace_bytes(int64_t tokens, int n_experts, int top_k);

/* The experts' rows back to their tokens, in a fixed order (qmm_moe_combine adds
 * in no fixed order, inside the last product):
 *   y[t] = residual[t] + sum_j weights[t][j] * rows[pair_row[t][j]]
 *   rows fp32 (fp16 with rows_fp16) [p_rows][n]; pair_row int32, weights fp32
 *   [tokens][top_k], as qmm_moe_route gives them; a row outside [0, p_rows) adds
 *   nothing.  residual fp32 [tokens][n] or NULL (zero); it may be y.
 *   y fp32 [tokens][n] (written).
 * Sums are fp32, in the order of j, the residual last.  top_k at most 64, tokens below 2^24,
 * n below 2^22, else QMM_ERR_UNSUPPORTED.  Pointers aligned to their elements;
 * n a multiple of 8 (of 4 for fp32 rows) and 16-byte aligned pointers are faster. */
QMM_API qmm_status qmm_moe_gather(const void *rows, int rows_fp16, const int32_t *pair_row,
                                  const float *weights, const float *residual, float *y,
                                  int64_t tokens, int top_k, int64_t p_rows, int64_t n,
                                  void *stream);

/* Products in 8-bit integers, with a scale for each row of either side
 * (prefill at twice the matrix cores' rate for fp16, and half of its bytes).
 *
 * Activations to codes, per row of k values: scale = max |x| / 127 (fp32), code
 * = round(x / scale), ties to even, within -127 .. 127 (0 where the scale is 0);
 * the row's values are scale * code.
 *   x fp32, or fp16 with x_fp16; rows x_stride elements apart
 *   codes int8 [rows][k], 16-byte aligned; scales fp32 [rows]
 * A row with a value that is not finite gets the scale NaN and codes 0, so
 * whatever it is multiplied with is NaN.  k a multiple of 32, at most 32768,
 * rows below 2^22 (else QMM_ERR_UNSUPPORTED).                               */
QMM_API qmm_status qmm_quantize_rows(const void *x, int x_fp16, int64_t x_stride, int8_t *codes,
                                     float *scales, int64_t rows, int64_t k, void *stream);

/* y[i][j] = x_scales[i] * w_scales[j] * sum_k x[i][k] * w[j][k]
 *   w int8 [n][k] with w_scales fp32 [n]; x int8 [m][k] with x_scales fp32 [m];
 *   any codes from -128 to 127.  y fp32 [m][n], or fp16 with y_fp16.
 * The sums are exact; scaling is fp32, by x_scales first, and fp16 outputs are
 * rounded once more.
 * w, x and y 16-byte aligned, scales 4-byte; k a multiple of 32, at most 32768;
 * one matrix and the activation block each below 4 GiB (else
 * QMM_ERR_UNSUPPORTED).  Any m and n; y must not overlap an input.          */
QMM_API qmm_status qmm_gemm_i8(const int8_t *w, const float *w_scales, const int8_t *x,
                               const float *x_scales, void *y, int y_fp16, int64_t m, int64_t n,
                               int64_t k, void *stream);

/* The same over rows grouped by expert, with stacks w int8 [n_experts][n][k] and
 * w_scales fp32 [n_experts][n]: row p of expert e's range reads activation row
 * x_rows[p] (int32 [p_rows]; p if NULL) of x_rows_count.  expert_offsets, rows
 * with an activation index out of range (NaN) and rows that no expert covers
 * (left as they were) are as for qmm_moe_gemm; expert_offsets NULL with one
 * expert: all rows are its.  n_experts at most 1024, p_rows below 2^31 (else
 * QMM_ERR_UNSUPPORTED).                                                     */
QMM_API qmm_status qmm_moe_gemm_i8(const int8_t *w, const float *w_scales, const int8_t *x,
                                   const float *x_scales, const int32_t *x_rows,
                                   int64_t x_rows_count, const int32_t *expert_offsets, void *y,
                                   int y_fp16, int64_t p_rows, int64_t n_experts, int64_t n,
                                   int64_t k, void *stream);

/* Gate and up products of the selected experts in one launch:
 *   h[p][j] = silu(g[p][j]) * u[p][j], g and u as qmm_moe_gemm_i8 over the two
 *   stacks, silu(v) = v / (1 + e^-v).  h fp32, or fp16 with h_fp16.          */
QMM_API qmm_status qmm_moe_swiglu_i8(const int8_t *gate_w, const float *gate_scales,
                                     const int8_t *up_w, const float *up_scales, const int8_t *x,
                                     const float *x_scales, const int32_t *x_rows,
                                     int64_t x_rows_count, const int32_t *expert_offsets, void *h,
                                     int h_fp16, int64_t p_rows, int64_t n_experts, int64_t n,
                                     int64_t k, void *stream);

/* One of the calls above, from qmm_norm_residual on, with its arguments as 64-bit
 * words in their order (pointers and whole numbers as int64, float as double):
 * for bindings in which every argument of a foreign call costs time.  Same
 * checks, same errors.  Words per call: 15, 23, 14, 16, 23, 8, 10, 14, 16 and 11. */
enum {
    QMM_CALL_NORM_RESIDUAL = 0, QMM_CALL_KV_APPEND = 1, QMM_CALL_ATTN_CACHE = 2, QMM_CALL_ATTN_PROMPT = 3,
    QMM_CALL_MOE_ROUTE = 4, QMM_CALL_QUANTIZE_ROWS = 5, QMM_CALL_GEMM_I8 = 6, QMM_CALL_MOE_GEMM_I8 = 7,
    QMM_CALL_MOE_SWIGLU_I8 = 8, QMM_CALL_MOE_GATHER = 9
};

QMM_API qmm_status qmm_call_words(int call, const void *words);

/* Codes as bytes: codes[n][k] = q[n][k] (uint8).  Bit-exact view of the
 * packed format, used to check the GPU's bit extraction.                   */
QMM_API qmm_status qmm_unpack(const void *w_packed, uint8_t *codes, int64_t n, int64_t k,
                      int bits, void *stream);

/* Launch plan the library would use (host only, no device call): which
 * kernel variant, grid and block.  `op` is 0 for qmm_gemv, 1 for qmm_gemm,
 * 2 for qmm_moe_gemm (m = rows per expert bound), 3 for qmm_gemv_batched
 * (n = total rows of the batch, k = its largest k).  cu_count <= 0 means
 * "query the current device" (then this does call the runtime).            */
typedef struct qmm_plan {
    int32_t variant;       /* library-internal variant id                   */
    int32_t lanes_per_row; /* GEMV: lanes cooperating on one output row     */
    int32_t units_per_lane;/* GEMV: 64- or 32-code units per lane per pass  */
    int32_t rows_per_iter; /* GEMV: rows per lane slot per loop iteration   */
    int32_t unit_codes;    /* GEMV: codes per unit (64 or 32)               */
    int32_t split_k;       /* GEMM: K split (1 = none)                      */
    int32_t tile_m, tile_n;/* GEMM: block tile                              */
    int64_t grid;          /* work-groups launched                          */
    int32_t block;         /* threads per work-group                        */
    int32_t reserved[5];   /* GEMV: [0] multi-pass rows, [1] row sums staged
                              in LDS, [2] activation units built after the
                              first weight loads; the rest zero              */
} qmm_plan;

QMM_API qmm_status qmm_get_plan(int op, int64_t m, int64_t n, int64_t k, int bits,
                        int group_size, int cu_count, size_t workspace_bytes,
                        qmm_plan *plan /* host */);

/* Launch-plan override for measurement sweeps and for tests that force a
 * kernel variant (host only, process-wide, not meant for production: a
 * forced variant may be slower, and a value the chosen kernel cannot take
 * is ignored).  name is one of QMM_UNIT, QMM_GEMV_LPR, QMM_GEMV_XC,
 * QMM_GEMV_U, QMM_GEMV_WAVES_PER_CU, QMM_BATCH_U, QMM_ROWS_MR,
 * QMM_ROWS_WAVES_PER_CU, QMM_GEMM_TILE_M, QMM_GEMM_TILE_N, QMM_GEMM_SPLIT,
 * QMM_GEMM_WIDE_SCALES, QMM_GEMM_ORDER, QMM_GEMM_GROUPED, QMM_GEMM_KERNEL
 * (1: the prefill GEMM that dequantizes into LDS, 2: the one that
 * dequantizes into registers), QMM_GEMV_STAGED (1/0: single GEMVs with
 * 64-lane rows do / do not stage their row sums in LDS), QMM_GEMV_LATE
 * (1/0: single Q4 GEMVs of one unit per lane on at most 32 lanes do / do
 * not build their activation units after the first weight loads); value < 0 removes
 * the override.  The same names are read from the environment once, when
 * the library is loaded.  Unknown name: QMM_ERR_INVALID_ARGUMENT.          */
QMM_API qmm_status qmm_set_override(const char *name, int value);

QMM_API const char *qmm_status_string(qmm_status s);
QMM_API const char *qmm_last_error(void);   /* thread-local; "" when none */
QMM_API int qmm_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* QMM_H */
