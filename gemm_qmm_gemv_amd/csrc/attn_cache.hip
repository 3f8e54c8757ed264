// attn_cache.hip -- attention of the newest tokens of many sequences over a
// paged cache held in 4- or 8-bit affine groups or in fp16.
//
//   k = s q + m, v = s q + m (per cached row and group),
//   S[r][t] = scale * sum_d Q[r][d] k[t][d],   t below the row's limit,
//   O[r] = sum_t exp(S[r][t] - max_t S) v[t] / sum_t exp(S[r][t] - max_t S).
//
// Bound by reading the cache, once.  The query heads that share a key head
// and the new tokens of a sequence are the rows of one 16-row matrix tile, so
// a cached row is read and unpacked once for all of them.  A wave owns tiles
// of 32 cached rows and keeps its own running maximum and sum, so waves meet
// only at the end; runs of `chunk` cached rows go to different work-groups
// and a second kernel joins their sums.
//
// Matrix products (v_mfma 16x16x32 fp16, fp32 sums), transposed so that no
// value changes lanes between the two:
//   S^T = K Q^T: rows = cached rows.  Lane (c, g) = (lane % 16, lane / 16)
//     gets S of query row c at cached rows 4g..4g+3 of each 16.
//   O^T = V^T P^T: its right operand wants, in lane (c, g), eight cached rows
//     of query row c; which eight is free as long as V^T uses the same, so
//     they are the ones the lane already holds.
// Keys stay exact: a code is a whole number in fp16, sums of Q times codes
// are kept per group and s and m are applied to the sums in fp32,
//   sum_d Q k = sum_group (s sum Q q + m sum Q).
// Values are rounded once to fp16 (the value the cache stands for).  The
// probabilities of quantized caches go in as fp16 high and low parts: the
// matrix cores idle most of the time, and with V's rounding in the result a
// second one of the same size would show.
#include "layer_kernels.h"
#include "qmm_device.h"

namespace qmm {
namespace {

typedef f16 f16x4v __attribute__((ext_vector_type(4)));

constexpr int WAVES = 4;
constexpr int TILE = 32;  // cached rows per wave step
constexpr float NEG_INF = -__builtin_huge_valf();

__device__ __forceinline__ f32x4 mfma16(f16x8 a, f16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f16x8 frag(u32 a, u32 b, u32 c, u32 d) {
    return __builtin_bit_cast(f16x8, u32x4{a, b, c, d});
}
// Max / sum over the four lane groups that share a query row.
__device__ __forceinline__ float groups_max(float v) {
    v = fmaxf(v, __shfl_xor(v, 16, 64));
    return fmaxf(v, __shfl_xor(v, 32, 64));
}
__device__ __forceinline__ float groups_sum(float v) {
    v += __shfl_xor(v, 16, 64);
    return v + __shfl_xor(v, 32, 64);
}

// N words from an address aligned to 4 N bytes (N = 1, 2 or 4 per access).
template <int N>
__device__ __forceinline__ void load_words(const char* p, u32 (&w)[N]) {
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const u32x4 v = reinterpret_cast<const u32x4*>(p)[i];
#pragma unroll
            for (int j = 0; j < 4; ++j) w[4 * i + j] = v[j];
        }
    } else if constexpr (N == 2) {
        const u32x2 v = *reinterpret_cast<const u32x2*>(p);
        w[0] = v[0];
        w[1] = v[1];
    } else {
        static_assert(N == 1, "words per access");
        w[0] = *reinterpret_cast<const u32*>(p);
    }
}

template <int BITS, int D, int GROUP>
struct Cfg {
    static constexpr bool Q = BITS != 16;               // quantized
    static constexpr int NG = Q ? D / GROUP : 1;        // groups per row
    static constexpr int GD = Q ? GROUP : D;            // elements per group
    static constexpr int ROW = D * BITS / 8;            // bytes per row
    static constexpr int KSTEPS = GD / 32;              // matrix steps per group
    static constexpr int KW = GD / 4 * BITS / 32;       // words per lane, group and cached row of K
    static constexpr int VC = D / 16;                   // values per lane and cached row of V
    static constexpr int VB = VC * BITS / 8;            // their bytes: 2, 4, 8 or 16
    static constexpr int VW = VB < 4 ? 1 : VB / 4;      // words holding them
};

// Everything one 32-row step reads, in registers.
template <class C>
struct Raw {
    u32 k[2][C::NG][C::KW];
    u32 v[8][C::VW];
    u32x2 ks[2][C::NG], km[2][C::NG];  // four fp16 each: cached rows 4g..4g+3
    u32x2 vs[2], vm[2];
};

template <int BITS, int D, int GROUP>
__device__ __forceinline__ void load_step(Raw<Cfg<BITS, D, GROUP>>& r, const CacheView& cv, const int (&page)[2],
                                          int first, int kvh, int c, int g) {
    using C = Cfg<BITS, D, GROUP>;
    const int mask = (1 << cv.page_shift) - 1;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        const int64_t unit = (int64_t)page[b] * cv.kv_heads + kvh;
        const int row0 = (first + 16 * b) & mask;
        const char* kp = static_cast<const char*>(cv.k) + ((unit << cv.page_shift) + row0) * C::ROW;
        const char* vp = static_cast<const char*>(cv.v) + ((unit << cv.page_shift) + row0) * C::ROW;
        if constexpr (C::Q) {
#pragma unroll
            for (int h = 0; h < C::NG; ++h)
                load_words<C::KW>(kp + c * C::ROW + (h * GROUP + g * (GROUP / 4)) * BITS / 8, r.k[b][h]);
        } else {
            // fp16 rows: step j takes elements 32 j + 8 g .. + 7.
#pragma unroll
            for (int j = 0; j < D / 32; ++j) {
                const u32x4 v = *reinterpret_cast<const u32x4*>(kp + c * C::ROW + (32 * j + 8 * g) * 2);
#pragma unroll
                for (int i = 0; i < 4; ++i) r.k[b][0][4 * j + i] = v[i];
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const char* p = vp + (4 * g + j) * C::ROW + c * C::VB;
            if constexpr (C::VB == 2)
                r.v[4 * b + j][0] = *reinterpret_cast<const uint16_t*>(p);
            else
                load_words<C::VW>(p, r.v[4 * b + j]);
        }
        if constexpr (C::Q) {
#pragma unroll
            for (int h = 0; h < C::NG; ++h) {
                const int64_t at = (((unit * C::NG + h) << cv.page_shift) + row0 + 4 * g) * 2;
                r.ks[b][h] = *reinterpret_cast<const u32x2*>(static_cast<const char*>(cv.ks) + at);
                r.km[b][h] = *reinterpret_cast<const u32x2*>(static_cast<const char*>(cv.km) + at);
            }
            const int64_t at = (((unit * C::NG + c * C::VC / GROUP) << cv.page_shift) + row0 + 4 * g) * 2;
            r.vs[b] = *reinterpret_cast<const u32x2*>(static_cast<const char*>(cv.vs) + at);
            r.vm[b] = *reinterpret_cast<const u32x2*>(static_cast<const char*>(cv.vm) + at);
        }
    }
}

// Codes of matrix step j of a lane's K words, as fp16 whole numbers in the
// order that q_order() gives Q: 4 bits, pairs (0,4) (1,5) (2,6) (3,7) of a
// word; 8 bits, pairs (0,2) (1,3) of each of two words.  1024 + code is exact
// in fp16 and so is the difference.
template <int BITS, int KW>
__device__ __forceinline__ f16x8 k_frag(const u32 (&w)[KW], int j) {
    const f16x2 m = as_h2(MAGIC2);
    if constexpr (BITS == 4) {
        const u32 v = w[j];
        return frag(as_u32(as_h2(mask_or_magic(v, 0x000F000Fu)) - m), as_u32(as_h2(mask_or_magic(v >> 4, 0x000F000Fu)) - m),
                    as_u32(as_h2(mask_or_magic(v >> 8, 0x000F000Fu)) - m), as_u32(as_h2(mask_or_magic(v >> 12, 0x000F000Fu)) - m));
    } else if constexpr (BITS == 8) {
        const u32 v0 = w[2 * j], v1 = w[2 * j + 1];
        return frag(as_u32(as_h2(mask_or_magic(v0, 0x00FF00FFu)) - m), as_u32(as_h2(mask_or_magic(v0 >> 8, 0x00FF00FFu)) - m),
                    as_u32(as_h2(mask_or_magic(v1, 0x00FF00FFu)) - m), as_u32(as_h2(mask_or_magic(v1 >> 8, 0x00FF00FFu)) - m));
    } else {
        return frag(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
    }
}
// Position, among the eight elements of a lane's matrix step, of operand element i.
template <int BITS>
__device__ constexpr int q_order(int i) {
    if (BITS == 4) return i / 2 + 4 * (i % 2);
    if (BITS == 8) return (i / 4) * 4 + (i % 4) / 2 + 2 * (i % 2);
    return i;
}

// V^T operand of value i (of the lane's VC) at the eight cached rows.
template <int BITS, int VW>
__device__ __forceinline__ f16x8 v_frag(const u32 (&w)[8][VW], int i, const u32x2 (&s)[2], const u32x2 (&m)[2]) {
    u32 out[4];
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        const int word = i * BITS / 32, bit = i * BITS % 32;
        const u32 a = w[2 * p][word], b = w[2 * p + 1][word];
        // Halves of both rows side by side, then the code at the same place of each.
        const u32 x = bit < 16 ? __builtin_amdgcn_perm(b, a, 0x05040100u) : __builtin_amdgcn_perm(b, a, 0x07060302u);
        if constexpr (BITS == 16) {
            out[p] = x;
        } else {
            const u32 mask = BITS == 4 ? 0x000F000Fu : 0x00FF00FFu;
            const f16x2 code = as_h2(mask_or_magic(x >> (bit % 16), mask)) - as_h2(MAGIC2);
            const f16x2 sc = as_h2(s[p / 2][p % 2]), mn = as_h2(m[p / 2][p % 2]);
            out[p] = as_u32(__builtin_elementwise_fma(code, sc, mn));
        }
    }
    return frag(out[0], out[1], out[2], out[3]);
}

__device__ __forceinline__ bool not_finite(u32 pair, int half) {
    return ((pair >> (16 * half)) & 0x7C00u) == 0x7C00u;
}

template <int BITS, int D, int GROUP>
__global__ void __launch_bounds__(64 * WAVES) attn_cache_kernel(CacheAttnArgs a) {
    using C = Cfg<BITS, D, GROUP>;
    constexpr int VC = C::VC;
    constexpr int OPAD = D + 4;  // floats per row of O in LDS: rows start on different banks
    __shared__ float lds_o[WAVES][16][OPAD];
    __shared__ float lds_m[WAVES][16], lds_l[WAVES][16];

    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int c = lane & 15, g = lane >> 4;
    // Row tiles of one (sequence, kv head) read the same cached rows: they
    // run eight work-groups apart, which the dispatcher's round robin over
    // the eight dies puts on one die and its L2.
    const int64_t per = 8LL * a.sh.row_tiles;
    const int64_t bx = blockIdx.x;
    const int rt = (int)(bx % per / 8);
    const int64_t pair = bx / per * 8 + bx % 8;
    if (pair >= a.n_seqs * a.c.kv_heads) return;
    const int kvh = (int)(pair % a.c.kv_heads);
    const int64_t seq = pair / a.c.kv_heads;
    const int split = blockIdx.y;

    int len = a.lens[seq];
    len = len < 0 ? 0 : len > a.max_len ? a.max_len : len;
    const int t0 = split * a.sh.chunk;
    if (split > 0 && t0 >= len) return;
    const int t1 = len - t0 < a.sh.chunk ? len : t0 + a.sh.chunk;
    const bool whole = len <= a.sh.chunk;  // one run: its sums are the result

    const int gq = a.q_heads / a.c.kv_heads;
    const int rows = a.q_len * gq;
    const int row = rt * 16 + c;
    const bool live = row < rows;
    const int step_i = live ? row / gq : 0;
    const int64_t q_row = (seq * a.q_len + step_i) * a.q_heads + kvh * gq + (live ? row % gq : 0);
    const int limit = live ? len - a.q_len + 1 + step_i : 0;  // cached rows this query row sees
    const int first_limit = len - a.q_len + 1;                // the fewest any row sees

    // Q operand and its sums per group.
    f16x8 qf[C::NG][C::KSTEPS];
    float qsum[C::NG];
    const float sc = a.scale * 1.44269504088896341f;  // scores in base 2
#pragma unroll
    for (int h = 0; h < C::NG; ++h) {
        qsum[h] = 0.f;
#pragma unroll
        for (int j = 0; j < C::KSTEPS; ++j) {
            const int d = C::Q ? h * GROUP + g * (GROUP / 4) + 8 * j : 32 * j + 8 * g;
            f16x8 v = {};
            if (live) v = *reinterpret_cast<const f16x8*>(static_cast<const f16*>(a.q) + q_row * D + d);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                qf[h][j][i] = v[q_order<BITS>(i)];
                qsum[h] += (float)v[i];
            }
        }
        qsum[h] = groups_sum(qsum[h]) * sc;
    }

    f32x4 o[VC];
#pragma unroll
    for (int i = 0; i < VC; ++i) o[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    float mx = NEG_INF, sum = 0.f;

    const int32_t* table = a.table + seq * a.table_stride;
    Raw<C> raw[2];
    int page[2];
    bool bad = false;
    auto pages_of = [&](int first) {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            // Past the last row there is no table entry to read; the entry
            // of the tile's first row stands in and its rows are masked.
            const int t = first + 16 * b < len ? first + 16 * b : first;
            const int p = uniform(table[t >> a.c.page_shift]);
            const bool in = p >= 0 && p < a.c.pages;
            page[b] = in ? p : 0;
            bad = bad || !in;
        }
    };

    auto compute = [&](Raw<C>& r, int first) {
        // Scores.
        float s[8];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            f32x4 acc[C::NG];
#pragma unroll
            for (int h = 0; h < C::NG; ++h) {
                acc[h] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int j = 0; j < C::KSTEPS; ++j) acc[h] = mfma16(k_frag<BITS>(r.k[b][h], j), qf[h][j], acc[h]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (C::Q) {
                    float dot = 0.f, low = 0.f;
#pragma unroll
                    for (int h = 0; h < C::NG; ++h) {
                        dot += (float)as_h2(r.ks[b][h][i / 2])[i % 2] * acc[h][i];
                        low += (float)as_h2(r.km[b][h][i / 2])[i % 2] * qsum[h];
                    }
                    s[4 * b + i] = dot * sc + low;
                } else {
                    s[4 * b + i] = acc[0][i] * sc;
                }
            }
        }
        if (first + TILE > first_limit) {
            // The end of a sequence: rows of pages behind it may hold
            // anything (a NaN times a probability of zero is NaN), so their
            // values are cleared and their scores dropped.  A drafted
            // token's row is seen by some rows only: if its values are not
            // finite they are cleared as well and the rows that see it get
            // a NaN score instead.
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int t = first + 16 * (j / 4) + 4 * g + j % 4;
                bool odd = false;
                if constexpr (C::Q) {
                    odd = not_finite(r.vs[j / 4][j % 4 / 2], j % 2) || not_finite(r.vm[j / 4][j % 4 / 2], j % 2);
                } else {
#pragma unroll
                    for (int w = 0; w < C::VW; ++w) odd = odd || not_finite(r.v[j][w], 0) || not_finite(r.v[j][w], 1);
                }
                const bool off = t >= len || (odd && t >= first_limit);
                if (off) {
                    if constexpr (C::Q) {
                        const u32 keep = j % 2 ? 0x0000FFFFu : 0xFFFF0000u;
                        r.vs[j / 4][j % 4 / 2] &= keep;
                        r.vm[j / 4][j % 4 / 2] &= keep;
                    } else {
#pragma unroll
                        for (int w = 0; w < C::VW; ++w) r.v[j][w] = 0;
                    }
                }
                // Any of the 16 lanes that hold this cached row.
                const uint64_t any = __ballot(odd && off);
                if ((any >> (16 * g)) & 0xFFFFu) s[j] = __builtin_nanf("");
                if (t >= limit) s[j] = NEG_INF;
            }
        }
        // Running maximum and sum.  A row that sees nothing yet keeps a
        // maximum of -inf; 0 stands in for it so that no inf - inf is formed.
        float top = fmaxf(fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3])), fmaxf(fmaxf(s[4], s[5]), fmaxf(s[6], s[7])));
        top = groups_max(top);
        const float m2 = fmaxf(mx, top);
        if (__any(m2 > mx)) {
            const float f = mx == NEG_INF ? 0.f : __builtin_amdgcn_exp2f(mx - m2);
            sum *= f;
#pragma unroll
            for (int i = 0; i < VC; ++i) o[i] = o[i] * f;
            mx = m2;
        }
        const float base = mx == NEG_INF ? 0.f : mx;
        float p[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            p[j] = __builtin_amdgcn_exp2f(s[j] - base);
            sum += p[j];
        }
        u32 hi[4], lo[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const f16x2 h2 = f16x2{(f16)p[2 * j], (f16)p[2 * j + 1]};
            hi[j] = as_u32(h2);
            lo[j] = as_u32(f16x2{(f16)(p[2 * j] - (float)h2[0]), (f16)(p[2 * j + 1] - (float)h2[1])});
        }
        const f16x8 pf = frag(hi[0], hi[1], hi[2], hi[3]), pl = frag(lo[0], lo[1], lo[2], lo[3]);
#pragma unroll
        for (int i = 0; i < VC; ++i) {
            const f16x8 vf = v_frag<BITS>(r.v, i, r.vs, r.vm);
            o[i] = mfma16(vf, pf, o[i]);
            if constexpr (C::Q) o[i] = mfma16(vf, pl, o[i]);
        }
    };

    const int stride = TILE * WAVES;
    int first = t0 + wave * TILE;
    if (first < t1) {
        pages_of(first);
        load_step<BITS, D, GROUP>(raw[0], a.c, page, first, kvh, c, g);
        while (true) {
            const int next = first + stride;
            const bool more = next < t1;
            if (more) {
                pages_of(next);
                load_step<BITS, D, GROUP>(raw[1], a.c, page, next, kvh, c, g);
            }
            compute(raw[0], first);
            if (!more) break;
            raw[0] = raw[1];
            first = next;
        }
    }
    // A page index outside the cache: nothing was read there, and every row
    // of this sequence and head becomes NaN.
    if (bad) sum = __builtin_nanf("");

    // The waves' sums meet.
    sum = groups_sum(sum);
    if (g == 0) {
        lds_m[wave][c] = mx;
        lds_l[wave][c] = sum;
    }
#pragma unroll
    for (int i = 0; i < VC; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) lds_o[wave][c][VC * (4 * g + r) + i] = o[i][r];
    __syncthreads();
    constexpr int EACH = 16 * D / (64 * WAVES);  // outputs per thread: neighbours of one row
    const int rr = tid * EACH / D, d0 = tid * EACH % D;
    float m = NEG_INF;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) m = fmaxf(m, lds_m[w][rr]);
    float l = 0.f, res[EACH];
#pragma unroll
    for (int e = 0; e < EACH; ++e) res[e] = 0.f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
        const float mw = lds_m[w][rr];
        const float f = mw == NEG_INF ? 0.f : __builtin_amdgcn_exp2f(mw - m);
        const float lw = lds_l[w][rr];
        l += lw * f;  // a NaN sum stays one, whatever its maximum
#pragma unroll
        for (int e = 0; e < EACH; ++e) res[e] += lds_o[w][rr][d0 + e] * f;
    }
    const int out_row = rt * 16 + rr;
    if (out_row >= rows) return;
    if (whole) {
        const float inv = l == 0.f ? 0.f : 1.f / l;  // a row that sees nothing is zero
        const int64_t at = (seq * a.q_len + out_row / gq) * a.q_heads + kvh * gq + out_row % gq;
        u32 w[EACH / 2];
#pragma unroll
        for (int e = 0; e < EACH / 2; ++e) w[e] = as_u32(f16x2{(f16)(res[2 * e] * inv), (f16)(res[2 * e + 1] * inv)});
        u32* p = reinterpret_cast<u32*>(static_cast<f16*>(a.out) + at * D + d0);
#pragma unroll
        for (int e = 0; e < EACH / 2; ++e) p[e] = w[e];
        return;
    }
    // Partial sums of a run: [pair][row tile][split][16][D + 2].
    float* part = a.part + (((pair * a.sh.row_tiles + rt) * a.sh.splits + split) * 16 + rr) * (D + 2);
#pragma unroll
    for (int e = 0; e < EACH; ++e) part[d0 + e] = res[e];
    if (d0 == 0) {
        part[D] = m;
        part[D + 1] = l;
    }
}

// One wave joins the runs of one query row.
template <int D>
__global__ void __launch_bounds__(256) attn_join_kernel(CacheAttnArgs a) {
    const int64_t q_row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (q_row >= a.n_seqs * a.q_len * a.q_heads) return;
    const int lane = threadIdx.x & 63;
    const int head = (int)(q_row % a.q_heads);
    const int64_t token = q_row / a.q_heads;
    const int64_t seq = token / a.q_len;
    int len = a.lens[seq];
    len = len < 0 ? 0 : len > a.max_len ? a.max_len : len;
    if (len <= a.sh.chunk) return;  // written by its only run
    const int gq = a.q_heads / a.c.kv_heads;
    const int row = (int)(token % a.q_len) * gq + head % gq;
    const int64_t pair = seq * a.c.kv_heads + head / gq;
    const int n = (len + a.sh.chunk - 1) / a.sh.chunk;
    const float* part = a.part + ((pair * a.sh.row_tiles + row / 16) * a.sh.splits * 16 + row % 16) * (D + 2);
    const int64_t step = 16LL * (D + 2);
    float m = NEG_INF;
    for (int i = 0; i < n; ++i) m = fmaxf(m, part[i * step + D]);
    float l = 0.f, o0 = 0.f, o1 = 0.f;
    for (int i = 0; i < n; ++i) {
        const float* p = part + i * step;
        const float f = p[D] == NEG_INF ? 0.f : __builtin_amdgcn_exp2f(p[D] - m);
        l += p[D + 1] * f;
        o0 += p[lane] * f;
        if (D > 64) o1 += p[64 + lane] * f;
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    f16* out = static_cast<f16*>(a.out) + q_row * D;
    out[lane] = (f16)(o0 * inv);
    if (D > 64) out[64 + lane] = (f16)(o1 * inv);
}

template <int BITS, int D, int GROUP>
hipError_t launch(const CacheAttnArgs& a, hipStream_t st) {
    const int64_t pairs = a.n_seqs * a.c.kv_heads;
    const dim3 grid((unsigned)((pairs + 7) / 8 * 8 * a.sh.row_tiles), (unsigned)a.sh.splits);
    attn_cache_kernel<BITS, D, GROUP><<<grid, 64 * WAVES, 0, st>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.sh.splits == 1) return e;
    const int64_t rows = a.n_seqs * a.q_len * a.q_heads;
    attn_join_kernel<D><<<dim3((unsigned)((rows + 3) / 4)), 256, 0, st>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_attn_cache(const CacheAttnArgs& a, hipStream_t st) {
    const int key = a.c.bits * 1000 + (a.c.bits == 16 ? 0 : a.c.group);
    if (a.c.head_dim == 64) {
        switch (key) {
            case 4032: return launch<4, 64, 32>(a, st);
            case 4064: return launch<4, 64, 64>(a, st);
            case 8032: return launch<8, 64, 32>(a, st);
            case 8064: return launch<8, 64, 64>(a, st);
            default: return launch<16, 64, 64>(a, st);
        }
    }
    switch (key) {
        case 4032: return launch<4, 128, 32>(a, st);
        case 4064: return launch<4, 128, 64>(a, st);
        case 4128: return launch<4, 128, 128>(a, st);
        case 8032: return launch<8, 128, 32>(a, st);
        case 8064: return launch<8, 128, 64>(a, st);
        case 8128: return launch<8, 128, 128>(a, st);
        default: return launch<16, 128, 128>(a, st);
    }
}

}  // namespace qmm
