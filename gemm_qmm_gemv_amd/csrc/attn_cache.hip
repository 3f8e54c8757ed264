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
// only at the end.  All cached rows are cut into equal shares, one per
// resident work-group, and whoever hands in the last part of a sequence joins
// them, in the same launch.
//
// 64 histories of 4000 to 16384 rows, 4 key heads of 128, 4 bits (348 MB) take
// 77 us, 4.5 TB/s; of 2000 to 8192 rows in 8 bits (369 MB) 77, 4.8, in fp16 (693 MB)
// 128, 5.4.  What is left above the rate of a copy (5.3) is 6 us before the
// first rows arrive and the ends: of the work-groups on a compute unit the one
// that was launched first is served first and done first.  The vector units
// alone would need 64 us.  Short calls are a chain of waits: lengths, page
// table, rows, the acknowledgement of partial sums, the join.
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
// second one of the same size would show.  Over an fp16 cache, where V is exact,
// they are rounded to fp16 once.
#include "layer_device.h"
#include "layer_kernels.h"

namespace qmm {
namespace {

constexpr int WAVES = 4;
constexpr int TILE = 32;  // cached rows per wave step
constexpr int STEP = CACHE_STEP;  // and per step of a work-group
constexpr uint32_t START = 2, LEAST = 2;  // see the kernel
static_assert(STEP == TILE * WAVES, "");
constexpr float NEG_INF = -__builtin_huge_valf();

__device__ __forceinline__ f32x4 mfma16(f16x8 a, f16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f16x8 frag(u32 a, u32 b, u32 c, u32 d) {
    return __builtin_bit_cast(f16x8, u32x4{a, b, c, d});
}
// Max / sum over the four lane groups that share a query row.
__device__ __forceinline__ float groups_max(float v) { return over_rows(v, [](float a, float b) { return fmaxf(a, b); }); }
__device__ __forceinline__ float groups_sum(float v) { return over_rows(v, add_f32); }
// a / b and the rest for 0 <= a < 2^20, 0 < b < 2^20: the quotient of the
// floats is off by less than 1/2 over b.
__device__ __forceinline__ int small_div(int a, int b) {
    return (int)(((float)a + 0.5f) * __builtin_amdgcn_rcpf((float)b));
}

// s_waitcnt: all vector memory done (expcnt and lgkmcnt not waited on).
constexpr int WAIT_MEMORY = 0x0F70;
// At most N vector memory operations in flight (vmcnt is split: bits 3:0 and
// 15:14); LDS operations done.
template <int N>
__device__ __forceinline__ void wait_loads() {
    static_assert(N < 64, "vmcnt");
    __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | (N >> 4) << 14);
    asm volatile("" : : : "memory");
}
__device__ __forceinline__ void wait_lds() {
    __builtin_amdgcn_s_waitcnt(0xC07F);
    asm volatile("" : : : "memory");
}

// Two neighbouring floats (8-byte aligned) past the caches of one die.
__device__ __forceinline__ void put2(float* p, float a, float b) {
    const uint64_t v = (uint64_t)__builtin_bit_cast(u32, b) << 32 | __builtin_bit_cast(u32, a);
    __hip_atomic_store(reinterpret_cast<uint64_t*>(p), v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void get2(const float* p, float& a, float& b) {
    const uint64_t v = __hip_atomic_load(reinterpret_cast<const uint64_t*>(p), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    const u32 lo = (u32)v, hi = (u32)(v >> 32);
    a = __builtin_bit_cast(float, lo);
    b = __builtin_bit_cast(float, hi);
}

template <int BITS, int D, int GROUP>
struct Cfg {
    static constexpr bool Q = BITS != 16;               // quantized
    static constexpr int NG = Q ? D / GROUP : 1;        // groups per row
    static constexpr int GD = Q ? GROUP : D;            // elements per group
    static constexpr int ROW = D * BITS / 8;            // bytes per row
    static constexpr int NG_BYTES = GD * BITS / 8;      // and per group
    static constexpr int KSTEPS = GD / 32;              // matrix steps per group
    static constexpr int KW = GD / 4 * BITS / 32;       // words per lane, group and cached row of K
    static constexpr int VC = D / 16;                   // values per lane and cached row of V
    static constexpr int VB = VC * BITS / 8;            // their bytes: 2, 4, 8 or 16
    static constexpr int VW = VB < 4 ? 1 : VB / 4;      // words holding them
    // Quantized rows go through LDS, two steps per wave.
    static constexpr int CHUNKS = ROW / 16;             // 16-byte chunks of a row
    static constexpr int LOADS = 32 * ROW / 1024;       // loads of a step's K rows (and of its V rows)
    static constexpr int STAGE = 2 * 32 * ROW + NG * 256;  // bytes of a step
    static constexpr int STAGES = 2;
    static constexpr int RING = Q ? WAVES * STAGES * STAGE : 16;
};

// Everything one 32-row step reads, in registers.
template <class C>
struct Raw {
    u32 k[2][C::NG][C::KW];
    u32 v[8][C::VW];
    u32x2 ks[2][C::NG], km[2][C::NG];  // four fp16 each: cached rows 4g..4g+3
    u32x2 vs[2], vm[2];
};

// Where a 32-row step's two halves of 16 rows lie: byte offsets of their rows
// and of their scales in each side's arrays.
struct Place {
    int64_t rows[2], scales[2];
};

// ---- Quantized rows.  Their pieces are small (4 to 8 bytes per lane and
// cached row) and asked for one by one they keep the address units busier than
// the memory: 24 loads per step took 57 us of a call of 106 us, in an earlier
// form, with all rows in the caches.  So a step's rows come into LDS as they lie, 1 KiB per load, and
// are taken apart from there.

// 16 (or 4) bytes per lane from memory to LDS at `to` + 16 (4) * lane, without
// passing through registers.  Instructions of their own text: the compiler,
// were it to know that they write LDS, would wait for all of them before any
// LDS read.  m0 holds the LDS address.  Scalar registers that a vector
// instruction wrote may be read by a memory instruction five wait states later,
// which the compiler sees to for its own instructions only: s_mov and s_nop
// make up five.  There is no register for the load to write, and the address
// registers are read when it is issued.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"  // m0 is a reserved register
__device__ __forceinline__ void rows_to_lds(const char* base, u32 offset, u32 to) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 3\n\tglobal_load_lds_dwordx4 %0, %1" : : "v"(offset), "s"(base), "s"(to) : "memory", "m0");
}
__device__ __forceinline__ void rows_to_lds(const char* from, u32 to) {
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 3\n\tglobal_load_lds_dwordx4 %0, off" : : "v"(from), "s"(to) : "memory", "m0");
}
__device__ __forceinline__ void words_to_lds(const char* from, u32 to) {
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 3\n\tglobal_load_lds_dword %0, off" : : "v"(from), "s"(to) : "memory", "m0");
}
#pragma clang diagnostic pop

// Where things lie in a stage.  K: chunk q of row r of a half at
// [r][q ^ fold(r)], so that the same chunk of 16 rows falls on 16 different
// places of the 256 bytes of banks.  V: row r at slot(r), so that rows 4 apart
// do.  Both permutations are their own inverses.
template <class C>
__device__ __forceinline__ int k_fold(int r) { return r / (256 / C::ROW) & (C::CHUNKS - 1); }
__device__ __forceinline__ int v_slot(int r) { return (r & ~3) | ((r ^ r >> 2) & 3); }

template <class C>
__device__ __forceinline__ void ask(const CacheView& cv, const Place& at, const char* scales, u32 to) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int n = 0; n < C::LOADS; ++n) {
        // Row and chunk, in their half, of what lands at 16 (64 n + lane).
        const int p = (n * 64 + lane) % (16 * C::CHUNKS), place = p / C::CHUNKS, q = p % C::CHUNKS;
        const u32 k_off = place * C::ROW + (q ^ k_fold<C>(place)) * 16, v_off = v_slot(place) * C::ROW + q * 16;
        const char* k = static_cast<const char*>(cv.k);
        const char* v = static_cast<const char*>(cv.v);
        if constexpr (16 * C::CHUNKS >= 64) {
            const int b = n * 64 / (16 * C::CHUNKS);
            rows_to_lds(k + at.rows[b], k_off, to + n * 1024);
            rows_to_lds(v + at.rows[b], v_off, to + 32 * C::ROW + n * 1024);
        } else {  // one load covers both halves
            const int64_t r0 = at.rows[0], r1 = at.rows[1], half = lane < 32 ? r0 : r1;
            rows_to_lds(k + half + k_off, to + n * 1024);
            rows_to_lds(v + half + v_off, to + 32 * C::ROW + n * 1024);
        }
    }
    // Per group 64 words: [K, V][8 quads of rows][scales, mins][2 pairs].
    const int64_t s0 = at.scales[0], s1 = at.scales[1], half = (lane >> 4 & 1) ? s1 : s0;
#pragma unroll
    for (int h = 0; h < C::NG; ++h)
        words_to_lds(scales + half + ((int64_t)h << (cv.page_shift + 1)), to + 64 * C::ROW + h * 256);
}
// The lane's array and place in it for the scale words of ask().
__device__ __forceinline__ const char* scale_words(const CacheView& cv, int lane) {
    const void* p = lane < 32 ? (lane & 2 ? cv.km : cv.ks) : (lane & 2 ? cv.vm : cv.vs);
    return static_cast<const char*>(p) + ((lane >> 2 & 3) * 4 + (lane & 1) * 2) * 2;
}

template <class C>
__device__ __forceinline__ void take_k(Raw<C>& r, const char* stage, int c, int g) {
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int h = 0; h < C::NG; ++h) {
            constexpr int BYTES = C::KW * 4;
            const int off = h * C::NG_BYTES + g * BYTES;  // of the row
            const char* row = stage + (16 * b + c) * C::ROW;
#pragma unroll
            for (int i = 0; i < (BYTES + 15) / 16; ++i) {
                const char* p = row + ((off / 16 + i) ^ k_fold<C>(c)) * 16 + off % 16;
                if constexpr (BYTES >= 16) {
                    const u32x4 w = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
                    for (int k = 0; k < 4; ++k) r.k[b][h][4 * i + k] = w[k];
                } else if constexpr (BYTES == 8) {
                    const u32x2 w = *reinterpret_cast<const u32x2*>(p);
                    r.k[b][h][0] = w[0];
                    r.k[b][h][1] = w[1];
                } else {
                    r.k[b][h][0] = *reinterpret_cast<const u32*>(p);
                }
            }
            const u32x4 w = *reinterpret_cast<const u32x4*>(stage + 64 * C::ROW + h * 256 + (4 * b + g) * 16);
            r.ks[b][h] = u32x2{w[0], w[1]};
            r.km[b][h] = u32x2{w[2], w[3]};
        }
}
template <class C>
__device__ __forceinline__ void take_v(Raw<C>& r, const char* stage, int c, int g) {
#pragma unroll
    for (int b = 0; b < 2; ++b) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const char* p = stage + (32 + 16 * b + v_slot(4 * g + j)) * C::ROW + c * C::VB;
            if constexpr (C::VB == 2) {
                r.v[4 * b + j][0] = *reinterpret_cast<const uint16_t*>(p);
            } else if constexpr (C::VB == 4) {
                r.v[4 * b + j][0] = *reinterpret_cast<const u32*>(p);
            } else {
                const u32x2 w = *reinterpret_cast<const u32x2*>(p);
                r.v[4 * b + j][0] = w[0];
                r.v[4 * b + j][1] = w[1];
            }
        }
        const u32x4 w = *reinterpret_cast<const u32x4*>(stage + 64 * C::ROW + (c * C::VC / C::GD) * 256 + 128 + (4 * b + g) * 16);
        r.vs[b] = u32x2{w[0], w[1]};
        r.vm[b] = u32x2{w[2], w[3]};
    }
}

// ---- fp16 rows: pieces of 16 bytes, straight into registers.  A step that is
// not there (`bytes` 0) is asked for all the same, of empty resources, which
// cost no memory access: the compiler counts the loads in flight and would
// wait for all of them behind loads that may not have been made.
template <class C>
__device__ __forceinline__ void load_k(Raw<C>& r, const CacheView& cv, const Place& at, u32 bytes, int c, int g) {
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        const rsrc_t kr = make_rsrc(static_cast<const char*>(cv.k) + at.rows[b], bytes);
        // Matrix step j takes elements 32 j + 8 g .. + 7.
#pragma unroll
        for (int j = 0; j < C::GD / 32; ++j) {
            u32 w[4];
            buffer_words<4, 16>(kr, c * C::ROW + g * 16 + j * 64, w);
#pragma unroll
            for (int i = 0; i < 4; ++i) r.k[b][0][4 * j + i] = w[i];
        }
    }
}
template <class C>
__device__ __forceinline__ void load_v(Raw<C>& r, const CacheView& cv, const Place& at, u32 bytes, int c, int g) {
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        const rsrc_t vr = make_rsrc(static_cast<const char*>(cv.v) + at.rows[b], bytes);
#pragma unroll
        for (int j = 0; j < 4; ++j) buffer_words<C::VW, C::VB>(vr, (4 * g + j) * C::ROW + c * C::VB, r.v[4 * b + j]);
    }
}

// Codes of matrix step j of a lane's K words, as fp16 in the order that
// q_order() gives Q: 4 bits, pairs (0,4) (1,5) (2,6) (3,7) of a word; 8 bits,
// pairs (0,2) (1,3) of each of two words.  A code alone in the low bits of an
// fp16 is the subnormal code * 2^-24, which the matrix cores take exactly; the
// 2^24 goes into the scale of the scores.
template <int BITS, int KW>
__device__ __forceinline__ f16x8 k_frag(const u32 (&w)[KW], int j) {
    if constexpr (BITS == 4) {
        const u32 v = w[j], m = 0x000F000Fu;
        return frag(v & m, v >> 4 & m, v >> 8 & m, v >> 12 & m);
    } else if constexpr (BITS == 8) {
        const u32 v0 = w[2 * j], v1 = w[2 * j + 1], m = 0x00FF00FFu;
        return frag(v0 & m, v0 >> 8 & m, v1 & m, v1 >> 8 & m);
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

// (v & mask) | magic in one instruction (an instruction holds one constant, so
// the compiler, which has two, makes it two).
__device__ __forceinline__ u32 and_or(u32 v, u32 mask, u32 magic) {
    u32 r;
    asm("v_and_or_b32 %0, %1, %2, %3" : "=v"(r) : "v"(v), "s"(mask), "v"(magic));
    return r;
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
            // 0x6400 + code is 1024 + code.  A nibble left at bits 4..7 under
            // 0x5400, whose last bit stands for 1/16, is 64 + code: one
            // shift serves two nibbles (17 ragged sequences 17.5 -> 17.3 us).
            const bool upper = BITS == 4 && bit % 8 == 4;
            const u32 mask = BITS == 8 ? 0x00FF00FFu : upper ? 0x00F000F0u : 0x000F000Fu;
            const u32 magic = upper ? 0x54005400u : MAGIC2;
            const f16x2 code = as_h2(and_or(x >> (bit % 16 & 8), mask, magic)) - as_h2(magic);
            const f16x2 sc = as_h2(s[p / 2][p % 2]), mn = as_h2(m[p / 2][p % 2]);
            out[p] = as_u32(__builtin_elementwise_fma(code, sc, mn));
        }
    }
    return frag(out[0], out[1], out[2], out[3]);
}

// Bits 15 and 31: of either half of a pair, whether its exponent is all ones
// (an infinity or a NaN): adding one to it carries into the sign's place.
__device__ __forceinline__ u32 carry_of_ones(u32 pair) { return (pair & 0x7C007C00u) + 0x04000400u; }
__device__ __forceinline__ bool not_finite(u32 pair, int half) {
    return ((pair >> (16 * half)) & 0x7C00u) == 0x7C00u;
}

// What a work-group needs of one unit (sequence, kv head, 16-row tile).
struct Segment {
    int64_t seq;
    int kvh, rt;
    int len;       // cached rows of the sequence
    int t0, t1;    // those of this run
    int runs, run; // runs of the unit, and which this is
};

template <int BITS, int D, int GROUP>
struct Shared {
    union {
        char ring[Cfg<BITS, D, GROUP>::RING];
        float o[WAVES][16][D + 4];  // rows start on different banks
    };
    float m[WAVES][16], l[WAVES][16];
    int sums[WAVES];
    int64_t seq;
    uint32_t base;
    bool last;
};

// `part_of(r)`: where run r of the unit leaves its sums: every thread's outputs,
// pair by pair so that a wave's accesses are contiguous, then (maximum, sum) of
// the 16 rows; 16 (D + 2) floats.
template <int BITS, int D, int GROUP, class PartOf>
__device__ __forceinline__ void attend(const CacheAttnArgs& a, const Segment& sg, int* count, PartOf part_of,
                                       Shared<BITS, D, GROUP>& sh) {
    using C = Cfg<BITS, D, GROUP>;
    constexpr int VC = C::VC;
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int c = lane & 15, g = lane >> 4;
    const int64_t seq = sg.seq;
    const int kvh = sg.kvh, len = sg.len, t0 = sg.t0, t1 = sg.t1;

    const int gq = a.group, rows = a.q_len * gq;
    const int first_limit = len - a.q_len + 1;  // cached rows that the first new token sees
    const int row = sg.rt * 16 + c;
    const bool live = row < rows;
    const int token = live ? small_div(row, gq) : 0;
    const int limit = live ? first_limit + token : 0;  // and that this lane's query row sees
    u32x4 qw[C::NG][C::KSTEPS];
    {
        const int64_t q_row = (seq * a.q_len + token) * a.q_heads + kvh * gq + (live ? row - token * gq : 0);
        const f16* qp = static_cast<const f16*>(a.q) + q_row * D;
#pragma unroll
        for (int h = 0; h < C::NG; ++h)
#pragma unroll
            for (int j = 0; j < C::KSTEPS; ++j)
                qw[h][j] = *reinterpret_cast<const u32x4*>(qp + (C::Q ? h * GROUP + g * (GROUP / 4) + 8 * j : 32 * j + 8 * g));
    }

    constexpr int STRIDE = TILE * WAVES;
    const int32_t* table = a.table + seq * a.table_stride;
    const int in_page = (1 << a.c.page_shift) - 1;
    bool bad = false;
    // Table entries of the wave's next 32 steps, two to a step, one per lane.
    // (An entry asked for step by step would be waited for with everything
    // asked for after it: the rows of the next step would never be under way
    // while this one's are worked on.)  Past the last row there is no
    // entry to read: that of row t0 stands in, and what comes of it is masked.
    int entries = 0, used = 32;
    auto place = [&](int first) {
        if (used == 32) {
            const int t = first + (lane >> 1) * STRIDE + (lane & 1) * 16;
            entries = table[(t < len ? t : t0) >> a.c.page_shift];
            asm volatile("" : "+v"(entries));  // waited for here and nowhere else
            used = 0;
        }
        Place at;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const int entry = __builtin_amdgcn_readlane(entries, 2 * used + b);
            const bool in = entry >= 0 && entry < a.c.pages;
            bad = bad || !in;
            const int64_t unit = (int64_t)(in ? entry : 0) * a.c.kv_heads + kvh;
            const int row0 = (first + 16 * b) & in_page;
            at.rows[b] = ((unit << a.c.page_shift) + row0) * C::ROW;
            at.scales[b] = ((unit * C::NG << a.c.page_shift) + row0) * 2;
        }
        ++used;
        return at;
    };

    // The first steps' rows are asked for before the queries are worked on.
    constexpr int PER_STEP = 2 * C::LOADS + C::NG;  // loads of ask()
    int first = t0 + wave * TILE;
    Raw<C> r;
    const char* const scales = C::Q ? scale_words(a.c, lane) : nullptr;
    char* const ring = sh.ring + (C::Q ? wave * C::STAGES * C::STAGE : 0);
    int stage = 0;
    if (first < t1) {
        if constexpr (C::Q) {
            ask<C>(a.c, place(first), scales, lds_address(ring));
        } else {
            const Place at = place(first);
            load_k<C>(r, a.c, at, 16 * C::ROW, c, g);
            load_v<C>(r, a.c, at, 16 * C::ROW, c, g);
        }
    }

    // Q operands and their sums per group.
    f16x8 qf[C::NG][C::KSTEPS];
    float qsum[C::NG];
    const float sc = a.scale * 1.44269504088896341f;  // scores in base 2
#pragma unroll
    for (int h = 0; h < C::NG; ++h) {
        qsum[h] = 0.f;
#pragma unroll
        for (int j = 0; j < C::KSTEPS; ++j) {
            const u32x4 w = live ? qw[h][j] : u32x4{0, 0, 0, 0};
            const f16x8 v = __builtin_bit_cast(f16x8, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                qf[h][j][i] = v[q_order<BITS>(i)];
                if constexpr (C::Q) qsum[h] += (float)v[i];
            }
        }
        if constexpr (C::Q) qsum[h] = groups_sum(qsum[h]) * sc;
    }

    f32x4 o[VC];
#pragma unroll
    for (int i = 0; i < VC; ++i) o[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    float mx = NEG_INF, sum = 0.f;

    for (; first < t1; first += STRIDE) {
        if constexpr (C::Q) {
            // The other stage is free (its reads are waited for) and takes
            // the next step's rows; then this step's own are waited for,
            // which were asked for before.
            wait_lds();
            if (first + STRIDE < t1) {
                ask<C>(a.c, place(first + STRIDE), scales, lds_address(ring + (stage ^ 1) * C::STAGE));
                wait_loads<PER_STEP>();
            } else {
                wait_loads<0>();
            }
            take_k<C>(r, ring + stage * C::STAGE, c, g);
        }
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
                    s[4 * b + i] = dot * (sc * 16777216.f) + low;
                } else {
                    s[4 * b + i] = acc[0][i] * sc;
                }
            }
        }
        // fp16: the keys' registers are free for the next step's, and the
        // values' once this step's are used.
        [[maybe_unused]] Place next;
        [[maybe_unused]] const u32 next_bytes = first + STRIDE < t1 ? 16 * C::ROW : 0;
        if constexpr (C::Q) {
            take_v<C>(r, ring + stage * C::STAGE, c, g);
        } else {
            next = place(first + STRIDE);
            load_k<C>(r, a.c, next, next_bytes, c, g);
        }
        if (first + TILE > first_limit) {
            // The end of a sequence: rows of pages behind it may hold
            // anything (a NaN times a probability of zero is NaN), so their
            // values are cleared and their scores dropped.  A drafted
            // token's row is seen by some rows only: if its values are not
            // finite they are cleared as well and the rows that see it get
            // a NaN score instead.
            [[maybe_unused]] u32 beyond[4] = {0, 0, 0, 0};  // of cached rows 2p and 2p + 1: bits 15 and 31
            if constexpr (C::Q) {
                // A value leaves fp16 with a scale or min that is not finite,
                // or with finite ones and a high code.  |scale| times the highest
                // code plus |min|, rounded once as the values are, bounds them
                // all, and only where that leaves fp16 are they looked at.
                constexpr float TOP = (float)((1 << BITS) - 1);
                u32 reach = 0;
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    const f16x2 sc = as_h2(r.vs[p / 2][p % 2] & 0x7FFF7FFFu), mn = as_h2(r.vm[p / 2][p % 2] & 0x7FFF7FFFu);
                    reach |= carry_of_ones(as_u32(__builtin_elementwise_fma(sc, f16x2{(f16)TOP, (f16)TOP}, mn)));
                }
                if (__any(reach & 0x80008000u)) {
#pragma unroll
                    for (int i = 0; i < VC; ++i) {
                        const u32x4 w = __builtin_bit_cast(u32x4, v_frag<BITS>(r.v, i, r.vs, r.vm));
#pragma unroll
                        for (int p = 0; p < 4; ++p) beyond[p] |= carry_of_ones(w[p]);
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int t = first + 16 * (j / 4) + 4 * g + j % 4;
                bool odd = false;
                if constexpr (C::Q) {
                    odd = (beyond[j / 2] & (j % 2 ? 0x80000000u : 0x8000u)) != 0;
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
        // Running maximum and sum.  The sums are kept relative to a maximum
        // that lags: it moves only when a score is past it by 2^8 (fp16 holds
        // 2^15).  A row that sees nothing yet keeps -inf; 0 stands in for it
        // so that no inf - inf is formed.
        float top = fmaxf(fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3])), fmaxf(fmaxf(s[4], s[5]), fmaxf(s[6], s[7])));
        top = groups_max(top);
        if (__any(top - mx > 8.f)) {
            const float m2 = fmaxf(mx, top);
            const float f = mx == NEG_INF ? 0.f : __builtin_amdgcn_exp2f(mx - m2);
            sum *= f;
#pragma unroll
            for (int i = 0; i < VC; ++i) o[i] = o[i] * f;
            mx = m2;
        }
        const float base = mx == NEG_INF ? 0.f : mx;
        u32 hi[4], lo[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float p0 = __builtin_amdgcn_exp2f(s[2 * j] - base), p1 = __builtin_amdgcn_exp2f(s[2 * j + 1] - base);
            sum += p0;
            sum += p1;
            if constexpr (C::Q) {
                hi[j] = __builtin_bit_cast(u32, __builtin_amdgcn_cvt_pkrtz(p0, p1));
                const f16x2 h2 = as_h2(hi[j]);
                lo[j] = __builtin_bit_cast(u32, __builtin_amdgcn_cvt_pkrtz(__builtin_fmaf((float)h2[0], -1.f, p0),
                                                                           __builtin_fmaf((float)h2[1], -1.f, p1)));
            } else {
                hi[j] = as_u32(f16x2{(f16)p0, (f16)p1});
            }
        }
#pragma unroll
        for (int i = 0; i < VC; ++i) {
            const f16x8 vf = v_frag<BITS>(r.v, i, r.vs, r.vm);
            o[i] = mfma16(vf, frag(hi[0], hi[1], hi[2], hi[3]), o[i]);
            if constexpr (C::Q) o[i] = mfma16(vf, frag(lo[0], lo[1], lo[2], lo[3]), o[i]);
        }
        if constexpr (C::Q)
            stage ^= 1;
        else
            load_v<C>(r, a.c, next, next_bytes, c, g);
    }
    // A page index outside the cache: nothing was read there, and every row
    // of this sequence and head becomes NaN.
    if (bad) sum = __builtin_nanf("");

    // The waves' sums meet (where the rows' ring was).
    sum = groups_sum(sum);
    __syncthreads();
    if (g == 0) {
        sh.m[wave][c] = mx;
        sh.l[wave][c] = sum;
    }
#pragma unroll
    for (int i = 0; i < VC; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) sh.o[wave][c][VC * (4 * g + k) + i] = o[i][k];
    __syncthreads();
    constexpr int EACH = 16 * D / (64 * WAVES);  // outputs per thread: neighbours of one row
    const int rr = tid * EACH / D, d0 = tid * EACH % D;
    float m = NEG_INF, l = 0.f, res[EACH];
#pragma unroll
    for (int w = 0; w < WAVES; ++w) m = fmaxf(m, sh.m[w][rr]);
#pragma unroll
    for (int e = 0; e < EACH; ++e) res[e] = 0.f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
        const float mw = sh.m[w][rr];
        const float f = mw == NEG_INF ? 0.f : __builtin_amdgcn_exp2f(mw - m);
        l += sh.l[w][rr] * f;  // a NaN sum stays one, whatever its maximum
#pragma unroll
        for (int e = 0; e < EACH; ++e) res[e] += sh.o[w][rr][d0 + e] * f;
    }
    const int out_row = sg.rt * 16 + rr;
    bool write = out_row < rows;
    if (sg.runs > 1) {
        // The work-group that hands in the unit's last run joins them all.
        // The stores and loads are device-scope atomics, which pass the L2 of
        // each die; the count goes up only after every thread's stores are
        // acknowledged.
        if (write) {
            float* part = part_of(sg.run);
#pragma unroll
            for (int e = 0; e < EACH; e += 2) put2(part + (e / 2 * 64 * WAVES + tid) * 2, res[e], res[e + 1]);
            if (d0 == 0) put2(part + 16 * D + rr * 2, m, l);
        }
        __builtin_amdgcn_s_waitcnt(WAIT_MEMORY);
        __syncthreads();
        if (tid == 0) {
            sh.last = __hip_atomic_fetch_add(count, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == sg.runs - 1;
            if (sh.last) __hip_atomic_store(count, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        __syncthreads();
        write = write && sh.last;
        if (write) {
            m = NEG_INF;
            l = 0.f;
#pragma unroll
            for (int e = 0; e < EACH; ++e) res[e] = 0.f;
            // Several runs are asked for before the first is used (behind the
            // last one it stands in, and is left out).
            constexpr int AT_ONCE = D == 128 ? 8 : 12;
            for (int i = 0; i < sg.runs; i += AT_ONCE) {
                float mi[AT_ONCE], li[AT_ONCE], x[AT_ONCE][EACH];
#pragma unroll
                for (int k = 0; k < AT_ONCE; ++k) {
                    const float* from = part_of(i + k < sg.runs ? i + k : sg.runs - 1);
                    get2(from + 16 * D + rr * 2, mi[k], li[k]);
#pragma unroll
                    for (int e = 0; e < EACH; e += 2) get2(from + (e / 2 * 64 * WAVES + tid) * 2, x[k][e], x[k][e + 1]);
                }
#pragma unroll
                for (int k = 0; k < AT_ONCE; ++k) {
                    if (i + k >= sg.runs) continue;
                    const float m2 = fmaxf(m, mi[k]);
                    const float f0 = m == NEG_INF ? 0.f : __builtin_amdgcn_exp2f(m - m2);
                    const float f1 = mi[k] == NEG_INF ? 0.f : __builtin_amdgcn_exp2f(mi[k] - m2);
                    m = m2;
                    l = l * f0 + li[k] * f1;
#pragma unroll
                    for (int e = 0; e < EACH; ++e) res[e] = res[e] * f0 + x[k][e] * f1;
                }
            }
        }
    }
    if (write) {
        const float inv = l == 0.f ? 0.f : 1.f / l;  // a row that sees nothing is zero
        const int i = small_div(out_row, gq);
        const int64_t at = (seq * a.q_len + i) * a.q_heads + kvh * gq + (out_row - i * gq);
        u32* p = reinterpret_cast<u32*>(static_cast<f16*>(a.out) + at * D + d0);
#pragma unroll
        for (int e = 0; e < EACH / 2; ++e) p[e] = as_u32(f16x2{(f16)(res[2 * e] * inv), (f16)(res[2 * e + 1] * inv)});
    }
    __syncthreads();  // the next segment writes the shared sums
}

// All steps of all units lie behind each other, a sequence's units together.
// The work-groups take equal shares of them, whatever the lengths, so a share
// may begin and end inside a unit; sums of such a run go to the workspace, at
// most two per work-group.
template <int BITS, int D, int GROUP>
__global__ void __launch_bounds__(64 * WAVES, cache_resident(BITS, D)) attn_cache_kernel(CacheAttnArgs a) {
    __shared__ __align__(16) Shared<BITS, D, GROUP> sh;
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int per_seq = a.c.kv_heads * a.row_tiles;  // units of a sequence
    auto length = [&](int64_t seq) {
        const int n = a.lens[seq];
        return n < 0 ? 0 : n > a.max_len ? a.max_len : n;
    };
    auto steps_of = [&](int len) { return (uint32_t)(len + STEP - 1) / STEP; };
    // A unit is counted as START steps more than it has: what beginning and
    // joining a run costs.  With 0, 1, 2 and 4 of them drafts over 8 bits
    // (5 steps a share) take 24.9, 22.8, 22.2 and 22.5 us, 17 ragged sequences (2
    // steps) 16.9, 15.7, 15.3 and 15.1, one of 1500 rows 8.8, 10.7, 8.8 and 8.8, 64
    // long histories (25 steps) 77 to 78 with any of them.
    auto size_of = [&](int len) { return len == 0 ? 0u : steps_of(len) + START; };

    Segment sg;
    uint32_t pos = 0, end = 0, me = 0, base = 0, unit = 0, size = 0;
    bool few = true;
    int last_len = 0;
    auto length_of = [&](int64_t seq) {
        return few ? __builtin_amdgcn_readlane(last_len, (int)seq) : uniform(length(seq));
    };
    const int n = (int)a.n_seqs;
    uint32_t small = 1, more = 0;
    // Share i begins at i * small + min(i, more): the first `more` shares have
    // one step more.
    auto begin_of = [&](uint32_t i) { return i * small + (i < more ? i : more); };
    auto share_of = [&](uint32_t step) {
        const uint32_t edge = more * (small + 1);
        return step < edge ? step / (small + 1) : more + (step - edge) / small;
    };
    if (a.share) {
        // Steps before each lane's (or thread's) sequences, and in all.  Up to
        // 64 sequences: a lane each, in every wave, and no meeting; the
        // lengths stay in the lanes.
        few = n <= 64;
        const int each = few ? 1 : (n + 64 * WAVES - 1) / (64 * WAVES);
        const int s0 = (few ? lane : tid) * each, s1 = s0 + each < n ? s0 + each : n;
        uint32_t own = 0;
        for (int s = s0; s < s1; ++s) {
            last_len = length(s);
            own += size_of(last_len);
        }
        uint32_t before = own;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const uint32_t x = __shfl_up(before, o, 64);
            if (lane >= o) before += x;
        }
        uint32_t total = __builtin_amdgcn_readlane(before, 63);
        if (!few) {
            if (lane == 63) sh.sums[wave] = before;
            __syncthreads();
            total = 0;
#pragma unroll
            for (int w = 0; w < WAVES; ++w) {
                if (w < wave) before += sh.sums[w];
                total += sh.sums[w];
            }
        }
        before -= own;
        total = uniform((int)(total * per_seq));
        // No more shares than make LEAST steps each (one sequence of 1500 rows
        // with 1, 2 and 4: 9.2, 8.8 and 11.8 us; 17 ragged ones 15.3, 15.3 and
        // 14.6; drafts and long ones the same).  Neighbouring shares go
        // to one die (work-groups go round the eight), so row tiles that read
        // the same cached rows share its L2.
        uint32_t shares = total / LEAST;
        if (shares < 8) shares = total < 8 ? total : 8;
        if (shares > gridDim.x) shares = gridDim.x;
        if (shares > 8) shares &= ~7u;
        me = shares % 8 == 0 ? blockIdx.x % 8 * (shares / 8) + blockIdx.x / 8 : blockIdx.x;
        if (blockIdx.x < shares) {
            small = total / shares;
            more = total - small * shares;
            pos = begin_of(me);
            end = begin_of(me + 1);
        }
        // The sequence that the share begins in, and the steps before it.
        const bool here = pos < end && pos >= before * per_seq && pos < (before + own) * per_seq;
        if (few) {
            const int at = __builtin_ctzll(__ballot(here) | 1ull << 63);
            sg.seq = at;
            base = __builtin_amdgcn_readlane(before, at);
        } else {
            if (here) {
                uint32_t up = before;
                int s = s0;
                for (;; ++s) {
                    const uint32_t st = size_of(length(s));
                    if (pos < (up + st) * per_seq) break;
                    up += st;
                }
                sh.seq = s;
                sh.base = up;
            }
            __syncthreads();
            sg.seq = uniform((int)sh.seq);
            base = uniform((int)sh.base);
        }
        if (pos < end) {
            sg.len = length_of(sg.seq);
            size = size_of(sg.len);
            unit = (pos - base * per_seq) / size;
        }
    } else {
        // One unit per work-group, in one run.
        sg.seq = blockIdx.x / per_seq;
        unit = blockIdx.x % per_seq;
        sg.len = uniform(length(sg.seq));
        end = 1;
    }
    while (pos < end) {
        sg.kvh = small_div(unit, a.row_tiles);
        sg.rt = unit - sg.kvh * a.row_tiles;
        sg.t0 = 0;
        sg.t1 = sg.len;
        sg.runs = 1;
        sg.run = 0;
        uint32_t one = me, behind = 1;
        bool leads = true, some = true;
        if (a.share) {
            const uint32_t start = base * per_seq + unit * size, first = start + START;  // where it begins, its first step
            behind = start + size;
            const uint32_t from = pos > first ? pos : first, to = behind < end ? behind : end;
            some = from < to;
            sg.t0 = (from - first) * STEP;
            if ((int)((to - first) * STEP) < sg.len) sg.t1 = (to - first) * STEP;
            // The unit's runs are handed in by shares from `one` on; it is
            // the first segment of all of them but for the first share, if
            // that has steps of units before.
            if (some && (from > first || to < behind)) {
                one = share_of(first);
                sg.runs = (int)(share_of(behind - 1) - one) + 1;
                sg.run = (int)(me - one);
                leads = begin_of(one) >= start;
            }
        }
        if (some)
            attend<BITS, D, GROUP>(a, sg, a.count + one, [&](int r) {
                return a.part + ((int64_t)(one + r) * 2 + (r > 0 || leads ? 0 : 1)) * 16 * (D + 2);
            }, sh);
        if (behind >= end) break;
        pos = behind;
        if (++unit == (uint32_t)per_seq) {
            unit = 0;
            base += size;
            do {
                ++sg.seq;
                sg.len = length_of(sg.seq);
                size = size_of(sg.len);
            } while (size == 0);
        }
    }
    if (!a.share) return;
    // Sequences without cached rows are in nobody's share.
    const int64_t width = (int64_t)a.q_len * a.q_heads * D / 8;
    for (int64_t s = blockIdx.x; s < n; s += gridDim.x)
        if (length(s) == 0)
            for (int64_t i = tid; i < width; i += 64 * WAVES) static_cast<u32x4*>(a.out)[s * width + i] = u32x4{0, 0, 0, 0};
}

template <int BITS, int D, int GROUP>
hipError_t launch(const CacheAttnArgs& a, hipStream_t st) {
    attn_cache_kernel<BITS, D, GROUP><<<dim3((unsigned)a.groups), 64 * WAVES, 0, st>>>(a);
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
