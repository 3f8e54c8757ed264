// attn_prompt.hip -- causal attention over whole prompts packed behind each
// other, with grouped heads:
//
//   O[i] = sum_j exp(S[i][j] - max_j S[i][j]) V[j] / sum_j exp(S[i][j] - max_j S[i][j]),
//   S[i][j] = scale * Q[i] . K[j],  j from the start of i's sequence to i.
//
// Bound by the matrix cores, the vector units (exponentials) and LDS, which
// have about the same load.  Short steps on many waves keep all three busy
// best: a wave holds 32 query rows of one head and takes 32 keys a step, and
// three (head size 128) or four waves on each SIMD are at different places of
// it.  8192 tokens, 32 query and 4 key heads of 128: 557 to 568 us among others,
// 583 to 604 alone under a kernel trace: 910 to 987 TFLOP/s, 79 to 84 % of what a
// large fp16 matrix product of the library reaches on the card (1146 to 1178; the
// clock drops to 1.9 GHz under either); of 64: 334 us, 822 TFLOP/s, vector units
// 77 % busy, as a score costs as much there and its products half.  Tried and
// slower at 128, where this took 558: two waves per SIMD with the next step's
// scores formed early (593 us), the same with matrix and vector instructions
// interleaved by hand (631), 64 rows per wave (829), K and V staged through
// registers (645).
//
// Query rows are cut by their place in the packing and not by sequence: a tile
// of rows may hold the end of one sequence and several short ones, which costs
// masked work at the borders only and needs no list of tiles.
//
// The products are transposed so that no value changes lanes between them:
//   S^T = K Q^T puts, in lane l, scores of query row l % 32 at sixteen of 32
//   keys; O^T = V^T P^T takes them as its right operand as they are, with V^T
//   read in the same order of keys.  A query row's maximum and sum need one
//   exchange with lane l ^ 32.
#include <type_traits>

#include "layer_device.h"
#include "layer_kernels.h"

namespace qmm {
namespace {

constexpr float NEG_INF = -__builtin_huge_valf();
typedef f16 f16x4v __attribute__((ext_vector_type(4)));

__device__ __forceinline__ f32x16 mfma32(f16x8 a, f16x8 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}

// First row of the sequence that each lane's packed row belongs to, or -1 if it
// belongs to none: the last offset that is not past the row.  Up to 63
// sequences take one load, an offset per lane, which all lanes then look
// through; more take a search.  Offsets are clamped so that whatever they
// hold stays in bounds.
template <int R>
__device__ __forceinline__ void sequence_starts(const int32_t* offsets, int n_seqs, int64_t tokens, const int (&row)[R],
                                                int (&start)[R]) {
    int before[R];  // offsets that are not past the row
#pragma unroll
    for (int r = 0; r < R; ++r) before[r] = start[r] = 0;
    if (n_seqs < 64) {
        const int lane = threadIdx.x & 63;
        const int mine = offsets[lane < n_seqs ? lane : n_seqs];
        for (int i = 0; i <= n_seqs; ++i) {
            const int at = __builtin_amdgcn_readlane(mine, i);
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (at <= row[r]) {
                    before[r] = i + 1;
                    start[r] = at;
                }
        }
    } else {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            int lo = 0, hi = n_seqs + 1;
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                const int at = offsets[mid];
                if (at <= row[r]) {
                    lo = mid + 1;
                    start[r] = at;
                } else {
                    hi = mid;
                }
            }
            before[r] = lo;
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        if (start[r] < 0) start[r] = 0;
        if (before[r] == 0 || before[r] > n_seqs || row[r] >= tokens) start[r] = -1;
    }
}

typedef short s16x4 __attribute__((ext_vector_type(4)));

// Max over lanes l and l ^ 32.
__device__ __forceinline__ float halves_max(float v) {
    return over_halves(v, [](float a, float b) { return fmaxf(a, b); });
}

// 16 bytes per lane from memory to LDS without passing through registers: lane
// i's land at `to` + 16 i.  An instruction of its own text, because the
// compiler waits for all loads before any later LDS read if it knows that
// this one writes LDS; here readers do, before the barrier they share.  m0
// holds the LDS address.  Scalar registers that a vector instruction wrote may
// be read by a memory instruction five wait states later, which the compiler
// sees to for its own instructions only: s_mov and s_nop make up five (the
// same times as with the one that m0 needs).  There is no register for the
// load to write, and the address registers are read when it is issued.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"  // m0 is a reserved register
__device__ __forceinline__ void load_to_lds(u32x4 rsrc, u32 offset, u32 to) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 3\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds"
                 :
                 : "v"(offset), "s"(rsrc), "s"(to)
                 : "memory", "m0");
}
#pragma clang diagnostic pop
// Buffer descriptor of everything from p on (offsets are clamped by the caller).
__device__ __forceinline__ u32x4 open_rsrc(const void* p) {
    const uint64_t a = reinterpret_cast<uint64_t>(p);
    return u32x4{(u32)uniform((int)a), (u32)uniform((int)(a >> 32)) & 0xffffu, 0xffffffffu, (u32)RSRC_WORD3};
}

// A tile of K or V lies in LDS row behind row, as the direct loads put it; the
// 16-byte chunk c of row r is at place c ^ swizzle(r) of its row.  One access
// to K reads the same chunk of 32 rows, one to V 32 bytes each of four rows:
// the exclusive or puts what an access touches at a time on different banks.
template <int D>
__device__ __forceinline__ int k_swizzle(int r) { return D == 128 ? r & 15 : r >> 1 & 7; }
template <int D>
__device__ __forceinline__ int v_swizzle(int r) { return D == 128 ? (r & 3) << 2 : (r >> 1 & 1) << 2; }

// RW waves hold 32 query rows each; KW of them share the rows, each taking 32 of
// every 32 KW keys, and join at the end.
template <int D, int RW, int KW, int BN>
__global__ void __launch_bounds__(64 * RW * KW, BN == 32 ? 3 : 2) attn_prompt_kernel(PromptArgs a) {
    constexpr int BM = RW * 32, T = 64 * RW * KW;
    constexpr int CR = D / 8;                // 16-byte chunks of a row
    constexpr int LROWS = 64 / CR;           // rows that one load of a wave covers
    constexpr int LOADS = BN * CR / T;       // loads of a tile of K (or of V) per wave
    constexpr int BUF = BN * D;
    __shared__ __align__(1024) f16 lds[4 * BUF];
    __shared__ int lds_bad[2][BN], lds_any[2];
    __shared__ int lds_lo[RW], lds_hi[RW], lds_late[RW], lds_large[RW];
    f16* const lds_k = lds;
    f16* const lds_v = lds + 2 * BUF;
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int rw = wave % RW, kw = wave / RW;
    const int h = lane >> 5, l32 = lane & 31;
    // Grid: kv heads, query heads of each, tiles of rows.  Work-groups go
    // round the eight dies, so with eight kv heads, or a divisor of eight,
    // one die reads few of them.  Later rows see more keys: they start first.
    const int kvh = blockIdx.x, head = kvh * (int)gridDim.y + blockIdx.y;
    const int tile = (int)(gridDim.z - 1 - blockIdx.z);
    const int row0 = tile * BM, wrow0 = row0 + rw * 32;
    const int row = wrow0 + l32;

    // The running maximum is of Q.K itself and the scale is applied in the
    // exponent, which needs a positive one: a negative scale negates Q
    // (exact), scale 0 makes Q zero.
    const float sc = a.scale == 0.f ? 1.f : fabsf(a.scale) * 1.44269504088896341f;
    const u32 flip = a.scale < 0.f ? 0x80008000u : 0u;
    u32x4 qw[D / 16];
    {
        const int64_t at = row < a.tokens ? row : a.tokens - 1;
        const f16* qp = static_cast<const f16*>(a.q) + at * a.q_stride + head * D;
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
            qw[j] = *reinterpret_cast<const u32x4*>(qp + 16 * j + 8 * h) ^ flip;
            if (a.scale == 0.f) qw[j] = u32x4{0, 0, 0, 0};
        }
    }

    // Keys start..row of this lane's query row; for the wave and the
    // work-group the earliest and latest start and the last row.
    int start;
    {
        const int rows[1] = {row};
        int starts[1];
        sequence_starts<1>(a.offsets, (int)a.n_seqs, a.tokens, rows, starts);
        start = starts[0];
    }
    // (Starts do not decrease from row to row in a packing, so the first and
    // last row that a sequence covers hold them.)
    const u32 covered = (u32)__ballot(start >= 0);
    const int from = covered ? __builtin_ctz(covered) : 0, to = covered ? 31 - __builtin_clz(covered) : 0;
    const int wlo = covered ? __builtin_amdgcn_readlane(start, from) : 0x7fffffff;
    const int wlate = covered ? __builtin_amdgcn_readlane(start, to) : 0;
    const int whi = covered ? wrow0 + to : -1;
    // Whether scores may be so large that s sc - mx sc has to be formed from
    // s - mx (see the step).  mx sc as a rounded number is off by up to 2^-24 of
    // itself: a factor that all probabilities of a row share and the quotient
    // drops, but past 2^26 one of more than 2^4, which with the lag's 2^8 nears
    // what fp16 holds.  With fp16 keys, whose rows are at most 65504 D^1/2 long,
    // a score is that large only if the query's row is longer than 1024 D^-1/2 / sc
    // (710 at D 128 and scale 128^-1/2).
    float square = 0.f;
#pragma unroll
    for (int j = 0; j < D / 16; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) square = __builtin_amdgcn_fdot2(as_h2(qw[j][i]), as_h2(qw[j][i]), square, false);
    square = over_halves(square, add_f32);
    const bool large = __any(!(square * (D * sc * sc) <= 1024.f * 1024.f));
    if (lane == 0) {
        lds_large[rw] = large;
        lds_lo[rw] = wlo;
        lds_hi[rw] = whi;
        lds_late[rw] = wlate;
    }
    if (tid < 2 * BN) (&lds_bad[0][0])[tid] = 0;
    if (tid < 2) lds_any[tid] = 0;
    __syncthreads();
    int blo = 0x7fffffff, bhi = -1, blate = 0, apart = 0;
#pragma unroll
    for (int w = 0; w < RW; ++w) {
        blo = lds_lo[w] < blo ? lds_lo[w] : blo;
        bhi = lds_hi[w] > bhi ? lds_hi[w] : bhi;
        blate = lds_late[w] > blate ? lds_late[w] : blate;
        apart |= lds_large[w];
    }
    blo = uniform(blo);
    bhi = uniform(bhi);
    blate = uniform(blate);
    apart = uniform(apart);
    if (bhi < 0) return;

    f32x16 o[D / 32];
    float mx = NEG_INF, sum = 0.f;
#pragma unroll
    for (int n = 0; n < D / 32; ++n) o[n] = f32x16{};
    const f16* kp = static_cast<const f16*>(a.k) + kvh * D;
    const f16* vp = static_cast<const f16*>(a.v) + kvh * D;
    const int tiles = (bhi - blo) / BN + 1;

    // Tile j of K and V goes from memory to buffer b of LDS without passing
    // through registers.  Rows behind the last key repeat it; they are masked.
    auto fetch = [&](int j, int b) {
        const int t0 = blo + j * BN, last = bhi - t0;
        const u32x4 kr = open_rsrc(kp + (int64_t)t0 * a.k_stride), vr = open_rsrc(vp + (int64_t)t0 * a.v_stride);
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const int r0 = (i * (T / 64) + wave) * LROWS, r = r0 + lane / CR, c = lane % CR;
            const int at = r < last ? r : last;
            load_to_lds(kr, (u32)(at * (int)a.k_stride + 8 * (c ^ k_swizzle<D>(r))) * 2, lds_address(lds_k + b * BUF + r0 * D));
            load_to_lds(vr, (u32)(at * (int)a.v_stride + 8 * (c ^ v_swizzle<D>(r))) * 2, lds_address(lds_v + b * BUF + r0 * D));
        }
    };
    // In a tile that not every row sees, values that are not finite must not
    // meet a probability of zero (their product is NaN): they are cleared,
    // and the rows that do see their key get a NaN score.  A thread looks at
    // the chunks that it loaded itself, before the waves meet.
    auto partial = [&](int j) { return blo + j * BN + BN - 1 > row0 || blo + j * BN < blate; };
    auto clean = [&](int j, int b) {
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const int at = i * T + tid;
            u32x4* p = reinterpret_cast<u32x4*>(lds_v + b * BUF) + at;
            const u32x4 v = *p;
            u32 odd = 0;  // an exponent of ones carries into the sign's place
#pragma unroll
            for (int k = 0; k < 4; ++k) odd |= (v[k] & 0x7C007C00u) + 0x04000400u;
            if (odd & 0x80008000u) {
                *p = u32x4{0, 0, 0, 0};
                lds_bad[b][at / CR] = j + 1;  // of this tile: never cleared
                lds_any[b] = j + 1;
            }
        }
    };

    // Scores of 32 keys, half u of the tile in buffer b.
    const int k_lane = l32 * D + 8 * (h ^ k_swizzle<D>(l32));
    const int q16 = lane & 15, v_row = 4 * h + (q16 >> 2);
    const int v_lane = v_row * D + 8 * ((2 * (lane >> 4 & 1) + (q16 >> 1 & 1)) ^ v_swizzle<D>(v_row)) + 4 * (q16 & 1);
    // One step of 32 keys, number u of tile j, which lies in buffer j & 1.
    auto step = [&](int j, int u, bool cleaned, auto apart) {
        const int t = blo + j * BN + 32 * u;
        if (t > whi || t + 31 < wlo) return;
        const int b = j & 1;
        const f16* kb = lds_k + b * BUF + 32 * u * D;
        f32x16 s = {};
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
            s = mfma32(*reinterpret_cast<const f16x8*>(kb + (k_lane ^ (16 * i))), __builtin_bit_cast(f16x8, qw[i]), s);
        // (Cleared for the work-group, so marked by waves that see every key too.)
        if (cleaned && __builtin_expect(uniform(lds_any[b]) == j + 1, 0)) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (lds_bad[b][32 * u + 8 * (i / 4) + 4 * h + i % 4] == j + 1) s[i] = __builtin_nanf("");
        }
        if (t + 31 > wrow0 || t < wlate) {  // not every row sees every key
            // This row sees key t + k if start <= t + k <= row: one unsigned
            // comparison of its distance from the start.
            const u32 seen = start < 0 ? 0 : (u32)(row - start + 1), from_start = (u32)(t + 4 * h - start);
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (from_start + (u32)(8 * (i / 4) + i % 4) >= seen) s[i] = NEG_INF;
        }
        float top = fmaxf(s[0], s[1]);
#pragma unroll
        for (int i = 2; i < 16; i += 2) top = fmaxf(fmaxf(top, s[i]), s[i + 1]);
        top = halves_max(top);
        // The sums are kept relative to a maximum that lags: it moves only
        // when a score is past it by 2^8 (fp16 holds 2^15), which is rare
        // after the first tiles.
        if (__any((top - mx) * sc > 8.f)) {
            const float m2 = fmaxf(mx, top);
            const float f = mx == NEG_INF ? 0.f : __builtin_amdgcn_exp2f((mx - m2) * sc);
            mx = m2;
            sum *= f;
#pragma unroll
            for (int n = 0; n < D / 32; ++n) o[n] = o[n] * f;
        }
        // One multiply-add per score, or with large ones the difference first.
        const float base = mx == NEG_INF ? 0.f : apart ? mx : mx * sc;
        auto power = [&](float x) { return __builtin_amdgcn_exp2f(apart ? (x - base) * sc : __builtin_fmaf(x, sc, -base)); };
        // Probabilities are rounded to fp16 for the second product (to the
        // nearest: two in one instruction, as cutting them is), and their
        // sum is of the rounded values, so that weights still add up to one.
        u32 w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float p0 = power(s[2 * i]), p1 = power(s[2 * i + 1]);
            w[i] = as_u32(f16x2{(f16)p0, (f16)p1});
            sum = __builtin_amdgcn_fdot2(as_h2(w[i]), f16x2{(f16)1.f, (f16)1.f}, sum, false);
        }
        // V^T operand: lane (h, l32) wants value 32 n + l32 of keys
        // 16 e + 4 h + 0..3 and + 8..11.  The transposing read takes four
        // rows of 16 values per 16 lanes, 8 bytes from each lane, and gives
        // lane i the four rows' value i.
        const f16* vb = lds_v + b * BUF + 32 * u * D;
        typedef __attribute__((address_space(3))) s16x4* lds_ptr;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const f16x8 pf = __builtin_bit_cast(f16x8, u32x4{w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]});
#pragma unroll
            for (int n = 0; n < D / 32; ++n) {
                const s16x4 v0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(vb + 16 * e * D + (v_lane ^ (32 * n))));
                const s16x4 v1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(vb + (16 * e + 8) * D + (v_lane ^ (32 * n))));
                o[n] = mfma32(__builtin_bit_cast(f16x8, __builtin_shufflevector(v0, v1, 0, 1, 2, 3, 4, 5, 6, 7)), pf, o[n]);
            }
        }
    };

    // The next tile is on its way while this one is worked on.  Waves meet
    // once per tile: each has waited for its own loads, so the tile is whole,
    // and none reads the other buffer any more, so it can be filled.
    fetch(0, 0);
    auto run = [&](auto apart) {
        for (int j = 0; j < tiles; ++j) {
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            const bool cleaned = partial(j);
            if (cleaned) clean(j, j & 1);
            __syncthreads();
            if (j + 1 < tiles) fetch(j + 1, (j + 1) & 1);
            constexpr int U = BN / 32;
#pragma unroll 1
            for (int u = 0; u < U; ++u)
                if (KW == 1 || u % KW == kw) step(j, u, cleaned, apart);
        }
    };
    if (__builtin_expect(apart, 0))
        run(std::true_type{});
    else
        run(std::false_type{});
    sum = over_halves(sum, add_f32);
    if constexpr (KW > 1) {
        // The waves that share rows hand their sums to the first of them.
        constexpr int EACH = 32 * (D + 4);  // floats: 16 D / 32 per lane, maximum and sum
        static_assert(RW * (KW - 1) * EACH * 4 <= (int)sizeof lds, "room for their sums");
        float* const sums = reinterpret_cast<float*>(lds) + rw * (KW - 1) * EACH + lane;
        __syncthreads();
        if (kw > 0) {
            float* const mine = sums + (kw - 1) * EACH;
            mine[D * 32] = mx;
            mine[D * 32 + 64] = sum;
#pragma unroll
            for (int n = 0; n < D / 32; ++n)
#pragma unroll
                for (int i = 0; i < 16; ++i) mine[(16 * n + i) * 64] = o[n][i];
        }
        __syncthreads();
        if (kw > 0) return;
#pragma unroll 1
        for (int w = 0; w < KW - 1; ++w) {
            const float* const theirs = sums + w * EACH;
            const float m1 = theirs[D * 32], s1 = theirs[D * 32 + 64];
            const float m2 = fmaxf(mx, m1);
            const float f0 = mx == NEG_INF ? 0.f : __builtin_amdgcn_exp2f((mx - m2) * sc);
            const float f1 = m1 == NEG_INF ? 0.f : __builtin_amdgcn_exp2f((m1 - m2) * sc);
            mx = m2;
            sum = sum * f0 + s1 * f1;
#pragma unroll
            for (int n = 0; n < D / 32; ++n)
#pragma unroll
                for (int i = 0; i < 16; ++i) o[n][i] = o[n][i] * f0 + theirs[(16 * n + i) * 64] * f1;
        }
    }
    if (start < 0) return;
    const float inv = 1.f / sum;
    f16* out = static_cast<f16*>(a.out) + (int64_t)row * a.out_stride + head * D;
#pragma unroll
    for (int n = 0; n < D / 32; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f16x4v w;
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = (f16)(o[n][4 * i + k] * inv);
            *reinterpret_cast<f16x4v*>(out + 32 * n + 8 * i + 4 * h) = w;
        }
}

template <int D, int RW, int KW, int BN>
hipError_t launch(const PromptArgs& a, hipStream_t st) {
    constexpr int BM = RW * 32;
    const dim3 grid(a.kv_heads, a.q_heads / a.kv_heads, (unsigned)((a.tokens + BM - 1) / BM));
    attn_prompt_kernel<D, RW, KW, BN><<<grid, 64 * RW * KW, 0, st>>>(a);
    return hipGetLastError();
}

// Work-groups of 128 rows where there are enough for every compute unit, else
// of 64 with two waves for every 32 rows, which halves the longest chain of
// steps.  A long sequence is such a chain: up to two and a half work-groups of
// 128 rows per unit 64 rows are faster (1, 2 and 3 of them, one prompt of 1000,
// 2048 and 3000 tokens, 32 heads of 64: 17.3, 34.2 and 64.6 us with 64 rows, 23.1,
// 41.1 and 61.4 with 128; two of 1000, 32 heads of 128: 41.0 against 46.8).  Short
// packed ones have no chain, and reading each key for 64 rows only costs more
// than it saves from two per unit on with heads of 64 and one and a half with
// 128 (2 per unit, 16 of 128 tokens: 11.7 us with 64 rows and 9.9 with 128 at
// head size 64, 21.2 and 16.5 at 128; 33 of up to 100, 1.6 per unit: 12.4 and
// 12.8, 22.8 and 19.2; 1 per unit, 16 of 64: 7.1 and 7.5, 10.9 and 12.0).  The
// host knows the mean length alone: 4 of 512 are faster with 128 rows (19.4
// against 17.0, 28.2 against 25.6) and count as short, one of 1000 among eight
// of up to 125, 1.6 per unit, would be with 64 at head size 128 (32.1 against 39.7).
// Four waves for 32 rows gain 10 % at 512 and 1024 tokens and lose 20 % at 128.
//
// Tiles of 32 keys let three work-groups share a compute unit at head size 128
// (8192 tokens, 32 heads: 558 us against 594 with 64 keys and two); at 64
// four fit either way, and fewer meetings won (2 % there, 4 % on 9 packed prompts
// of up to 700 tokens).
template <int D>
hipError_t launch_rows(const PromptArgs& a, hipStream_t st) {
    const int64_t blocks = (a.tokens + 127) / 128 * a.q_heads;
    const bool lengthy = a.tokens >= 800 * a.n_seqs;
    const int halves = lengthy ? 5 : D == 64 ? 4 : 3;  // of a work-group per unit
    if (blocks * 2 < halves * (int64_t)a.cus && a.tokens <= 65535 * 64) return launch<D, 2, 2, 64>(a, st);
    return launch<D, 4, 1, D == 128 ? 32 : 64>(a, st);
}

}  // namespace

hipError_t launch_attn_prompt(const PromptArgs& a, hipStream_t st) {
    return a.head_dim == 64 ? launch_rows<64>(a, st) : launch_rows<128>(a, st);
}

}  // namespace qmm
