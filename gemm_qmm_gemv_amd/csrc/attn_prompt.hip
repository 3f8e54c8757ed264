// attn_prompt.hip -- causal attention over whole prompts packed behind each
// other, with grouped heads:
//
//   O[i] = sum_j exp(S[i][j] - max_j S[i][j]) V[j] / sum_j exp(S[i][j] - max_j S[i][j]),
//   S[i][j] = scale * Q[i] . K[j],  j from the start of i's sequence to i.
//
// Bound by the matrix cores.  A work-group holds 128 packed rows of one query
// head (32 per wave) and walks over the rows' keys in tiles of 64, with a
// running maximum and sum.  Rows are cut by their place in the packing and
// not by sequence: a tile of rows may hold the end of one sequence and several
// short ones, which costs masked work at the borders only and needs no list
// of tiles.
//
// The products are transposed so that no value changes lanes between them:
//   S^T = K Q^T puts, in lane l, scores of query row l % 32 at sixteen of 32
//   keys; O^T = V^T P^T takes them as its right operand as they are, with V^T
//   read in the same order of keys.  A query row's maximum and sum need one
//   exchange with lane l ^ 32.
#include <type_traits>

#include "layer_kernels.h"
#include "qmm_device.h"

namespace qmm {
namespace {

constexpr int BN = 64;   // keys per step
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

// Max over lanes l and l ^ 32: the swap exchanges one operand's upper lanes
// with the other's lower ones, so with the same value in both each result
// holds one half twice.
__device__ __forceinline__ float halves_max(float v) {
    const u32 x = __builtin_bit_cast(u32, v);
    const auto r = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    const u32 a = r[0], b = r[1];
    return fmaxf(__builtin_bit_cast(float, a), __builtin_bit_cast(float, b));
}

// Elements from one row of a tile to the next in LDS.  One access to K reads
// the same 16 bytes of 32 rows, one to V 32 bytes each of four rows: rows
// start 16 bytes (K) and 64 bytes (V) further into the 256 bytes of banks, so
// what an access touches at a time lies on different banks, and every address
// of a lane is one register plus a constant.
template <int D> constexpr int K_ROW = D + 8;
template <int D> constexpr int V_ROW = D + 32;

// RW waves hold 32 query rows each; with KW = 2 two waves share the rows, each
// taking one half of every tile's keys, and join at the end.
template <int D, int RW, int KW>
__global__ void __launch_bounds__(64 * RW * KW, 2) attn_prompt_kernel(PromptArgs a) {
    constexpr int BM = RW * 32, T = 64 * RW * KW;
    constexpr int CH = BN * D / 8 / T;     // 16-byte chunks of a tile of K (or of V) per thread
    constexpr int ROWS = T / (D / 8);      // rows that the work-group's chunks of one round cover
    constexpr int KBUF = BN * K_ROW<D>, VBUF = BN * V_ROW<D>;
    __shared__ __align__(16) f16 lds[2 * KBUF + 2 * VBUF];
    __shared__ int lds_bad[2][BN], lds_any[2];
    __shared__ int lds_lo[RW], lds_hi[RW], lds_late[RW];
    f16* const lds_k = lds;
    f16* const lds_v = lds + 2 * KBUF;
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int rw = wave % RW, kw = wave / RW;
    const int h = lane >> 5, l32 = lane & 31;
    // Query heads of one key head lie kv_heads work-groups apart: with eight
    // or a divisor of eight of them, one die (work-groups go round the eight)
    // reads few key heads.  Later rows see more keys: they start first.
    const int pos = blockIdx.x % a.q_heads;
    const int kvh = pos % a.kv_heads, head = kvh * (a.q_heads / a.kv_heads) + pos / a.kv_heads;
    const int tile = (int)gridDim.x / a.q_heads - 1 - blockIdx.x / a.q_heads;
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
    int lo = start < 0 ? 0x7fffffff : start, hi = start < 0 ? -1 : row, late = start < 0 ? 0 : start;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const int x = __shfl_xor(lo, o, 64), y = __shfl_xor(hi, o, 64), z = __shfl_xor(late, o, 64);
        lo = x < lo ? x : lo;
        hi = y > hi ? y : hi;
        late = z > late ? z : late;
    }
    const int wlo = uniform(lo), whi = uniform(hi), wlate = uniform(late);
    if (lane == 0) {
        lds_lo[rw] = wlo;
        lds_hi[rw] = whi;
        lds_late[rw] = wlate;
    }
    if (tid < 2 * BN) (&lds_bad[0][0])[tid] = 0;
    if (tid < 2) lds_any[tid] = 0;
    __syncthreads();
    int blo = 0x7fffffff, bhi = -1, blate = 0;
#pragma unroll
    for (int w = 0; w < RW; ++w) {
        blo = lds_lo[w] < blo ? lds_lo[w] : blo;
        bhi = lds_hi[w] > bhi ? lds_hi[w] : bhi;
        blate = lds_late[w] > blate ? lds_late[w] : blate;
    }
    blo = uniform(blo);
    bhi = uniform(bhi);
    blate = uniform(blate);
    if (bhi < 0) return;

    f32x16 o[D / 32];
    float mx = NEG_INF, sum = 0.f;
#pragma unroll
    for (int n = 0; n < D / 32; ++n) o[n] = f32x16{};
    const f16* kp = static_cast<const f16*>(a.k) + kvh * D;
    const f16* vp = static_cast<const f16*>(a.v) + kvh * D;
    const int tiles = (bhi - blo) / BN + 1;

    // The thread's chunks of a tile: rows sr, sr + ROWS, ...  Rows past the
    // last key read as zero: they lie behind the end of the buffer resource
    // (the offset is all in the vector operand, which the bound is checked
    // against).
    const int sr = tid / (D / 8), scol = tid % (D / 8) * 8;
    auto load_tile = [&](const f16* base, int64_t stride, int j, u32x4 (&w)[CH]) {
        const int t0 = blo + j * BN;
        const int left = bhi + 1 - t0 < BN ? bhi + 1 - t0 : BN;
        const rsrc_t rs = make_rsrc(base + (int64_t)t0 * stride, (uint32_t)(left * (int)stride * 2));
#pragma unroll
        for (int i = 0; i < CH; ++i)
            w[i] = __builtin_amdgcn_raw_buffer_load_b128(rs, ((sr + i * ROWS) * (int)stride + scol) * 2, 0, 0);
    };
    auto store_k = [&](int j, const u32x4 (&w)[CH]) {
        f16* p = lds_k + (j & 1) * KBUF + sr * K_ROW<D> + scol;
#pragma unroll
        for (int i = 0; i < CH; ++i) *reinterpret_cast<u32x4*>(p + i * ROWS * K_ROW<D>) = w[i];
    };
    auto store_v = [&](int j, u32x4 (&w)[CH]) {
        // In a tile that not every row sees, values that are not finite must
        // not meet a probability of zero (their product is NaN): they are
        // cleared, and the rows that do see their key get a NaN score.
        const int t0 = blo + j * BN, b = j & 1;
        if (t0 + BN - 1 > row0 || t0 < blate) {
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                bool odd = false;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    odd = odd || (w[i][k] & 0x7C00u) == 0x7C00u || (w[i][k] & 0x7C000000u) == 0x7C000000u;
                if (odd) {
                    w[i] = u32x4{0, 0, 0, 0};
                    lds_bad[b][sr + i * ROWS] = j + 1;  // of this tile: never cleared
                    lds_any[b] = j + 1;
                }
            }
        }
        f16* p = lds_v + b * VBUF + sr * V_ROW<D> + scol;
#pragma unroll
        for (int i = 0; i < CH; ++i) *reinterpret_cast<u32x4*>(p + i * ROWS * V_ROW<D>) = w[i];
    };

    // One step of 32 keys, t..t+31, in half u of the tile.
    const f16* const k_lane = lds_k + l32 * K_ROW<D> + 8 * h;
    const f16* const v_lane = lds_v + (4 * h + (lane >> 2 & 3)) * V_ROW<D> + 16 * (lane >> 4 & 1) + 4 * (lane & 3);
    auto step = [&](int j, int u) {
        const int t = blo + j * BN + 32 * u;
        if (t > whi || t + 31 < wlo) return;
        const int b = j & 1;
        const f16* kb = k_lane + b * KBUF + 32 * u * K_ROW<D>;
        f32x16 s = {};
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
            s = mfma32(*reinterpret_cast<const f16x8*>(kb + 16 * i), __builtin_bit_cast(f16x8, qw[i]), s);
        if (t + 31 > wrow0 || t < wlate) {  // not every row sees every key
            const bool bad = lds_any[b] == j + 1;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int key = t + 8 * (i / 4) + 4 * h + i % 4;
                if (bad && lds_bad[b][32 * u + key - t] == j + 1) s[i] = __builtin_nanf("");
                if (key > row || key < start || start < 0) s[i] = NEG_INF;
            }
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
        const float base = mx == NEG_INF ? 0.f : mx * sc;
        // Probabilities are cut to fp16, and their sum is of the cut values:
        // what the cutting takes away on average it takes from both sides of
        // the quotient.
        u32 w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float p0 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[2 * i], sc, -base));
            const float p1 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[2 * i + 1], sc, -base));
            w[i] = __builtin_bit_cast(u32, __builtin_amdgcn_cvt_pkrtz(p0, p1));
            sum = __builtin_amdgcn_fdot2(as_h2(w[i]), f16x2{(f16)1.f, (f16)1.f}, sum, false);
        }
        // V^T operand: lane (h, l32) wants value 32 n + l32 of keys
        // 16 e + 4 h + 0..3 and + 8..11.  The transposing read takes four
        // rows of 16 values per 16 lanes, 8 bytes from each lane, and gives
        // lane i the four rows' value i.
        const f16* vb = v_lane + b * VBUF + 32 * u * V_ROW<D>;
        typedef __attribute__((address_space(3))) s16x4* lds_ptr;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const f16x8 pf = __builtin_bit_cast(f16x8, u32x4{w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]});
#pragma unroll
            for (int n = 0; n < D / 32; ++n) {
                const s16x4 v0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(vb + 16 * e * V_ROW<D> + 32 * n));
                const s16x4 v1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(vb + (16 * e + 8) * V_ROW<D> + 32 * n));
                o[n] = mfma32(__builtin_bit_cast(f16x8, __builtin_shufflevector(v0, v1, 0, 1, 2, 3, 4, 5, 6, 7)), pf, o[n]);
            }
        }
    };
    // Keys and values of the next tile are on their way while this one is
    // worked on, and go to the other buffer: one barrier per tile.
    u32x4 kr[CH], vr[CH];
    load_tile(kp, a.k_stride, 0, kr);
    load_tile(vp, a.v_stride, 0, vr);
    store_k(0, kr);
    store_v(0, vr);
    if (tiles > 1) load_tile(kp, a.k_stride, 1, kr);
    for (int j = 0; j < tiles; ++j) {
        const bool more = j + 1 < tiles;
        __syncthreads();
        if (more) {
            store_k(j + 1, kr);
            load_tile(vp, a.v_stride, j + 1, vr);
        }
#pragma unroll 1
        for (int u = 0; u < 2; ++u) {
            if (KW == 1 || u == kw) step(j, u);
            if (u == 0 && more) {
                store_v(j + 1, vr);
                if (j + 2 < tiles) load_tile(kp, a.k_stride, j + 2, kr);
            }
        }
    }
    sum += __shfl_xor(sum, 32, 64);
    if constexpr (KW == 2) {
        // The second wave of each pair hands its sums over.
        static_assert(RW * 32 * (D + 4) * 4 <= (int)sizeof lds, "room for one wave's sums of each pair");
        float* const mine = reinterpret_cast<float*>(lds) + rw * 32 * (D + 4);
        __syncthreads();
        if (kw == 1) {
            mine[D * 32 + lane] = mx;
            mine[D * 32 + 64 + lane] = sum;
#pragma unroll
            for (int n = 0; n < D / 32; ++n)
#pragma unroll
                for (int i = 0; i < 16; ++i) mine[(16 * n + i) * 64 + lane] = o[n][i];
        }
        __syncthreads();
        if (kw == 1) return;
        const float m1 = mine[D * 32 + lane], s1 = mine[D * 32 + 64 + lane];
        const float m2 = fmaxf(mx, m1);
        const float f0 = mx == NEG_INF ? 0.f : __builtin_amdgcn_exp2f((mx - m2) * sc);
        const float f1 = m1 == NEG_INF ? 0.f : __builtin_amdgcn_exp2f((m1 - m2) * sc);
        sum = sum * f0 + s1 * f1;
#pragma unroll
        for (int n = 0; n < D / 32; ++n)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[n][i] = o[n][i] * f0 + mine[(16 * n + i) * 64 + lane] * f1;
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

template <int D, int RW, int KW>
hipError_t launch(const PromptArgs& a, hipStream_t st) {
    constexpr int BM = RW * 32;
    const dim3 grid((unsigned)((a.tokens + BM - 1) / BM * a.q_heads));
    attn_prompt_kernel<D, RW, KW><<<grid, 64 * RW * KW, 0, st>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_attn_prompt(const PromptArgs& a, hipStream_t st) {
#ifndef PW
#define PW 4
#define PR 1
#endif
    return a.head_dim == 64 ? launch<64, PW, PR>(a, st) : launch<128, PW, PR>(a, st);
}

}  // namespace qmm
