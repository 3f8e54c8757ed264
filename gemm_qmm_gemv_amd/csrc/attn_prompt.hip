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
#include "layer_kernels.h"
#include "qmm_device.h"

namespace qmm {
namespace {

constexpr int BM = 128;  // query rows per work-group
constexpr int BN = 64;   // keys per step
constexpr float NEG_INF = -__builtin_huge_valf();

typedef f16 f16x4v __attribute__((ext_vector_type(4)));

__device__ __forceinline__ f32x16 mfma32(f16x8 a, f16x8 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}

// First row of the sequence that packed row r belongs to, or -1 if it belongs
// to none.  Offsets are clamped so that whatever they hold stays in bounds.
__device__ __forceinline__ int sequence_start(const int32_t* offsets, int n_seqs, int64_t tokens, int r) {
    int lo = 0, hi = n_seqs + 1;  // offsets[lo - 1] <= r < offsets[hi]
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (offsets[mid] <= r)
            lo = mid + 1;
        else
            hi = mid;
    }
    if (lo == 0 || lo > n_seqs || r >= tokens) return -1;
    const int s = offsets[lo - 1];
    return s < 0 ? 0 : s;
}

template <int D>
__global__ void __launch_bounds__(256) attn_prompt_kernel(PromptArgs a) {
    constexpr int PAD = D + 8;
    __shared__ f16 lds_k[BN][PAD], lds_v[BN][PAD];
    __shared__ int lds_bad[BN];
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int h = lane >> 5, l32 = lane & 31;
    const int head = blockIdx.x % a.q_heads;
    // Later rows see more keys: the longest work starts first.
    const int tile = (int)gridDim.x / a.q_heads - 1 - blockIdx.x / a.q_heads;
    const int kvh = head / (a.q_heads / a.kv_heads);
    const int row0 = tile * BM, wrow0 = row0 + wave * 32;
    const int row = wrow0 + l32;

    const int start = sequence_start(a.offsets, (int)a.n_seqs, a.tokens, row);
    const int first = start < 0 ? 0x7fffffff : start;  // keys first..row
    // The work-group's keys: from the earliest start to the last row.
    __shared__ int lds_lo[4], lds_hi[4];
    int lo = first, hi = start < 0 ? -1 : row;
    for (int o = 16; o > 0; o >>= 1) {
        const int x = __shfl_xor(lo, o, 64), y = __shfl_xor(hi, o, 64);
        lo = x < lo ? x : lo;
        hi = y > hi ? y : hi;
    }
    const int wlo = uniform(lo), whi = uniform(hi);
    if (lane == 0) {
        lds_lo[wave] = wlo;
        lds_hi[wave] = whi;
    }
    __syncthreads();
    int blo = 0x7fffffff, bhi = -1;
    for (int w = 0; w < 4; ++w) {
        blo = lds_lo[w] < blo ? lds_lo[w] : blo;
        bhi = lds_hi[w] > bhi ? lds_hi[w] : bhi;
    }
    if (bhi < 0) return;

    f16x8 qf[D / 16];
    const f16* qp = static_cast<const f16*>(a.q) + (int64_t)(start < 0 ? 0 : row) * a.q_stride + head * D;
#pragma unroll
    for (int j = 0; j < D / 16; ++j) qf[j] = *reinterpret_cast<const f16x8*>(qp + 16 * j + 8 * h);
    const float sc = a.scale * 1.44269504088896341f;

    f32x16 o[D / 32] = {};
    float mx = NEG_INF, sum = 0.f;
    const f16* kp = static_cast<const f16*>(a.k) + kvh * D;
    const f16* vp = static_cast<const f16*>(a.v) + kvh * D;

    for (int t0 = blo; t0 <= bhi; t0 += BN) {
        __syncthreads();
        if (tid < BN) lds_bad[tid] = 0;
        __syncthreads();
        for (int i = tid; i < BN * (D / 8); i += 256) {
            const int r = i / (D / 8), d = i % (D / 8) * 8;
            u32x4 kv = {0, 0, 0, 0}, vv = {0, 0, 0, 0};
            if (t0 + r <= bhi) {
                kv = *reinterpret_cast<const u32x4*>(kp + (int64_t)(t0 + r) * a.k_stride + d);
                vv = *reinterpret_cast<const u32x4*>(vp + (int64_t)(t0 + r) * a.v_stride + d);
            }
            bool odd = false;
            for (int w = 0; w < 4; ++w) odd = odd || (vv[w] & 0x7C00u) == 0x7C00u || (vv[w] & 0x7C000000u) == 0x7C000000u;
            if (odd) lds_bad[r] = 1;
            *reinterpret_cast<u32x4*>(&lds_k[r][d]) = kv;
            *reinterpret_cast<u32x4*>(&lds_v[r][d]) = vv;
        }
        __syncthreads();
        // A key whose values are not finite must not reach rows that do not
        // see it (a NaN times a probability of zero is NaN): its values are
        // cleared and the rows that do see it get a NaN score.
        for (int i = tid; i < BN * (D / 8); i += 256) {
            const int r = i / (D / 8), d = i % (D / 8) * 8;
            if (lds_bad[r]) *reinterpret_cast<u32x4*>(&lds_v[r][d]) = u32x4{0, 0, 0, 0};
        }
        __syncthreads();
        for (int u = 0; u < 2; ++u) {
            const int t = t0 + 32 * u;
            if (t > whi || t + 31 < wlo) continue;
            f32x16 s = {};
#pragma unroll
            for (int j = 0; j < D / 16; ++j)
                s = mfma32(*reinterpret_cast<const f16x8*>(&lds_k[32 * u + l32][16 * j + 8 * h]), qf[j], s);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int key = t + 8 * (i / 4) + 4 * h + i % 4;
                s[i] *= sc;
                if (lds_bad[key - t0]) s[i] = __builtin_nanf("");
                if (key > row || key < first) s[i] = NEG_INF;
            }
            float top = s[0];
#pragma unroll
            for (int i = 1; i < 16; ++i) top = fmaxf(top, s[i]);
            top = fmaxf(top, __shfl_xor(top, 32, 64));
            const float m2 = fmaxf(mx, top);
            const float f = mx == NEG_INF ? 0.f : __builtin_amdgcn_exp2f(mx - m2);
            mx = m2;
            const float base = mx == NEG_INF ? 0.f : mx;
            sum *= f;
#pragma unroll
            for (int n = 0; n < D / 32; ++n) o[n] = o[n] * f;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                s[i] = __builtin_amdgcn_exp2f(s[i] - base);
                sum += s[i];
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                f16x8 pf;
#pragma unroll
                for (int j = 0; j < 8; ++j) pf[j] = (f16)s[8 * e + j];
#pragma unroll
                for (int n = 0; n < D / 32; ++n) {
                    f16x8 vf;
#pragma unroll
                    for (int j = 0; j < 8; ++j) vf[j] = lds_v[32 * u + 16 * e + 4 * h + (j & 3) + 8 * (j >> 2)][32 * n + l32];
                    o[n] = mfma32(vf, pf, o[n]);
                }
            }
        }
    }
    if (start < 0) return;
    sum += __shfl_xor(sum, 32, 64);
    const float inv = 1.f / sum;
    f16* out = static_cast<f16*>(a.out) + (int64_t)row * a.out_stride + head * D;
#pragma unroll
    for (int n = 0; n < D / 32; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f16x4v w;
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = (f16)(o[n][4 * i + j] * inv);
            *reinterpret_cast<f16x4v*>(out + 32 * n + 8 * i + 4 * h) = w;
        }
}

}  // namespace

hipError_t launch_attn_prompt(const PromptArgs& a, hipStream_t st) {
    const dim3 grid((unsigned)((a.tokens + BM - 1) / BM * a.q_heads));
    if (a.head_dim == 64)
        attn_prompt_kernel<64><<<grid, 256, 0, st>>>(a);
    else
        attn_prompt_kernel<128><<<grid, 256, 0, st>>>(a);
    return hipGetLastError();
}

}  // namespace qmm
