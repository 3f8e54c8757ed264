// kv_append.hip -- what happens to the q, k and v rows of new tokens between
// their projections and attention: optional per-head norm of q and k, the
// rotation of q and k by position, q to fp16, k and v into a paged cache in
// 4- or 8-bit affine groups or in fp16.
//
//   rotation of pair i by angle t = position * inv_freq[i]:
//     (a, b) -> (a cos t - b sin t, b cos t + a sin t),
//     a, b = elements i and i + rot/2 (or 2i and 2i + 1, interleaved)
//   group of `group` neighbours of a row, b bits:
//     m = fp16(min), s = fp16((max - min) / (2^b - 1))  (NaN where m is infinite),
//     code = round((x - m) / s) clamped to [0, 2^b - 1]  (0 where s = 0 or not finite)
//
// Bound by memory into fp16 (8192 tokens of 40 heads of 128: 56.6 us, 4.7 TB/s), by
// the vector units into codes (4096 tokens of 48 heads of 64: 15 to 16 us into 4
// bits and into 8, 3.5 TB/s, units 87 and 85 % busy).  A lane holds 8 neighbours of a row, so D/8 lanes make a
// row and sums, minima and maxima over a row or group are butterflies within
// those lanes.  The angle is formed in 64 bits: at position 131071 a 32-bit
// product is off by up to 0.004 rad.  Sines and cosines depend on the token
// alone, so a work-group forms them once per token in LDS and uses them for
// all its heads.
#include "layer_device.h"
#include "layer_kernels.h"

namespace qmm {
namespace {

constexpr int THREADS = 256;

// v of lane l ^ 4: row_ror:12 brings it to the lower four of eight lanes,
// row_ror:4 to the upper four (banks 1 and 3 of a row of 16).
__device__ __forceinline__ float lane_xor4(float v) {
    const int x = __builtin_bit_cast(int, v);
    const int up = __builtin_amdgcn_mov_dpp(x, 0x12C, 0xF, 0xF, true);
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(up, x, 0x124, 0xF, 0xA, false));
}

// Sine and cosine of an angle, both rounded once: whole quarter turns are dropped
// in 64 bits, and within an eighth of a turn the Taylor series to x^11 and
// x^12 are off by less than 10^-11.  (As fp32 functions of an angle rounded to
// fp32 they were off by up to two steps, which showed as minima of groups
// that fell on the other side of a border of fp16.)
__device__ __forceinline__ void sin_cos(double angle, float& s, float& c) {
    const double quarters = rint(angle * 0.63661977236758134308);
    const double x = __builtin_fma(quarters, -1.57079632679489661923, angle) - quarters * 6.123233995736766e-17;
    const double y = x * x;
    double p = -1.0 / 39916800, q = 1.0 / 479001600;
    p = __builtin_fma(p, y, 1.0 / 362880);
    p = __builtin_fma(p, y, -1.0 / 5040);
    p = __builtin_fma(p, y, 1.0 / 120);
    p = __builtin_fma(p, y, -1.0 / 6);
    p = __builtin_fma(p * y, x, x);
    q = __builtin_fma(q, y, -1.0 / 3628800);
    q = __builtin_fma(q, y, 1.0 / 40320);
    q = __builtin_fma(q, y, -1.0 / 720);
    q = __builtin_fma(q, y, 1.0 / 24);
    q = __builtin_fma(q, y, -0.5);
    q = __builtin_fma(q, y, 1.0);
    const int turn = (int)(quarters - 4 * floor(quarters * 0.25));  // 0 to 3
    const float sine = (float)p, cosine = (float)q;
    s = turn & 1 ? cosine : sine;
    c = turn & 1 ? sine : cosine;
    if (turn & 2) s = -s;
    if (turn == 1 || turn == 2) c = -c;
}

// min and max that keep a NaN.
__device__ __forceinline__ float min_nan(float a, float b) { return __builtin_elementwise_minimum(a, b); }
__device__ __forceinline__ float max_nan(float a, float b) { return __builtin_elementwise_maximum(a, b); }

__device__ __forceinline__ u32 pack2(float a, float b) { return as_u32(f16x2{(f16)a, (f16)b}); }

__device__ __forceinline__ void store_half8(void* p, const float (&x)[8]) {
    *static_cast<u32x4*>(p) = u32x4{pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7])};
}

// The eight values of a lane as they are in memory.
template <bool IN16>
struct Raw8;
template <>
struct Raw8<true> {
    u32x4 w;
};
template <>
struct Raw8<false> {
    f32x4 lo, hi;
};

// `tile` tokens (1 << tile_log2) and `heads_per_block` of the q, k and v heads
// per work-group.  A row's values are asked for one round ahead: the first
// round's while the sines and cosines are formed.
template <int D, int BITS, bool IN16>
__global__ void __launch_bounds__(THREADS) append_kernel(AppendArgs a, int tile_log2, int heads_per_block) {
    constexpr int L = D / 8;  // lanes per row
    extern __shared__ __align__(16) float2 trig[];  // [tile][rot/2]
    const int tile = 1 << tile_log2;
    const int64_t t0 = (int64_t)blockIdx.x * tile;
    const int nt = (int)(a.tokens - t0 < tile ? a.tokens - t0 : tile);
    const int half = a.rot / 2;
    const int heads = a.q_heads + 2 * a.c.kv_heads;
    const int h0 = blockIdx.y * heads_per_block;
    const int nh = heads - h0 < heads_per_block ? heads - h0 : heads_per_block;
    const int sub = threadIdx.x % L;
    // Row r of the work-group is token r % tile of head r / tile:
    // neighbouring rows are neighbouring tokens of one head, whose scales and
    // mins fall into one run of memory.
    auto fetch = [&](int r) {
        Raw8<IN16> x = {};
        const int tt = r & (tile - 1), head = h0 + (r >> tile_log2);
        if (tt >= nt || r >= tile * nh) return x;
        const int kind = head < a.q_heads ? 0 : head < a.q_heads + a.c.kv_heads ? 1 : 2;
        const int hh = kind == 0 ? head : kind == 1 ? head - a.q_heads : head - a.q_heads - a.c.kv_heads;
        const void* src = kind == 0 ? a.q : kind == 1 ? a.k : a.v;
        const int64_t stride = kind == 0 ? a.q_stride : kind == 1 ? a.k_stride : a.v_stride;
        const int64_t off = (t0 + tt) * stride + hh * D + sub * 8;
        if constexpr (IN16) {
            x.w = *reinterpret_cast<const u32x4*>(static_cast<const f16*>(src) + off);
        } else {
            const f32x4* p = reinterpret_cast<const f32x4*>(static_cast<const float*>(src) + off);
            x.lo = p[0];
            x.hi = p[1];
        }
        return x;
    };
    constexpr int ROWS = THREADS / L;
    Raw8<IN16> ahead = fetch(threadIdx.x / L);
    for (int i = threadIdx.x; i < nt * half; i += THREADS) {
        float s, c;
        sin_cos((double)a.positions[t0 + i / half] * (double)a.inv_freq[i % half], s, c);
        trig[i] = float2{c, s};
    }
    __syncthreads();

    for (int r = threadIdx.x / L; r < tile * nh; r += ROWS) {
        const Raw8<IN16> raw = ahead;
        ahead = fetch(r + ROWS);
        const int tt = r & (tile - 1), head = h0 + (r >> tile_log2);
        if (tt >= nt) continue;
        const int64_t t = t0 + tt;
        const int kind = head < a.q_heads ? 0 : head < a.q_heads + a.c.kv_heads ? 1 : 2;
        const int hh = kind == 0 ? head : kind == 1 ? head - a.q_heads : head - a.q_heads - a.c.kv_heads;
        float x[8];
        if constexpr (IN16) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const f16x2 p = as_h2(raw.w[i]);
                x[2 * i] = (float)p[0];
                x[2 * i + 1] = (float)p[1];
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[i] = raw.lo[i];
                x[4 + i] = raw.hi[i];
            }
        }
        if (kind != 2) {
            const float* nw = kind == 0 ? a.q_norm : a.k_norm;
            if (nw) {
                float s = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) s += x[i] * x[i];
                s = over_lanes<L>(s, add_f32);
                const float rs = 1.f / sqrtf(s / (float)D + a.eps);
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = x[i] * rs * nw[sub * 8 + i];
            }
            const float2* tr = trig + tt * half;
            if (a.interleaved) {
                if (sub * 8 < a.rot) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 cs = tr[sub * 4 + i];
                        const float lo = x[2 * i], hi = x[2 * i + 1];
                        x[2 * i] = lo * cs.x - hi * cs.y;
                        x[2 * i + 1] = hi * cs.x + lo * cs.y;
                    }
                }
            } else if (half > 0) {
                // rot is a multiple of 16, so a lane's eight partners are
                // the eight of one other lane of the row.
                const int lanes = half / 8;
                const int other = sub < lanes ? sub + lanes : sub < 2 * lanes ? sub - lanes : sub;
                float p[8];
                if (lanes == 8) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) p[i] = dpp_move<0x128>(x[i]);  // row_ror:8
                } else if (lanes == 4) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) p[i] = lane_xor4(x[i]);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) p[i] = __shfl(x[i], other, L);
                }
                if (sub < 2 * lanes) {
                    const float sign = sub < lanes ? -1.f : 1.f;
                    const f32x4* cs = reinterpret_cast<const f32x4*>(tr + (sub < lanes ? sub : sub - lanes) * 8);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const f32x4 t2 = cs[i];  // two cosines with their sines
                        x[2 * i] = x[2 * i] * t2[0] + sign * (p[2 * i] * t2[1]);
                        x[2 * i + 1] = x[2 * i + 1] * t2[2] + sign * (p[2 * i + 1] * t2[3]);
                    }
                }
            }
        }
        if (kind == 0) {
            if (a.q_out) store_half8(static_cast<f16*>(a.q_out) + (t * a.q_heads + hh) * D + sub * 8, x);
            continue;
        }
        void* out = kind == 1 ? a.k_out : a.v_out;
        if (out) out = static_cast<f16*>(out) + (t * a.c.kv_heads + hh) * D + sub * 8;
        const int64_t slot = a.slots ? a.slots[t] : -1;
        const int64_t page = slot >> a.c.page_shift;
        const bool keep = slot >= 0 && page < a.c.pages;
        const int64_t unit = page * a.c.kv_heads + hh;  // (page, head)
        const int in_page = (int)(slot & ((1 << a.c.page_shift) - 1));
        char* rows = static_cast<char*>(kind == 1 ? a.c.k : a.c.v);
        if constexpr (BITS == 16) {
            if (keep) store_half8(reinterpret_cast<f16*>(rows) + ((unit << a.c.page_shift) + in_page) * D + sub * 8, x);
            if (out) store_half8(out, x);
        } else {
            if (out && !a.out_cached) store_half8(out, x);
            float lo = x[0], hi = x[0];
#pragma unroll
            for (int i = 1; i < 8; ++i) {
                lo = min_nan(lo, x[i]);
                hi = max_nan(hi, x[i]);
            }
            const int span = a.c.group / 8;  // lanes per group
            if (span == 4) {
                lo = over_lanes<4>(lo, min_nan);
                hi = over_lanes<4>(hi, max_nan);
            } else if (span == 8) {
                lo = over_lanes<8>(lo, min_nan);
                hi = over_lanes<8>(hi, max_nan);
            } else {
                lo = over_lanes<16>(lo, min_nan);
                hi = over_lanes<16>(hi, max_nan);
            }
            constexpr float TOP = (float)((1 << BITS) - 1);
            const f16 m16 = (f16)lo;
            const float m = (float)m16;
            // With a min that has become an infinity the group stands for
            // nothing: its scale is NaN, so that attention spoils what sees
            // it instead of leaving out a key of score -inf.
            const f16 s16 = (f16)(__builtin_isinf(m) ? __builtin_nanf("") : (hi - lo) / TOP);
            const float s = (float)s16;
            u32 w[BITS / 4];
#pragma unroll
            for (int i = 0; i < BITS / 4; ++i) w[i] = 0;
            float held[8];
            // One division for the group; each quotient is put right by what
            // it leaves of the dividend, as nearly as a division would (8 % of a
            // call of 4096 tokens of 48 heads of 64; without putting right 1 %
            // more, but more codes next to a border would go the other way).
            const float inv = s > 0.f ? 1.f / s : 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float d = x[i] - m, z = d * inv;
                const float c = fminf(fmaxf(rintf(__builtin_fmaf(__builtin_fmaf(-z, s, d), inv, z)), 0.f), TOP);
                held[i] = c * s + m;
                w[i * BITS / 32] |= (u32)c << (i * BITS % 32);
            }
            if (keep) {
                u32* p = reinterpret_cast<u32*>(rows) + ((unit << a.c.page_shift) + in_page) * (D * BITS / 32) + sub * (BITS / 4);
                if constexpr (BITS == 4)
                    *p = w[0];
                else
                    *reinterpret_cast<u32x2*>(p) = u32x2{w[0], w[1]};
                if (sub % span == 0) {
                    const int64_t at = ((unit * (D / a.c.group) + sub / span) << a.c.page_shift) + in_page;
                    static_cast<f16*>(kind == 1 ? a.c.ks : a.c.vs)[at] = s16;
                    static_cast<f16*>(kind == 1 ? a.c.km : a.c.vm)[at] = m16;
                }
            }
            if (out && a.out_cached) store_half8(out, held);
        }
    }
}

template <int D, int BITS>
hipError_t launch(const AppendArgs& a, hipStream_t st) {
    const int heads = a.q_heads + 2 * a.c.kv_heads;
    // Up to 16 tokens share their sines and cosines; with fewer tokens one
    // per work-group, and the heads are cut so that the device is filled: 16
    // work-groups for each unit.  With 2, 4, 8, 16 and 32 of them 8192 tokens of
    // 32 + 2 x 4 heads of 128 into an fp16 cache take 94, 62, 67, 56 and 53 us, 8192
    // of 16 + 2 x 8 heads of 128 into 4 bits 76, 52, 51, 46 and 48, 4096 of 32 + 2 x 8
    // heads of 64 into 4 bits 19.2, 14.4, 14.5, 15.1 and 17.3.
    const int64_t want = 16 * (int64_t)a.cus;
    int tile_log2 = 4;
    while (tile_log2 > 0 && (a.tokens + (1 << tile_log2) - 1) >> tile_log2 < want) --tile_log2;
    const int tile = 1 << tile_log2;
    const int64_t tiles = (a.tokens + tile - 1) >> tile_log2;
    const int rows_per_pass = THREADS / (D / 8);
    const int cuts = (int)((want + tiles - 1) / tiles);
    int per = (heads + cuts - 1) / cuts;
    const int least = (rows_per_pass + tile - 1) / tile;  // at least one full pass of rows
    if (per < least) per = least;
    if (per > heads) per = heads;
    const dim3 grid((unsigned)tiles, (unsigned)((heads + per - 1) / per));
    const size_t lds = (size_t)tile * (a.rot / 2) * sizeof(float2);
    if (a.in_fp16)
        append_kernel<D, BITS, true><<<grid, THREADS, lds, st>>>(a, tile_log2, per);
    else
        append_kernel<D, BITS, false><<<grid, THREADS, lds, st>>>(a, tile_log2, per);
    return hipGetLastError();
}

template <int D>
hipError_t launch_bits(const AppendArgs& a, hipStream_t st) {
    switch (a.c.bits) {
        case 4: return launch<D, 4>(a, st);
        case 8: return launch<D, 8>(a, st);
        default: return launch<D, 16>(a, st);
    }
}

}  // namespace

hipError_t launch_append(const AppendArgs& a, hipStream_t st) {
    return a.c.head_dim == 64 ? launch_bits<64>(a, st) : launch_bits<128>(a, st);
}

}  // namespace qmm
