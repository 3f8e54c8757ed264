// kv_append.hip -- what happens to the q, k and v rows of new tokens between
// their projections and attention: optional per-head norm of q and k, the
// rotation of q and k by position, q to fp16, k and v into a paged cache in
// 4- or 8-bit affine groups or in fp16.
//
//   rotation of pair i by angle t = position * inv_freq[i]:
//     (a, b) -> (a cos t - b sin t, b cos t + a sin t),
//     a, b = elements i and i + rot/2 (or 2i and 2i + 1, interleaved)
//   group of `group` neighbours of a row, b bits:
//     m = fp16(min), s = fp16((max - min) / (2^b - 1)),
//     code = round((x - m) / s) clamped to [0, 2^b - 1]  (0 where s = 0)
//
// Bound by memory.  A lane holds 8 neighbours of a row, so D/8 lanes make a
// row and sums, minima and maxima over a row or group are butterflies within
// those lanes.  The angle is formed in 64 bits: at position 131071 a 32-bit
// product is off by up to 0.004 rad.  Sines and cosines depend on the token
// alone, so a work-group forms them once per token in LDS and uses them for
// all its heads.
#include "layer_kernels.h"
#include "qmm_device.h"

namespace qmm {
namespace {

constexpr int THREADS = 256;

template <int N, class F>
__device__ __forceinline__ float butterfly(float v, F f) {
#pragma unroll
    for (int o = 1; o < N; o <<= 1) v = f(v, __shfl_xor(v, o, 64));
    return v;
}

// min and max that keep a NaN.
__device__ __forceinline__ float min_nan(float a, float b) { return (a < b || a != a) ? a : b; }
__device__ __forceinline__ float max_nan(float a, float b) { return (a > b || a != a) ? a : b; }

__device__ __forceinline__ u32 pack2(float a, float b) { return as_u32(f16x2{(f16)a, (f16)b}); }

__device__ __forceinline__ void store_half8(void* p, const float (&x)[8]) {
    *static_cast<u32x4*>(p) = u32x4{pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7])};
}

template <int D, int BITS, bool IN16>
__global__ void __launch_bounds__(THREADS) append_kernel(AppendArgs a, int tile, int heads_per_block) {
    constexpr int L = D / 8;  // lanes per row
    extern __shared__ float2 trig[];  // [tile][rot/2]
    const int64_t t0 = (int64_t)blockIdx.x * tile;
    const int nt = (int)(a.tokens - t0 < tile ? a.tokens - t0 : tile);
    const int half = a.rot / 2;
    for (int i = threadIdx.x; i < nt * half; i += THREADS) {
        // Turns in 64 bits, the whole ones dropped there; what is left is in
        // [-1/2, 1/2] and fits fp32.
        const double turns = (double)a.positions[t0 + i / half] * (double)a.inv_freq[i % half] * 0.15915494309189533577;
        float s, c;
        sincospif(2.f * (float)(turns - rint(turns)), &s, &c);
        trig[i] = float2{c, s};
    }
    __syncthreads();

    const int heads = a.q_heads + 2 * a.c.kv_heads;
    const int h0 = blockIdx.y * heads_per_block;
    const int nh = heads - h0 < heads_per_block ? heads - h0 : heads_per_block;
    const int sub = threadIdx.x % L;
    // Neighbouring rows of a work-group are neighbouring tokens of one head:
    // their scales and mins then fall into one run of memory.
    for (int r = threadIdx.x / L; r < nt * nh; r += THREADS / L) {
        const int tt = r % nt, head = h0 + r / nt;
        const int64_t t = t0 + tt;
        const int kind = head < a.q_heads ? 0 : head < a.q_heads + a.c.kv_heads ? 1 : 2;
        const int hh = kind == 0 ? head : kind == 1 ? head - a.q_heads : head - a.q_heads - a.c.kv_heads;
        const void* src = kind == 0 ? a.q : kind == 1 ? a.k : a.v;
        const int64_t stride = kind == 0 ? a.q_stride : kind == 1 ? a.k_stride : a.v_stride;
        float x[8];
        const int64_t off = t * stride + hh * D + sub * 8;
        if constexpr (IN16) {
            const u32x4 w = *reinterpret_cast<const u32x4*>(static_cast<const f16*>(src) + off);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const f16x2 p = as_h2(w[i]);
                x[2 * i] = (float)p[0];
                x[2 * i + 1] = (float)p[1];
            }
        } else {
            const f32x4* p = reinterpret_cast<const f32x4*>(static_cast<const float*>(src) + off);
            const f32x4 u = p[0], v = p[1];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[i] = u[i];
                x[4 + i] = v[i];
            }
        }
        if (kind != 2) {
            const float* nw = kind == 0 ? a.q_norm : a.k_norm;
            if (nw) {
                float s = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) s += x[i] * x[i];
                s = butterfly<L>(s, [](float p, float q) { return p + q; });
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
#pragma unroll
                for (int i = 0; i < 8; ++i) p[i] = __shfl(x[i], other, L);
                if (sub < 2 * lanes) {
                    const float sign = sub < lanes ? -1.f : 1.f;
                    const int at = (sub < lanes ? sub : sub - lanes) * 8;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float2 cs = tr[at + i];
                        x[i] = x[i] * cs.x + sign * (p[i] * cs.y);
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
            for (int o = 1; o < span; o <<= 1) {
                lo = min_nan(lo, __shfl_xor(lo, o, 64));
                hi = max_nan(hi, __shfl_xor(hi, o, 64));
            }
            constexpr float TOP = (float)((1 << BITS) - 1);
            const f16 m16 = (f16)lo, s16 = (f16)((hi - lo) / TOP);
            const float m = (float)m16, s = (float)s16;
            u32 w[BITS / 4];
#pragma unroll
            for (int i = 0; i < BITS / 4; ++i) w[i] = 0;
            float held[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float c = s > 0.f ? fminf(fmaxf(rintf((x[i] - m) / s), 0.f), TOP) : 0.f;
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
    // Up to 16 tokens share their sines and cosines; with few tokens one per
    // work-group, and the heads are cut so that the device is filled.
    const int64_t want = 2 * (int64_t)a.cus;
    int tile = 16;
    while (tile > 1 && (a.tokens + tile - 1) / tile < want) tile >>= 1;
    const int64_t tiles = (a.tokens + tile - 1) / tile;
    const int rows_per_pass = THREADS / (D / 8);
    int cuts = (int)((want + tiles - 1) / tiles);
    int per = (heads + cuts - 1) / cuts;
    const int least = (rows_per_pass + tile - 1) / tile;  // at least one full pass of rows
    if (per < least) per = least;
    if (per > heads) per = heads;
    const dim3 grid((unsigned)tiles, (unsigned)((heads + per - 1) / per));
    const size_t lds = (size_t)tile * (a.rot / 2) * sizeof(float2);
    if (a.in_fp16)
        append_kernel<D, BITS, true><<<grid, THREADS, lds, st>>>(a, tile, per);
    else
        append_kernel<D, BITS, false><<<grid, THREADS, lds, st>>>(a, tile, per);
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
