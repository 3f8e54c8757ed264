// quantize.hip -- rows of activations to 8-bit codes with a scale for each row:
//   scale = fp32(max |x| / 127),  code = round(x / scale), ties to even.
//
// Bound by memory, and nearly as much by the vector units (32768 rows of 768 in
// fp16, 76 MB: 17.7 us = 4.3 TB/s, vector units 94 % busy; 8192 of 2048, 50 MB:
// 11.6 to 14.9, 78 %; of 8192: 42 us = 4.8): what a value costs there is kept to a
// handful of instructions.  The whole number next to x / scale
// comes out of one fused step with 1.5 * 2^23 (its low bits are the code, two's
// complement), and what it leaves over, x - code * scale, is exact in another: the
// code is the right one if that is less than half a scale.  Where it is not
// (the inverse is rounded, so next to a border it may not be), and on it, the
// codes are worked out again with the border looked at.
#include "layer_device.h"
#include "moe_kernels.h"

namespace qmm {
namespace {

typedef f16 f16x4v __attribute__((ext_vector_type(4)));

__device__ __forceinline__ int code_of(float x, float scale, float inv) {
    float q = rintf(x * inv);
    const float left = fmaf(-q, scale, x), half = 0.5f * scale;
    // The product with the rounded inverse is off by less than one.
    const bool odd = ((int)q & 1) != 0;
    if (left > half || (left == half && odd)) q += 1.f;
    if (left < -half || (left == -half && odd)) q -= 1.f;
    return (int)fminf(fmaxf(q, -127.f), 127.f);
}

// A row's scale from its largest magnitude, and what its codes are made with.
struct Unit {
    float scale, up, s, inv;
};
__device__ __forceinline__ Unit unit_of(float top) {
    Unit u;
    const bool finite = top < __builtin_huge_valf();
    u.scale = finite ? top / 127.f : __builtin_nanf("");
    // 1 / scale may leave fp32 for the smallest scales: such rows are scaled up
    // first, which is exact.
    u.up = u.scale < 0x1p-100f ? 0x1p100f : 1.f;
    u.s = u.scale * u.up;
    u.inv = finite && u.s > 0.f ? 1.f / u.s : 0.f;
    return u;
}
// Largest magnitude so far, as its bits: a NaN's are above an infinity's, that are
// above all others.
__device__ __forceinline__ void larger(u32& top, float v) {
    const u32 b = __builtin_bit_cast(u32, v) & 0x7fffffffu;
    top = b > top ? b : top;
}
__device__ __forceinline__ float max_f32(float a, float b) { return fmaxf(a, b); }
// Over a wave; infinite if any value is not finite.
__device__ __forceinline__ float top_of(u32 top) {
    if (top > 0x7f800000u) top = 0x7f800000u;
    return over_lanes<64>(__builtin_bit_cast(float, top), max_f32);
}

__device__ __forceinline__ u32 four_codes_checked(float a, float b, float c, float d, float up, float s, float inv) {
    const float v[4] = {a, b, c, d};
    u32 w = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int q = inv > 0.f ? code_of(v[j] * up, s, inv) : 0;
        w |= ((u32)q & 255u) << (8 * j);
    }
    return w;
}
__device__ __forceinline__ u32 four_codes(const float* v, const Unit& u) {
    u32 r[4];
    float off = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float m = fmaf(v[j], u.inv, 12582912.f);  // rounds to a whole number
        r[j] = __builtin_bit_cast(u32, m);
        off = fmaxf(off, fabsf(fmaf(12582912.f - m, u.s, v[j])));
    }
    // (Rows of zeros, of tiny and of values that are not finite come here, too.)
    if (__any(!(off < 0.5f * u.s) || u.up != 1.f))
        return four_codes_checked(v[0], v[1], v[2], v[3], u.up, u.s, u.inv);
    const u32 lo = __builtin_amdgcn_perm(r[1], r[0], 0x0c0c0400u), hi = __builtin_amdgcn_perm(r[3], r[2], 0x04000c0cu);
    return lo | hi;
}

// A work-group for each row, which it holds in registers, PER runs of four values
// a thread (VEC: one load each).
template <int T, int PER, bool VEC>
__global__ void __launch_bounds__(T) quantize_kernel(QuantizeArgs a) {
    __shared__ float lds[T / 64];
    const int64_t row = blockIdx.x;
    const int tid = threadIdx.x;
    float v[PER][4];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[i][j] = 0.f;
        const int e = (i * T + tid) * 4;
        if (e >= a.k) continue;
        if (a.f16) {
            const f16* p = static_cast<const f16*>(a.x) + row * a.stride + e;
            if constexpr (VEC) {
                const f16x4v w = *reinterpret_cast<const f16x4v*>(p);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[i][j] = (float)w[j];
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) v[i][j] = (float)p[j];
            }
        } else {
            const float* p = static_cast<const float*>(a.x) + row * a.stride + e;
            if constexpr (VEC) {
                const f32x4 w = *reinterpret_cast<const f32x4*>(p);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[i][j] = w[j];
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) v[i][j] = p[j];
            }
        }
    }
    // A value that is not finite makes the row's scale NaN.
    u32 bits = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) larger(bits, v[i][j]);
    float top = top_of(bits);
    if constexpr (T > 64) {
        if ((tid & 63) == 0) lds[tid >> 6] = top;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < T / 64; ++i) top = fmaxf(top, lds[i]);
    }
    const Unit u = unit_of(top);
    int8_t* const out = a.codes + row * (int64_t)a.k;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = (i * T + tid) * 4;
        if (e >= a.k) continue;
        *reinterpret_cast<u32*>(out + e) = four_codes(v[i], u);
    }
    if (tid == 0) a.scales[row] = u.scale;
}

// Many rows: a wave for each, N runs of eight values a lane (16 bytes of fp16,
// one store of codes), no meeting of waves.
template <int N, bool F16>
__global__ void __launch_bounds__(256) quantize_rows_kernel(QuantizeArgs a) {
    const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (row >= a.rows) return;
    const int lane = threadIdx.x & 63;
    float v[N][8];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int e = (i * 64 + lane) * 8;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
        if (e >= a.k) continue;
        if constexpr (F16) {
            const f16x8 w = *reinterpret_cast<const f16x8*>(static_cast<const f16*>(a.x) + row * a.stride + e);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = (float)w[j];
        } else {
            const f32x4* const p = reinterpret_cast<const f32x4*>(static_cast<const float*>(a.x) + row * a.stride + e);
            const f32x4 x = p[0], y = p[1];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[i][j] = x[j];
                v[i][j + 4] = y[j];
            }
        }
    }
    u32 bits = 0;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) larger(bits, v[i][j]);
    const Unit u = unit_of(top_of(bits));
    int8_t* const out = a.codes + row * (int64_t)a.k;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int e = (i * 64 + lane) * 8;
        if (e >= a.k) continue;
        *reinterpret_cast<u32x2*>(out + e) = u32x2{four_codes(v[i], u), four_codes(v[i] + 4, u)};
    }
    if (lane == 0) a.scales[row] = u.scale;
}

template <int T, int PER>
hipError_t launch(const QuantizeArgs& a, hipStream_t st) {
    if (a.vec)
        quantize_kernel<T, PER, true><<<dim3((unsigned)a.rows), dim3(T), 0, st>>>(a);
    else
        quantize_kernel<T, PER, false><<<dim3((unsigned)a.rows), dim3(T), 0, st>>>(a);
    return hipGetLastError();
}

template <int N>
hipError_t launch_rows(const QuantizeArgs& a, hipStream_t st) {
    const dim3 grid((unsigned)((a.rows + 3) / 4));
    if (a.f16)
        quantize_rows_kernel<N, true><<<grid, dim3(256), 0, st>>>(a);
    else
        quantize_rows_kernel<N, false><<<grid, dim3(256), 0, st>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize(const QuantizeArgs& a, hipStream_t st) {
    // A wave for each row, where a work-group has little to do for one and there are
    // rows for all waves (32768 rows of 768 in fp16: 17.8 us against 26.7); longer
    // rows take the same either way (8192 of 2048: 14.6 against 13.9), and few are
    // quicker through with four waves each (37 of 2048: 4.5 against 2.8).
    if (a.vec8 && a.k <= 1024 && a.rows >= 2048) return a.k <= 512 ? launch_rows<1>(a, st) : launch_rows<2>(a, st);
    if (a.k <= 1024) return launch<256, 1>(a, st);
    if (a.k <= 2048) return launch<256, 2>(a, st);
    if (a.k <= 4096) return launch<256, 4>(a, st);
    if (a.k <= 8192) return launch<512, 4>(a, st);
    if (a.k <= 16384) return launch<1024, 4>(a, st);
    return launch<1024, 8>(a, st);
}

}  // namespace qmm
