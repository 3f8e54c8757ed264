// quantize.hip -- rows of activations to 8-bit codes with a scale for each row:
//   scale = fp32(max |x| / 127),  code = round(x / scale), ties to even.
//
// Bound by memory.  A work-group holds one row in registers (PER runs of four
// per thread), so that the maximum and the codes cost one read.  The quotient
// is formed by a product with 1 / scale and put right by what it leaves over:
// x - code * scale is exact in one fused step (the code's product with the scale
// and x agree in all leading bits), so the code is the whole number next to
// the real quotient, at less than a division's cost.
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
    // A value that is not finite makes the row's scale NaN (x - x is NaN then,
    // and the sum of zeros elsewhere).
    float top = 0.f, bad = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            top = fmaxf(top, fabsf(v[i][j]));
            bad += v[i][j] - v[i][j];
        }
    if (bad != bad) top = __builtin_huge_valf();
    const auto larger = [](float x, float y) { return fmaxf(x, y); };
    top = over_lanes<64>(top, larger);
    if constexpr (T > 64) {
        if ((tid & 63) == 0) lds[tid >> 6] = top;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < T / 64; ++i) top = fmaxf(top, lds[i]);
    }
    const bool finite = top < __builtin_huge_valf();
    const float scale = finite ? top / 127.f : __builtin_nanf("");
    // 1 / scale may leave fp32 for the smallest scales: such rows are scaled up
    // first, which is exact.
    const float up = scale < 0x1p-100f ? 0x1p100f : 1.f;
    const float s = scale * up, inv = finite && s > 0.f ? 1.f / s : 0.f;
    int8_t* const out = a.codes + row * (int64_t)a.k;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = (i * T + tid) * 4;
        if (e >= a.k) continue;
        u32 w = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int q = inv > 0.f ? code_of(v[i][j] * up, s, inv) : 0;
            w |= ((u32)q & 255u) << (8 * j);
        }
        *reinterpret_cast<u32*>(out + e) = w;
    }
    if (tid == 0) a.scales[row] = scale;
}

template <int T, int PER>
hipError_t launch(const QuantizeArgs& a, hipStream_t st) {
    if (a.vec)
        quantize_kernel<T, PER, true><<<dim3((unsigned)a.rows), dim3(T), 0, st>>>(a);
    else
        quantize_kernel<T, PER, false><<<dim3((unsigned)a.rows), dim3(T), 0, st>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize(const QuantizeArgs& a, hipStream_t st) {
    if (a.k <= 1024) return launch<256, 1>(a, st);
    if (a.k <= 2048) return launch<256, 2>(a, st);
    if (a.k <= 4096) return launch<256, 4>(a, st);
    if (a.k <= 8192) return launch<512, 4>(a, st);
    if (a.k <= 16384) return launch<1024, 4>(a, st);
    return launch<1024, 8>(a, st);
}

}  // namespace qmm
