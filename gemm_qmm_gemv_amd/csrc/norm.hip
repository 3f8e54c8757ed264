// norm.hip -- the step between two products of a decoder layer:
//   u = y [* rsqrt(mean(y^2) + eps) * post] [* gate],
//   h = residual + scale * u                                   (fp32, written)
//   x = fp16(h * rsqrt(mean(h^2) + eps) * pre)                 (written)
//
// Bound by memory: every operand is read once and every result written once.
// A work-group holds one row in registers (PER runs of four per thread), so
// both sums of squares and the two products cost no second read.  8192 rows of
// 4096 with all operands (537 MB) take 94 us, 5.7 TB/s, the rate of a copy of
// that size (5.4); 512 threads a row took 1 % more, 1024 13 %.  4096 rows of 4095
// (268 MB), element by element, take 72 us, 3.8 TB/s.  Sums of squares
// are fp32: lanes add their own terms, then the lanes of each wave, then the
// waves' sums in wave order (a fixed order, so results repeat bit for bit).
#include "layer_device.h"
#include "layer_kernels.h"

namespace qmm {
namespace {

typedef float f32x4v __attribute__((ext_vector_type(4)));
typedef f16 f16x4v __attribute__((ext_vector_type(4)));

template <int T>
__device__ __forceinline__ float block_sum(float v, float* lds) {
    v = over_lanes<64>(v, add_f32);
    if constexpr (T > 64) {
        if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
        __syncthreads();
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < T / 64; ++i) s += lds[i];
        v = s;
    }
    return v;
}

// Element j of run i of this thread.  With VEC a run is four neighbours (one
// 16-byte access); otherwise (an odd n or stride, or pointers aligned to
// their elements only) neighbours lie on neighbouring threads.
template <int T, bool VEC>
__device__ __forceinline__ int at(int i, int j) {
    return VEC ? (i * T + (int)threadIdx.x) * 4 + j : (i * 4 + j) * T + (int)threadIdx.x;
}

// Run i of a row of fp32 or fp16; zeros behind its end.
template <int T, bool VEC, typename F>
__device__ __forceinline__ f32x4v load_run(const F* p, int n, int i) {
    typedef F f4 __attribute__((ext_vector_type(4)));
    f32x4v r = {0.f, 0.f, 0.f, 0.f};
    if constexpr (VEC) {
        const int e = at<T, VEC>(i, 0);
        if (e < n) {
            const f4 v = *reinterpret_cast<const f4*>(p + e);
            r = f32x4v{(float)v[0], (float)v[1], (float)v[2], (float)v[3]};
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int e = at<T, VEC>(i, j);
            if (e < n) r[j] = (float)p[e];
        }
    }
    return r;
}

template <int T, int PER, bool VEC, typename F>
__device__ __forceinline__ void load_row(const F* p, int n, f32x4v (&r)[PER]) {
#pragma unroll
    for (int i = 0; i < PER; ++i) r[i] = load_run<T, VEC>(p, n, i);
}

template <int T, int PER, bool VEC>
__global__ void __launch_bounds__(T) norm_kernel(NormArgs a) {
    // Up to 2048 elements, where a call is a chain of latencies, weights and
    // gate are asked for with the rest (1.5 us for one row of 1024).  Longer
    // rows take them where they are used: held from the start they cost three
    // waves of eight (8192 rows of 4096 with all operands: 2 % more).
    constexpr bool EARLY = PER <= 2;
    __shared__ float lds[2][T / 64];
    const int64_t row = blockIdx.x;
    const int n = a.n;
    const float* gate = a.gate + row * a.gate_stride;
    f32x4v h[PER], y[PER], g[PER], post[PER], pre[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) h[i] = y[i] = f32x4v{0.f, 0.f, 0.f, 0.f};
    if (a.y) {
        if (a.y_fp16)
            load_row<T, PER, VEC>(static_cast<const f16*>(a.y) + row * a.y_stride, n, y);
        else
            load_row<T, PER, VEC>(static_cast<const float*>(a.y) + row * a.y_stride, n, y);
    }
    if (a.res) load_row<T, PER, VEC>(a.res + row * n, n, h);
    if constexpr (EARLY) {
        if (a.gate) load_row<T, PER, VEC>(gate, n, g);
        if (a.post) load_row<T, PER, VEC>(a.post, n, post);
        if (a.pre) load_row<T, PER, VEC>(a.pre, n, pre);
    }
    if (a.y) {
        if (a.post) {
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < PER; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) s += y[i][j] * y[i][j];
            s = block_sum<T>(s, lds[0]);
            const float r = 1.f / sqrtf(s / (float)n + a.eps);
#pragma unroll
            for (int i = 0; i < PER; ++i) y[i] = y[i] * r * (EARLY ? post[i] : load_run<T, VEC>(a.post, n, i));
        }
        if (a.gate) {
#pragma unroll
            for (int i = 0; i < PER; ++i) y[i] = y[i] * (EARLY ? g[i] : load_run<T, VEC>(gate, n, i));
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) h[i] = h[i] + y[i] * a.scale;
        if (a.h) {
            float* out = a.h + row * n;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                if constexpr (VEC) {
                    const int e = at<T, VEC>(i, 0);
                    if (e < n) *reinterpret_cast<f32x4v*>(out + e) = h[i];
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int e = at<T, VEC>(i, j);
                        if (e < n) out[e] = h[i][j];
                    }
                }
            }
        }
    }
    if (!a.x) return;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s += h[i][j] * h[i][j];
    s = block_sum<T>(s, lds[1]);
    const float r = 1.f / sqrtf(s / (float)n + a.eps);
    f16* out = static_cast<f16*>(a.x) + row * n;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        f32x4v v = h[i] * r;
        if (a.pre) v = v * (EARLY ? pre[i] : load_run<T, VEC>(a.pre, n, i));
        // One rounding to fp16, the type the products take.
        if constexpr (VEC) {
            const int e = at<T, VEC>(i, 0);
            if (e < n) *reinterpret_cast<f16x4v*>(out + e) = f16x4v{(f16)v[0], (f16)v[1], (f16)v[2], (f16)v[3]};
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int e = at<T, VEC>(i, j);
                if (e < n) out[e] = (f16)v[j];
            }
        }
    }
}

template <int T, int PER>
hipError_t launch(const NormArgs& a, hipStream_t st) {
    if (a.vec)
        norm_kernel<T, PER, true><<<dim3((unsigned)a.rows), dim3(T), 0, st>>>(a);
    else
        norm_kernel<T, PER, false><<<dim3((unsigned)a.rows), dim3(T), 0, st>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_norm(const NormArgs& a, hipStream_t st) {
    if (a.n <= 1024) return launch<256, 1>(a, st);
    if (a.n <= 2048) return launch<256, 2>(a, st);
    if (a.n <= 4096) return launch<256, 4>(a, st);
    if (a.n <= 8192) return launch<512, 4>(a, st);
    if (a.n <= 16384) return launch<1024, 4>(a, st);
    return launch<1024, 8>(a, st);
}

}  // namespace qmm
