// moe_gather.hip -- the experts' rows back to their tokens:
//   y[t] = residual[t] + sum_j weights[t][j] * rows[pair_row[t][j]],
// summed in the order of j in fp32, so results repeat bit for bit.
//
// Bound by memory: every row is read once, y written once.
#include "layer_device.h"
#include "moe_kernels.h"

namespace qmm {
namespace {

typedef f16 f16x4v __attribute__((ext_vector_type(4)));

// A thread owns V neighbouring columns of one token.
template <int V, typename F>
__global__ void __launch_bounds__(256) gather_kernel(GatherArgs a) {
    typedef F vec __attribute__((ext_vector_type(V)));
    typedef float fvec __attribute__((ext_vector_type(V)));
    const int64_t t = blockIdx.x;
    const int64_t c = ((int64_t)blockIdx.y * 256 + threadIdx.x) * V;
    if (c >= a.n) return;
    float sum[V];
#pragma unroll
    for (int i = 0; i < V; ++i) sum[i] = 0.f;
    for (int j = 0; j < a.top_k; ++j) {
        const int64_t row = a.pair_row[t * a.top_k + j];
        if (row < 0 || row >= a.p_rows) continue;
        const float w = a.weights[t * a.top_k + j];
        const F* p = static_cast<const F*>(a.rows) + row * a.n + c;
        if constexpr (V > 1) {
            const vec v = *reinterpret_cast<const vec*>(p);
#pragma unroll
            for (int i = 0; i < V; ++i) sum[i] = fmaf(w, (float)v[i], sum[i]);
        } else {
            sum[0] = fmaf(w, (float)p[0], sum[0]);
        }
    }
    if (a.residual) {
#pragma unroll
        for (int i = 0; i < V; ++i) sum[i] += a.residual[t * a.n + c + i];
    }
    if constexpr (V > 1) {
        fvec v;
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = sum[i];
        *reinterpret_cast<fvec*>(a.y + t * a.n + c) = v;
    } else {
        a.y[t * a.n + c] = sum[0];
    }
}

}  // namespace

hipError_t launch_gather(const GatherArgs& a, hipStream_t st) {
    const unsigned width = a.vec ? 1024 : 256;
    const dim3 grid((unsigned)a.tokens, (unsigned)((a.n + width - 1) / width));
    if (a.vec && a.f16)
        gather_kernel<4, f16><<<grid, 256, 0, st>>>(a);
    else if (a.vec)
        gather_kernel<4, float><<<grid, 256, 0, st>>>(a);
    else if (a.f16)
        gather_kernel<1, f16><<<grid, 256, 0, st>>>(a);
    else
        gather_kernel<1, float><<<grid, 256, 0, st>>>(a);
    return hipGetLastError();
}

}  // namespace qmm
