// moe_gather.hip -- the experts' rows back to their tokens:
//   y[t] = residual[t] + sum_j weights[t][j] * rows[pair_row[t][j]],
// summed in the order of j in fp32, so results repeat bit for bit.
//
// Bound by memory: every row is read once, y written once (8192 tokens of 8
// rows of 2048 in fp16, residual, 403 MB: 67.5 us = 6.0 TB/s; 16 tokens: 3.4 us,
// of which the launch is half).  A thread owns 16 bytes of a row (one load);
// indices and weights are the same for a whole work-group, and the rows of up
// to eight choices are asked for before the first is added.
#include "layer_device.h"
#include "moe_kernels.h"

namespace qmm {
namespace {

// A thread owns V neighbouring columns of one token.
template <int V, typename F, bool PAST>
__global__ void __launch_bounds__(256) gather_kernel(GatherArgs a) {
    typedef F vec __attribute__((ext_vector_type(V)));
    constexpr int AHEAD = 8;
    const int64_t t = blockIdx.x;
    const int64_t c = ((int64_t)blockIdx.y * 256 + threadIdx.x) * V;
    if (c >= a.n) return;
    const int32_t* const at = a.pair_row + t * a.top_k;
    const float* const w = a.weights + t * a.top_k;
    const F* const rows = static_cast<const F*>(a.rows) + c;
    float sum[V];
#pragma unroll
    for (int i = 0; i < V; ++i) sum[i] = 0.f;
    for (int j0 = 0; j0 < a.top_k; j0 += AHEAD) {
        vec v[AHEAD];
        bool there[AHEAD];
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
            const int64_t row = j0 + j < a.top_k ? at[j0 + j] : -1;
            there[j] = row >= 0 && row < a.p_rows;
            if (!there[j]) continue;
            const vec* const from = reinterpret_cast<const vec*>(rows + row * a.n);
            if constexpr (PAST)
                v[j] = __builtin_nontemporal_load(from);
            else
                v[j] = *from;
        }
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
            if (!there[j]) continue;
            const float f = w[j0 + j];
#pragma unroll
            for (int i = 0; i < V; ++i) sum[i] = fmaf(f, (float)v[j][i], sum[i]);
        }
    }
    float* const y = a.y + t * a.n + c;
    if constexpr (V == 1) {
        y[0] = a.residual ? a.residual[t * a.n + c] + sum[0] : sum[0];
    } else {
        f32x4 out[V / 4];
#pragma unroll
        for (int i = 0; i < V; ++i) out[i / 4][i % 4] = sum[i];
#pragma unroll
        for (int i = 0; i < V / 4; ++i) {
            if (a.residual) out[i] += reinterpret_cast<const f32x4*>(a.residual + t * a.n + c)[i];
            reinterpret_cast<f32x4*>(y)[i] = out[i];
        }
    }
}

template <int V, typename F, bool PAST>
hipError_t launch(const GatherArgs& a, hipStream_t st) {
    const dim3 grid((unsigned)a.tokens, (unsigned)((a.n + 256 * V - 1) / (256 * V)));
    gather_kernel<V, F, PAST><<<grid, dim3(256), 0, st>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_gather(const GatherArgs& a, hipStream_t st) {
    // Rows that the 256 MB of memory-side cache cannot hold are read past the
    // caches (8192 tokens of 8 rows of 2048, fp16, 256 MiB: 86 -> 69 us; fp32 132 ->
    // 107); what fits may lie there from the product before (128 MiB read from
    // there: 33 us, past it 36).
    const bool past = a.tokens * a.top_k * a.n * (a.f16 ? 2 : 4) >= (int64_t)192 << 20;
    if (!a.vec) return a.f16 ? launch<1, f16, false>(a, st) : launch<1, float, false>(a, st);
    if (a.f16) return past ? launch<8, f16, true>(a, st) : launch<8, f16, false>(a, st);
    return past ? launch<4, float, true>(a, st) : launch<4, float, false>(a, st);
}

}  // namespace qmm
