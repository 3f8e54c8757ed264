// gemm_i8.hip -- products of 8-bit codes with a scale for each row of either
// side, on the integer matrix cores:
//   y[p][j] = xs[r] ws[e][j] sum_k x[r][k] w[e][j][k],   r = x_rows[p] or p,
// over one weight matrix or over rows grouped by expert, and its gated form
// h = silu(gate) * up over two stacks.
//
// Sums of products are exact in 32-bit integers, whatever their order, so K
// can be cut anywhere and results repeat bit for bit.
#include <type_traits>

#include "layer_device.h"
#include "moe_kernels.h"

namespace qmm {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));
typedef f16 f16x4v __attribute__((ext_vector_type(4)));

__device__ __forceinline__ u32x4 bounded_rsrc(const void* p, u32 bytes) {
    const uint64_t a = reinterpret_cast<uint64_t>(p);
    return u32x4{(u32)uniform((int)a), (u32)uniform((int)(a >> 32)) & 0xffffu, (u32)uniform((int)bytes), (u32)RSRC_WORD3};
}

// Which rows a work-group takes: expert e's rows from..to (at most BM of them),
// or none.
struct RowTile {
    int e;
    int64_t from, to;
};

// Row tile `tile` of a launch: experts' rows are cut into tiles of `bm`, one
// expert's behind the other's.  Offsets are clamped to the given rows.
__device__ __forceinline__ RowTile find_rows(const GemmI8Args& a, int tile, int bm) {
    if (!a.offsets) {
        const int64_t from = (int64_t)tile * bm;
        return {0, from, from + bm < a.rows ? from + bm : a.rows};
    }
    const int lane = threadIdx.x & 63;
    int left = tile;  // tiles of the experts before
    for (int e0 = 0; e0 < a.experts; e0 += 64) {
        const int e = e0 + lane;
        int64_t lo = 0, hi = 0;
        if (e < a.experts) {
            lo = a.offsets[e];
            hi = a.offsets[e + 1];
            lo = lo < 0 ? 0 : lo > a.rows ? a.rows : lo;
            hi = hi < lo ? lo : hi > a.rows ? a.rows : hi;
        }
        const int n = (int)((hi - lo + bm - 1) / bm);
        int sum = n;
        for (int d = 1; d < 64; d *= 2) {
            const int x = __shfl_up(sum, d, 64);
            if (lane >= d) sum += x;
        }
        const uint64_t past = __ballot(sum > left);
        if (past) {
            const int who = __ffsll((unsigned long long)past) - 1;
            const int from = __shfl((int)lo + (left - (sum - n)) * bm, who, 64), end = __shfl((int)hi, who, 64);
            return {uniform(e0 + who), uniform(from), uniform(from + bm < end ? from + bm : end)};
        }
        left -= __shfl(sum, 63, 64);
    }
    return {0, 0, 0};
}

// Where activation row of product row p lies, -1 if p has none.
__device__ __forceinline__ int64_t activation_row(const GemmI8Args& a, int64_t p) {
    const int64_t r = a.x_rows ? (int64_t)a.x_rows[p] : p;
    return r >= 0 && r < a.x_rows_count ? r : -1;
}

__device__ __forceinline__ float silu(float v) { return v / (1.f + expf(-v)); }

// Four neighbouring columns j.. of row p: sums times scales, out.
template <bool GLU>
__device__ __forceinline__ void store4(const GemmI8Args& a, int64_t p, int e, int64_t j, float xs, const int (&g)[4], const int (&u)[4]) {
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t at = (int64_t)e * a.n + j + i;
        const bool in = j + i < a.n;
        v[i] = (float)g[i] * xs * (in ? a.ws[at] : 0.f);
        if constexpr (GLU) v[i] = silu(v[i]) * ((float)u[i] * xs * (in ? a.ws2[at] : 0.f));
    }
    const int64_t at = p * a.n + j;
    if (a.n % 4 == 0) {
        if (j >= a.n) return;
        if (a.y16)
            *reinterpret_cast<f16x4v*>(static_cast<f16*>(a.y) + at) = f16x4v{(f16)v[0], (f16)v[1], (f16)v[2], (f16)v[3]};
        else
            *reinterpret_cast<f32x4*>(static_cast<float*>(a.y) + at) = f32x4{v[0], v[1], v[2], v[3]};
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (j + i >= a.n) continue;
        if (a.y16)
            static_cast<f16*>(a.y)[at + i] = (f16)v[i];
        else
            static_cast<float*>(a.y)[at + i] = v[i];
    }
}

// ---- few rows: bound by the weights' bytes -------------------------------
// Each of W waves takes its share of K of 16 NB columns and 16 MB rows, weights
// from memory to registers in the order of the matrix instruction, and the
// shares meet in LDS.
template <int W, int NB, int MB, bool GLU>
__global__ void __launch_bounds__(64 * W) rows_i8_kernel(GemmI8Args a) {
    constexpr int S = GLU ? 2 : 1;
    __shared__ i32x4 part[W][S][NB][MB][64];
    const int lane = threadIdx.x & 63, wave = uniform((int)(threadIdx.x >> 6));
    const int ncols = (int)((a.n + 16 * NB - 1) / (16 * NB));
    const RowTile rt = find_rows(a, (int)(blockIdx.x / ncols), 16 * MB);
    if (rt.from >= rt.to) return;
    const int64_t n0 = (int64_t)(blockIdx.x % ncols) * (16 * NB);
    const int r = lane & 15, piece = lane >> 4;
    const u32 wbytes = (u32)(a.n * a.k), xbytes = (u32)(a.x_rows_count * a.k);
    const rsrc_t wr = make_rsrc(a.w + (int64_t)rt.e * a.n * a.k, wbytes);
    const rsrc_t ur = make_rsrc(GLU ? a.w2 + (int64_t)rt.e * a.n * a.k : a.w, wbytes);
    const rsrc_t xr = make_rsrc(a.x, xbytes);
    u32 woff[NB], xoff[MB];
#pragma unroll
    for (int b = 0; b < NB; ++b) woff[b] = n0 + 16 * b + r < a.n ? (u32)(n0 + 16 * b + r) * (u32)a.k : wbytes;
#pragma unroll
    for (int b = 0; b < MB; ++b) {
        const int64_t p = rt.from + 16 * b + r;
        const int64_t x = p < rt.to ? activation_row(a, p) : -1;
        xoff[b] = x >= 0 ? (u32)x * (u32)a.k : xbytes;
    }
    i32x4 acc[S][NB][MB];
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int c = 0; c < MB; ++c) acc[s][b][c] = i32x4{0, 0, 0, 0};
    // 64 codes a step; behind K the loads give zeros.
    const int steps = (a.k + 63) / 64;
#pragma unroll 2
    for (int st = wave; st < steps; st += W) {
        const int k = st * 64 + 16 * piece;
        const bool in = k < a.k;
        i32x4 w[S][NB], x[MB];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const u32 at = in && woff[b] < wbytes ? woff[b] + (u32)k : wbytes;
            w[0][b] = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(wr, at, 0, 0));
            if constexpr (GLU) w[S - 1][b] = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(ur, at, 0, 0));
        }
#pragma unroll
        for (int c = 0; c < MB; ++c) {
            const u32 at = in && xoff[c] < xbytes ? xoff[c] + (u32)k : xbytes;
            x[c] = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(xr, at, 0, 0));
        }
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int c = 0; c < MB; ++c)
                    acc[s][b][c] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[s][b], x[c], acc[s][b][c], 0, 0, 0);
    }
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int c = 0; c < MB; ++c) part[wave][s][b][c][lane] = acc[s][b][c];
    __syncthreads();
    // Lane l of a 16 x 16 block holds columns 4 (l / 16) .. of row l % 16.
    for (int q = threadIdx.x; q < NB * MB * 64; q += 64 * W) {
        const int l = q & 63, b = (q >> 6) % NB, c = (q >> 6) / NB;
        i32x4 sum[S];
#pragma unroll
        for (int s = 0; s < S; ++s) {
            sum[s] = part[0][s][b][c][l];
#pragma unroll
            for (int w = 1; w < W; ++w) sum[s] += part[w][s][b][c][l];
        }
        const int64_t p = rt.from + 16 * c + (l & 15);
        if (p >= rt.to) continue;
        const int64_t x = activation_row(a, p);
        const float xs = x >= 0 ? a.xs[x] : __builtin_nanf("");
        int g[4], u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            g[i] = sum[0][i];
            u[i] = sum[S - 1][i];
        }
        store4<GLU>(a, p, rt.e, n0 + 16 * b + 4 * (l >> 4), xs, g, u);
    }
}

// ---- many rows: bound by the matrix cores --------------------------------
// A work-group of WM x WN waves holds BM rows and BN columns (of each stack, if
// gated); both sides go straight from memory to LDS, 128 codes a step, two
// stages.  LDS rows are 128 bytes of eight 16-byte pieces; piece q of row r is
// in slot q ^ f(r), so that sixteen rows' same piece lies on all banks.
__device__ __forceinline__ int slot_of(int r, int q) { return q ^ ((r & 7) ^ ((r >> 3) & 1)); }

template <int WM, int WN, int MF, int NF, bool GLU>
__global__ void __launch_bounds__(64 * WM * WN) tile_i8_kernel(GemmI8Args a) {
    constexpr int S = GLU ? 2 : 1, WAVES = WM * WN;
    constexpr int BM = 32 * MF * WM, BN = 32 * NF * WN;  // columns of each stack
    constexpr int BK = 128, ROWS = BM + S * BN, STAGE = ROWS * BK;
    constexpr int LOADS = ROWS / 8 / WAVES;  // of one kilobyte, eight rows, per wave
    static_assert(ROWS % (8 * WAVES) == 0, "whole loads");
    __shared__ __attribute__((aligned(1024))) unsigned char lds[2 * STAGE];
    const int lane = threadIdx.x & 63, wave = uniform((int)(threadIdx.x >> 6));
    const int ncols = (int)((a.n + BN - 1) / BN);
    const RowTile rt = find_rows(a, (int)(blockIdx.x / ncols), BM);
    if (rt.from >= rt.to) return;
    const int64_t n0 = (int64_t)(blockIdx.x % ncols) * BN;
    const u32 wbytes = (u32)(a.n * a.k), xbytes = (u32)(a.x_rows_count * a.k);
    const int64_t stack = (int64_t)rt.e * a.n * a.k;
    const u32x4 wr = bounded_rsrc(a.w + stack, wbytes), xr = bounded_rsrc(a.x, xbytes);
    const u32x4 ur = GLU ? bounded_rsrc(a.w2 + stack, wbytes) : wr;
    // Load i of this wave brings LDS rows 8 (LOADS wave + i) .. + 7: first the
    // activations', then the gate's (or the only) columns', then the up's.
    u32 off[LOADS];
    int at_k[LOADS];
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
        const int row = 8 * (LOADS * wave + i) + (lane >> 3);
        at_k[i] = 16 * slot_of(row, lane & 7);
        if (row < BM) {
            const int64_t p = rt.from + row;
            const int64_t x = p < rt.to ? activation_row(a, p) : -1;
            off[i] = x >= 0 ? (u32)x * (u32)a.k + (u32)at_k[i] : xbytes;
        } else {
            const int64_t j = n0 + (row - BM) % BN;
            off[i] = j < a.n ? (u32)j * (u32)a.k + (u32)at_k[i] : wbytes;
        }
    }
    auto load = [&](int st) {
        const u32 stage = (u32)(st & 1) * STAGE;
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const int row = 8 * (LOADS * wave + i);  // of the first lane: one side for all of them
            const u32 to = lds_address(lds + stage + row * BK);
            // Behind K, and where there is no row, the load gives zeros.
            const u32 end = row < BM ? xbytes : wbytes;
            const u32 o = st * BK + at_k[i] < a.k && off[i] < end ? off[i] + (u32)(st * BK) : end;
            if (row < BM)
                load_to_lds(xr, o, to);
            else if (row < BM + BN)
                load_to_lds(wr, o, to);
            else
                load_to_lds(ur, o, to);
        }
    };
    const int wm = wave % WM, wn = wave / WM;
    const int r = lane & 31, h = lane >> 5;
    i32x16 acc[S][NF][MF];
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
        for (int i = 0; i < NF; ++i)
#pragma unroll
            for (int j = 0; j < MF; ++j)
#pragma unroll
                for (int v = 0; v < 16; ++v) acc[s][i][j][v] = 0;
    const int steps = (a.k + BK - 1) / BK;
    load(0);
    for (int st = 0; st < steps; ++st) {
        // The stage's loads, this wave's, are there, and what it read of the
        // other stage too; behind the barrier everybody's.
        __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0), lgkmcnt(0)
        asm volatile("s_barrier" ::: "memory");
        if (st + 1 < steps) load(st + 1);
        const unsigned char* base = lds + (st & 1) * STAGE;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
            i32x4 w[S][NF], x[MF];
#pragma unroll
            for (int j = 0; j < MF; ++j) {
                const int row = (wm * MF + j) * 32 + r;
                x[j] = *reinterpret_cast<const i32x4*>(base + row * BK + 16 * slot_of(row, 2 * kk + h));
            }
#pragma unroll
            for (int s = 0; s < S; ++s)
#pragma unroll
                for (int i = 0; i < NF; ++i) {
                    const int row = BM + s * BN + (wn * NF + i) * 32 + r;
                    w[s][i] = *reinterpret_cast<const i32x4*>(base + row * BK + 16 * slot_of(row, 2 * kk + h));
                }
#pragma unroll
            for (int s = 0; s < S; ++s)
#pragma unroll
                for (int i = 0; i < NF; ++i)
#pragma unroll
                    for (int j = 0; j < MF; ++j)
                        acc[s][i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(w[s][i], x[j], acc[s][i][j], 0, 0, 0);
        }
    }
    // Lane l of a 32 x 32 block holds columns 8 b + 4 (l / 32) .. + 3 of row l % 32.
#pragma unroll
    for (int j = 0; j < MF; ++j) {
        const int64_t p = rt.from + (wm * MF + j) * 32 + r;
        if (p >= rt.to) continue;
        const int64_t x = activation_row(a, p);
        const float xs = x >= 0 ? a.xs[x] : __builtin_nanf("");
#pragma unroll
        for (int i = 0; i < NF; ++i)
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                int g[4], u[4];
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    g[v] = acc[0][i][j][4 * b + v];
                    u[v] = acc[S - 1][i][j][4 * b + v];
                }
                store4<GLU>(a, p, rt.e, n0 + (wn * NF + i) * 32 + 8 * b + 4 * h, xs, g, u);
            }
    }
}

// Row tiles of `bm` that a launch needs at most: every expert's last one may be
// begun.
int64_t row_tiles(const GemmI8Args& a, int bm) {
    if (!a.offsets) return (a.rows + bm - 1) / bm;
    const int64_t begun = a.rows < a.experts ? a.rows : a.experts;
    return a.rows / bm + begun;
}

template <int W, int NB, int MB, bool GLU>
hipError_t launch_rows(const GemmI8Args& a, hipStream_t st) {
    const int64_t grid = row_tiles(a, 16 * MB) * ((a.n + 16 * NB - 1) / (16 * NB));
    if (grid > 0x7fffffff / (64 * W)) return hipErrorInvalidConfiguration;
    rows_i8_kernel<W, NB, MB, GLU><<<dim3((unsigned)grid), dim3(64 * W), 0, st>>>(a);
    return hipGetLastError();
}

template <int WM, int WN, int MF, int NF, bool GLU>
hipError_t launch_tile(const GemmI8Args& a, hipStream_t st) {
    constexpr int BM = 32 * MF * WM, BN = 32 * NF * WN;
    const int64_t grid = row_tiles(a, BM) * ((a.n + BN - 1) / BN);
    if (grid > 0x7fffffff / (64 * WM * WN)) return hipErrorInvalidConfiguration;
    tile_i8_kernel<WM, WN, MF, NF, GLU><<<dim3((unsigned)grid), dim3(64 * WM * WN), 0, st>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_gemm_i8(const GemmI8Args& a, hipStream_t st) {
    // Rows that a matrix meets.
    const int64_t per = a.offsets ? (a.rows + a.experts - 1) / a.experts : a.rows;
    if (a.w2) {
        if (per <= 16) return launch_rows<8, 1, 1, true>(a, st);
        if (per <= 64) return launch_rows<8, 1, 2, true>(a, st);
        return launch_tile<2, 2, 2, 1, true>(a, st);
    }
    if (per <= 16) return launch_rows<8, 1, 1, false>(a, st);
    if (per <= 64) return launch_rows<8, 1, 4, false>(a, st);
    return launch_tile<2, 2, 2, 2, false>(a, st);
}

}  // namespace qmm
