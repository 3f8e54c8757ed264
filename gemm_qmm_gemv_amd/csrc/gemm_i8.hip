// gemm_i8.hip -- products of 8-bit codes with a scale for each row of either
// side, on the integer matrix cores:
//   y[p][j] = xs[r] ws[e][j] sum_k x[r][k] w[e][j][k],   r = x_rows[p] or p,
// over one weight matrix or over rows grouped by expert, and its gated form
// h = silu(gate) * up over two stacks.
//
// Sums of products are exact in 32-bit integers, whatever their order (32768
// codes of -128 make 2^29), so K can be cut anywhere and results repeat bit for
// bit.
#include <algorithm>
#include <cmath>

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
// shares meet in LDS.  16 tokens, 8 of 128 experts each, gate and up (768 of
// 2048; 193 MB of weights): 34.6 us = 5.6 TB/s.  Where a matrix is small the waits
// are what is left, for both sides and then for the other waves: one row of 2048
// x 1024 3.2 us, 37 of 8192 x 2048 (17 MB) 8.1.
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
    // 128 codes of each row at a time, in two steps of the matrix instruction;
    // behind K the loads give zeros.
    const int chunks = (a.k + 127) / 128;
    for (int ch = wave; ch < chunks; ch += W) {
        i32x4 w[2][S][NB], x[2][MB];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int k = ch * 128 + 64 * q + 16 * piece;
            const bool in = k < a.k;
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const u32 at = in && woff[b] < wbytes ? woff[b] + (u32)k : wbytes;
                w[q][0][b] = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(wr, at, 0, 0));
                if constexpr (GLU) w[q][S - 1][b] = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(ur, at, 0, 0));
            }
#pragma unroll
            for (int c = 0; c < MB; ++c) {
                const u32 at = in && xoff[c] < xbytes ? xoff[c] + (u32)k : xbytes;
                x[q][c] = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(xr, at, 0, 0));
            }
        }
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int s = 0; s < S; ++s)
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int c = 0; c < MB; ++c)
                        acc[s][b][c] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[q][s][b], x[q][c], acc[s][b][c], 0, 0, 0);
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
//
// A work-group stays for several tiles: the first stage of the next one is
// fetched during the last step of this one, and its sums leave through the
// stage that this step has read, while the other fills.
//
// A tile of 256 x 256 brings 64 KB for each step and multiplies 8 million pairs
// of codes with them; one of 128 x 128, two of which share a compute unit and
// hide each other's ends, brings twice as much for that.  8192 cubed: 442 to 446
// us = 2.5 POP/s, matrix cores 82 % busy at the clock that this load leaves (a loop
// of the instruction alone, 3.6); 8192 x 16384 of 2048 in fp16 254 us = 2.2.
// 4096 tokens, 8 of 128 experts each: gate and up (768 of 2048) 169 to 184 us,
// down (2048 of 768, fp32) 124 to 127; there, what an expert's last tile lacks in
// rows, weights that arrive only one step ahead, and tiles that do not come out
// even for the device leave the matrix cores 36 % and 23 % busy, memory at 3.7
// and 4.2 TB/s.
//
// What was slower: steps of 64 codes in four stages (8192 cubed, at a time when
// this took 495 us: 523), tiles of 256 x 128 with such steps, two on a unit
// (593), four waves of 128 x 128 (676) and eight for 256 x 256 (3 %), weights
// asked for into the L2 a step earlier (6 %), the 16 x 16 x 64 instruction (2.3
// against 3.6 POP/s by itself), a branch for each block of 32 rows without rows
// (spills), higher priority for waves that multiply (1 %) or load (4 %), bands
// of whole experts (3 %).
constexpr int BK = 128;
__device__ __forceinline__ int slot_of(int r, int q) { return q ^ ((r & 7) ^ ((r >> 3) & 1)); }

// Work-group barrier behind this wave's LDS reads and writes, and its loads.
__device__ __forceinline__ void loads_barrier() {
    __builtin_amdgcn_s_waitcnt(7 << 4);  // vmcnt(0), lgkmcnt(0)
    asm volatile("s_barrier" ::: "memory");
}
// The same behind all but the newest N of its loads.
template <int N>
__device__ __forceinline__ void older_loads_barrier() {
    static_assert(N < 64, "what the counter holds");
    __builtin_amdgcn_s_waitcnt((N & 15) | (N >> 4) << 14 | 7 << 4);  // vmcnt(N), lgkmcnt(0)
    asm volatile("s_barrier" ::: "memory");
}
// The same without the loads.
__device__ __forceinline__ void lds_barrier() {
    __builtin_amdgcn_s_waitcnt(15 | 3 << 14 | 7 << 4);  // lgkmcnt(0)
    asm volatile("s_barrier" ::: "memory");
}

// Where each expert's row tiles begin: table [2][experts + 1], filled by the
// first wave: tiles before (behind the last expert: all), offsets inside the
// rows.  (Offsets that fall and rise again may count more tiles than a launch can
// have; 2^30 is more than any has.)
__device__ __forceinline__ void fill_table(const GemmI8Args& a, int bm, int* table) {
    constexpr u32 MOST = 1u << 30;
    const int lane = threadIdx.x & 63;
    u32 before = 0;
    for (int e0 = 0; e0 < a.experts; e0 += 64) {
        const int e = e0 + lane;
        int64_t lo = 0, hi = 0;
        if (e < a.experts) {
            lo = a.offsets[e];
            hi = a.offsets[e + 1];
            lo = lo < 0 ? 0 : lo > a.rows ? a.rows : lo;
            hi = hi < lo ? lo : hi > a.rows ? a.rows : hi;
        }
        const u32 n = (u32)((hi - lo + bm - 1) / bm);
        u32 sum = n;
        for (int d = 1; d < 64; d *= 2) {
            const u32 x = __shfl_up(sum, d, 64);
            if (lane >= d) sum += x;
        }
        if (e < a.experts) {
            table[e] = (int)(before + sum - n < MOST ? before + sum - n : MOST);
            table[a.experts + 1 + e] = (int)lo;
            if (e == a.experts - 1) table[a.experts + 1 + a.experts] = (int)hi;
        }
        before += __shfl(sum, 63, 64);
        before = before < MOST ? before : MOST;
    }
    if (lane == 0) table[a.experts] = (int)before;
}

struct Tile {
    int e, from, to;  // rows from .. to - 1 of expert e
    int n0;
};

// v, of which the compiler does not know that it is the same every time: what
// is worked out of it stays where it is used and holds no registers elsewhere.
__device__ __forceinline__ int again(int v) {
    asm volatile("" : "+v"(v));
    return v;
}

// Tile t of rtiles x ncols, in bands of row tiles, so that what a die's L2 holds
// of both sides is used again: of five (8192 cubed: 442 us, of two or four 449, of
// one 488), and of two where experts follow each other, which share no weights
// (8192 tokens through 128 experts' gate and up of 768: 278, of four 293).
__device__ __forceinline__ Tile tile_at(const GemmI8Args& a, int t, int rtiles, int ncols, int bm, int bn, const int* table) {
    const int band = a.offsets ? 2 : 5, first = t / (band * ncols) * band;
    const int high = rtiles - first < band ? rtiles - first : band;
    const int in = t - first * ncols, row = first + in % high;
    Tile r;
    r.n0 = (in / high) * bn;
    if (!a.offsets) {
        r.e = 0;
        r.from = row * bm;
        r.to = a.rows - r.from < bm ? (int)a.rows : r.from + bm;
        return r;
    }
    // The last expert whose tiles begin at or before this one: 64 places
    // apart, then among those between.
    const int lane = threadIdx.x & 63, apart = (a.experts + 63) / 64;
    const int far = lane * apart;
    const uint64_t some = __ballot(far < a.experts && table[far < a.experts ? far : 0] <= row);
    const int e0 = ((int)__popcll(some) - 1) * apart;
    const int near = e0 + lane;
    const uint64_t those = __ballot(lane < apart && near < a.experts && table[near < a.experts ? near : 0] <= row);
    r.e = uniform(e0 + (int)__popcll(those) - 1);
    r.from = uniform(table[a.experts + 1 + r.e] + (row - table[r.e]) * bm);
    const int end = uniform(table[a.experts + 1 + r.e + 1]);  // the tile has rows, so it is not below the first one
    r.to = end - r.from < bm ? end : r.from + bm;
    return r;
}

// A wave's sums to memory.  Lane l of a 32 x 32 block holds columns
// 8 b + 4 (l / 32) .. + 3 of row l % 32; scaled and rounded they go through LDS
// (32 rows of 128 bytes, pieces swizzled as above), from where whole pieces of
// rows leave 16 bytes a lane.
constexpr int OUT = 32 * 128;  // bytes of LDS per wave

template <typename T, int NF, int MF, bool GLU>
__device__ __forceinline__ void store_block(const GemmI8Args& a, const Tile& t, int m0, int64_t c0, const float* sx,
                                            const float* sg, const float* su, const i32x16 (&acc)[GLU ? 2 : 1][NF][MF],
                                            unsigned char* lds) {
    constexpr int FIT = 128 / (int)sizeof(T), COLS = FIT < 32 * NF ? FIT : 32 * NF;  // at a time
    constexpr int PIECE = 16 / (int)sizeof(T), PIECES = COLS / PIECE;
    static_assert(COLS % 32 == 0 && NF * 32 % COLS == 0, "whole blocks at a time");
    typedef T vec4 __attribute__((ext_vector_type(4)));
    const int lane = again(threadIdx.x & 63), r = lane & 31, h = lane >> 5;
    const bool wide = a.n % PIECE == 0;
    T* const y = static_cast<T*>(a.y);
#pragma unroll
    for (int j = 0; j < MF; ++j) {
        const int64_t p0 = (int64_t)t.from + m0 + 32 * j;
        if (p0 >= t.to) break;
        const float xs = sx[m0 + 32 * j + r];
#pragma unroll
        for (int i0 = 0; i0 < NF; i0 += COLS / 32) {
#pragma unroll
            for (int i = i0; i < i0 + COLS / 32; ++i)
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    const int c = 32 * i + 8 * b + 4 * h;
                    const f32x4 g = *reinterpret_cast<const f32x4*>(sg + c);
                    f32x4 u;
                    if constexpr (GLU) u = *reinterpret_cast<const f32x4*>(su + c);
                    vec4 out;
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        float s = (float)acc[0][i][j][4 * b + v] * xs * g[v];
                        if constexpr (GLU) s = silu(s) * ((float)acc[1][i][j][4 * b + v] * xs * u[v]);
                        out[v] = (T)s;
                    }
                    const int at = (c - 32 * i0) * (int)sizeof(T);
                    *reinterpret_cast<vec4*>(lds + r * 128 + 16 * slot_of(r, at >> 4) + (at & 15)) = out;
                }
            if (wide) {
#pragma unroll
                for (int q0 = 0; q0 < 32 * PIECES; q0 += 64) {
                    const int row = (q0 + lane) / PIECES, piece = (q0 + lane) % PIECES;
                    const u32x4 v = *reinterpret_cast<const u32x4*>(lds + row * 128 + 16 * slot_of(row, piece));
                    const int64_t c = c0 + 32 * i0 + piece * PIECE;
                    if (p0 + row >= t.to || c >= a.n) continue;
                    u32x4* const to = reinterpret_cast<u32x4*>(y + (p0 + row) * a.n + c);
                    if (a.past_caches) {
                        asm volatile("" ::: "memory");  // else the two stores are made one, a plain one
                        __builtin_nontemporal_store(v, to);
                        asm volatile("" ::: "memory");
                    } else {
                        *to = v;
                    }
                }
            } else {
                for (int q = lane; q < 32 * COLS; q += 64) {
                    const int row = q / COLS, at = q % COLS * (int)sizeof(T);
                    const T v = *reinterpret_cast<const T*>(lds + row * 128 + 16 * slot_of(row, at >> 4) + (at & 15));
                    const int64_t c = c0 + 32 * i0 + q % COLS;
                    if (p0 + row < t.to && c < a.n) y[(p0 + row) * a.n + c] = v;
                }
            }
        }
    }
}

template <int WM, int WN, int MF, int NF, bool GLU, int STAGES>
struct TileShape {
    static constexpr int S = GLU ? 2 : 1, WAVES = WM * WN, T = 64 * WAVES;
    static constexpr int BM = 32 * MF * WM, BN = 32 * NF * WN;  // columns of each stack
    static constexpr int ROWS = BM + S * BN, STAGE = ROWS * BK;
    static constexpr int LOADS = ROWS / 8 / WAVES;  // of one kilobyte, eight rows, per wave
    static constexpr int SCALES = (ROWS + T - 1) / T;  // per thread
    static_assert(BM % (8 * WAVES) == 0 && BN % (8 * WAVES) == 0, "a load brings rows of one side in all waves");
    static_assert(BM <= T, "a thread for each row");
    static_assert(WAVES * OUT <= STAGE * (STAGES - 1), "outputs pass through the stages that are read");
};

// STAGES 2: as above.  More: a work-group has one tile, and a step in flight for
// each stage from the start, for launches of few tiles, where the wait for the
// next step is what counts (256 rows, 2048 columns of 8192: tiles of 64 x 64 in
// four stages 19.6 us, in two 30; 512 rows, 4096 of 4096: 128 x 64 in three 15.5,
// the best of two 23).
template <int WM, int WN, int MF, int NF, bool GLU, int OCC, int STAGES>
__global__ void __launch_bounds__(64 * WM * WN, OCC) tile_i8_kernel(GemmI8Args a) {
    using Shape = TileShape<WM, WN, MF, NF, GLU, STAGES>;
    constexpr int S = Shape::S, BM = Shape::BM, BN = Shape::BN, ROWS = Shape::ROWS, STAGE = Shape::STAGE, LOADS = Shape::LOADS;
    constexpr int T = Shape::T, SCALES = Shape::SCALES, WAVES = Shape::WAVES;
    __shared__ __attribute__((aligned(1024))) unsigned char lds[STAGES * STAGE];
    __shared__ __attribute__((aligned(16))) float scales[2 * ROWS];  // of two tiles
    __shared__ int rows_of[BM];
    __shared__ int table[2 * (I8_EXPERTS + 1)];
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int ncols = (int)((a.n + BN - 1) / BN);
    int rtiles;
    if (a.offsets) {
        if (wave == 0) fill_table(a, BM, table);
        __syncthreads();
        const int64_t most = a.rows / BM + (a.rows < a.experts ? a.rows : a.experts);  // as the host has it
        rtiles = uniform(table[a.experts]);
        rtiles = rtiles < most ? rtiles : (int)most;
    } else {
        rtiles = (int)((a.rows + BM - 1) / BM);
    }
    // Each of the 8 dies (work-group i runs on die i % 8) takes neighbouring tiles.
    const int tiles = rtiles * ncols, per = (tiles + 7) / 8, base = (int)(blockIdx.x % 8) * per;
    int count = tiles - base < per ? tiles - base : per;
    const int hop = (int)(gridDim.x / 8);
    int t = (int)(blockIdx.x / 8);
    // A last round for at most half of the work-groups is cut into tiles of half
    // the rows, for twice as many (4500 x 4096 of 4096: 98 -> 91 us; 4096 tokens
    // through 128 experts' down projection 133 -> 129).
    const int whole = count / hop * hop, rest = count - whole;
    const bool halves = whole > 0 && 2 * rest <= hop;
    if (halves) count += rest;
    const auto nth = [&](int i) {
        if (!halves || i < whole) return tile_at(a, base + i, rtiles, ncols, BM, BN, table);
        Tile q = tile_at(a, base + whole + (i - whole) / 2, rtiles, ncols, BM, BN, table);
        const int cut = q.to - q.from < BM / 2 ? q.to : q.from + BM / 2;
        if ((i - whole) % 2)
            q.from = cut;
        else
            q.to = cut;
        return q;
    };
    if (t >= count) return;

    const u32 wbytes = (u32)(a.n * a.k), xbytes = (u32)(a.x_rows_count * a.k);
    const int steps = (a.k + BK - 1) / BK;
    // Load i of this wave brings the eight LDS rows from 8 (i WAVES + wave) on:
    // first the activations', then the gate's (or the only) columns', then the
    // up's.  Which of them is the same for all waves.
    const auto lds_row = [&](int i) { return 8 * (i * WAVES + wave); };
    const auto side = [](int i) constexpr { return 8 * i * WAVES < BM ? 0 : 8 * i * WAVES < BM + BN ? 1 : 2; };
    const u32x4 xr = bounded_rsrc(a.x, xbytes);
    // Activation row of row `tid` of a tile (-1: none); they wait in LDS.
    const auto fetch_row = [&](const Tile& q) {
        const int l = again(tid);
        int x = l < BM && l < q.to - q.from ? (a.x_rows ? a.x_rows[q.from + l] : q.from + l) : -1;
        return x < a.x_rows_count ? x : -1;
    };
    const auto fetch_scales = [&](const Tile& q, float (&s)[SCALES]) {
#pragma unroll
        for (int i = 0; i < SCALES; ++i) {
            const int at = again(tid) + i * T;
            s[i] = __builtin_nanf("");  // no such activation row
            if (at < BM) {
                const int x = rows_of[at];
                if (x >= 0) s[i] = a.xs[x];
            } else if (at < ROWS) {
                const int64_t c = (int64_t)q.n0 + (at - BM) % BN;
                if (c < a.n) s[i] = (at < BM + BN ? a.ws : a.ws2)[(int64_t)q.e * a.n + c];
            }
        }
    };
    u32x4 wr, ur;
    const auto offsets = [&](const Tile& q, u32 (&off)[LOADS]) {
        const int64_t stack = (int64_t)q.e * a.n * a.k;
        wr = bounded_rsrc(a.w + stack, wbytes);
        ur = GLU ? bounded_rsrc(a.w2 + stack, wbytes) : wr;
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const int me = again(lane), l = lds_row(i) + (me >> 3), at_k = 16 * slot_of(l, me & 7);
            if (side(i) == 0) {
                const int x = rows_of[l];
                off[i] = x >= 0 ? (u32)x * (u32)a.k + (u32)at_k : xbytes;
            } else {
                const int64_t j = (int64_t)q.n0 + (l - BM) % BN;
                off[i] = j < a.n ? (u32)j * (u32)a.k + (u32)at_k : wbytes;
            }
        }
    };
    const auto load = [&](const u32 (&off)[LOADS], int st, int stage) {
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            // Behind K, and where there is no row, the load gives zeros.
            const u32 end = side(i) == 0 ? xbytes : wbytes;
            const bool there = st * BK + 16 * slot_of(lds_row(i) + (lane >> 3), lane & 7) < a.k && off[i] < end;
            load_to_lds(side(i) == 0 ? xr : side(i) == 1 ? wr : ur, there ? off[i] + (u32)(st * BK) : end,
                        lds_address(lds + stage * STAGE + lds_row(i) * BK));
        }
    };
    const auto keep_scales = [&](const float (&s)[SCALES], int which) {
#pragma unroll
        for (int i = 0; i < SCALES; ++i)
            if (tid + i * T < ROWS) scales[which * ROWS + tid + i * T] = s[i];
    };
    // (Waves of one row block on different SIMDs: where an expert has no rows for a
    // block, all four have less to do.)
    const int wm = wave / WN, wn = wave % WN;
    const int r = lane & 31, h = lane >> 5;
    struct Pieces {
        i32x4 w[S][NF], x[MF];
    };
    // Quarter kk (32 codes) of a stage.
    const auto read = [&](Pieces& f, int stage, int kk) {
        const unsigned char* from = lds + stage * STAGE;
#pragma unroll
        for (int j = 0; j < MF; ++j) {
            const int row = (wm * MF + j) * 32 + r;
            f.x[j] = *reinterpret_cast<const i32x4*>(from + row * BK + 16 * slot_of(row, 2 * kk + h));
        }
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
            for (int i = 0; i < NF; ++i) {
                const int row = BM + s * BN + (wn * NF + i) * 32 + r;
                f.w[s][i] = *reinterpret_cast<const i32x4*>(from + row * BK + 16 * slot_of(row, 2 * kk + h));
            }
    };

    using Sums = i32x16[S][NF][MF];
    const auto multiply = [](Sums& acc, const Pieces& f) {
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
            for (int i = 0; i < NF; ++i)
#pragma unroll
                for (int j = 0; j < MF; ++j)
                    acc[s][i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(f.w[s][i], f.x[j], acc[s][i][j], 0, 0, 0);
    };
    // Quarters of a stage: all but the last one's products.
    const auto quarters = [&](Sums& acc, Pieces& even, Pieces& odd, int stage) {
        read(odd, stage, 1);
        multiply(acc, even);
        read(even, stage, 2);
        multiply(acc, odd);
        read(odd, stage, 3);
        multiply(acc, even);
        __builtin_amdgcn_sched_barrier(0);
    };
    const auto put = [&](const Tile& q, const Sums& acc, int which, unsigned char* through) {
        unsigned char* const mine = through + wave * OUT;
        const float* const sx = scales + which * ROWS;
        const float* const sg = sx + BM + wn * NF * 32;
        if (a.y16)
            store_block<f16, NF, MF, GLU>(a, q, wm * MF * 32, (int64_t)q.n0 + wn * NF * 32, sx, sg, sg + BN, acc, mine);
        else
            store_block<float, NF, MF, GLU>(a, q, wm * MF * 32, (int64_t)q.n0 + wn * NF * 32, sx, sg, sg + BN, acc, mine);
    };

    Tile cur = nth(t);
    u32 off[LOADS];
    if constexpr (STAGES > 2) {
        float s[SCALES];
        const int x = fetch_row(cur);
        if (tid < BM) rows_of[tid] = x;
        __syncthreads();
        fetch_scales(cur, s);
        offsets(cur, off);
        for (int i = 0; i < STAGES; ++i) load(off, i, i);
        older_loads_barrier<(STAGES - 1) * LOADS>();
        Sums acc;
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
            for (int i = 0; i < NF; ++i)
#pragma unroll
                for (int j = 0; j < MF; ++j)
#pragma unroll
                    for (int v = 0; v < 16; ++v) acc[s][i][j][v] = 0;
        // Steps behind the last one are zeros that nothing reads.
        const auto turn = [](int stage) { return stage + 1 == STAGES ? 0 : stage + 1; };
        if (wm * MF * 32 < cur.to - cur.from) {
            Pieces even, odd;
            read(even, 0, 0);
            for (int st = 0, stage = 0; st < steps; ++st) {
                quarters(acc, even, odd, stage);
                older_loads_barrier<(STAGES - 2) * LOADS>();
                load(off, st + STAGES, stage);
                stage = turn(stage);
                read(even, stage, 0);
                multiply(acc, odd);
            }
        } else {
            for (int st = 0, stage = 0; st < steps; ++st) {
                older_loads_barrier<(STAGES - 2) * LOADS>();
                load(off, st + STAGES, stage);
                stage = turn(stage);
            }
        }
        keep_scales(s, 0);
        loads_barrier();
        put(cur, acc, 0, lds);
        return;
    }
    int stage = 0, which = 0;
    {
        float s[SCALES];
        const int x = fetch_row(cur);
        if (tid < BM) rows_of[tid] = x;
        __syncthreads();
        offsets(cur, off);
        load(off, 0, 0);
        fetch_scales(cur, s);
        keep_scales(s, 0);
    }
    loads_barrier();
    for (;;) {
        Sums acc;
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
            for (int i = 0; i < NF; ++i)
#pragma unroll
                for (int j = 0; j < MF; ++j)
#pragma unroll
                    for (int v = 0; v < 16; ++v) acc[s][i][j][v] = 0;
        const bool more = t + hop < count;
        Tile next{};
        int x = -1;
        float s[SCALES];
        if (more) {
            next = nth(t + hop);
            x = fetch_row(next);
            if (steps == 1) {
                if (tid < BM) rows_of[tid] = x;
                __syncthreads();
            }
        }
        // The next tile's first step.  (Not inside the loop: what it loads into
        // registers would be waited for on every turn, and the stages with it.)
        const auto bring_next = [&](int to) {
            if (!more) return;
            fetch_scales(next, s);
            offsets(next, off);
            load(off, 0, to);
        };
        if (steps > 1)
            load(off, 1, stage ^ 1);
        else
            bring_next(stage ^ 1);
        if (wm * MF * 32 < cur.to - cur.from) {
            Pieces even, odd;
            read(even, stage, 0);
            // Behind the barrier the other stage is there, and this one is read no more.
            for (int st = 0; st + 2 < steps; ++st) {
                quarters(acc, even, odd, stage);
                loads_barrier();
                load(off, st + 2, stage);
                stage ^= 1;
                read(even, stage, 0);
                multiply(acc, odd);
            }
            if (steps > 1) {
                quarters(acc, even, odd, stage);
                if (tid < BM) rows_of[tid] = x;
                loads_barrier();
                bring_next(stage);
                stage ^= 1;
                read(even, stage, 0);
                multiply(acc, odd);
            }
            quarters(acc, even, odd, stage);
            loads_barrier();
            stage ^= 1;
            multiply(acc, odd);
        } else {
            // A tile of fewer rows, none of which are this wave's: it only loads, in
            // step with the others.
            for (int st = 0; st + 2 < steps; ++st) {
                loads_barrier();
                load(off, st + 2, stage);
                stage ^= 1;
            }
            if (steps > 1) {
                if (tid < BM) rows_of[tid] = x;
                loads_barrier();
                bring_next(stage);
                stage ^= 1;
            }
            loads_barrier();
            stage ^= 1;
        }
        if (more) keep_scales(s, which ^ 1);
        put(cur, acc, which, lds + (stage ^ 1) * STAGE);
        if (!more) return;
        lds_barrier();  // before the next step's loads go where the sums passed
        cur = next;
        t += hop;
        which ^= 1;
    }
}

// Row tiles of `bm` that a launch needs at most: every expert's last one may be
// begun.
int64_t row_tiles(const GemmI8Args& a, int bm) {
    if (!a.offsets) return (a.rows + bm - 1) / bm;
    const int64_t begun = a.rows < a.experts ? a.rows : a.experts;
    return a.rows / bm + begun;
}
// Work-groups that a launch has at most where each has one tile (of up to 512
// threads, which a launch counts in 31 bits).
constexpr int64_t ONE_EACH = 0x3fffff;

template <int W, int NB, int MB, bool GLU>
hipError_t launch_rows(const GemmI8Args& a, hipStream_t st) {
    const int64_t grid = row_tiles(a, 16 * MB) * ((a.n + 16 * NB - 1) / (16 * NB));
    if (grid > 0x7fffffff / (64 * W)) return hipErrorInvalidConfiguration;
    rows_i8_kernel<W, NB, MB, GLU><<<dim3((unsigned)grid), dim3(64 * W), 0, st>>>(a);
    return hipGetLastError();
}

template <int WM, int WN, int MF, int NF, bool GLU, int OCC, int STAGES = 2>
hipError_t launch_tile(const GemmI8Args& a, hipStream_t st) {
    using Shape = TileShape<WM, WN, MF, NF, GLU, STAGES>;
    const int64_t tiles = row_tiles(a, Shape::BM) * ((a.n + Shape::BN - 1) / Shape::BN);
    if (tiles > (STAGES > 2 ? ONE_EACH : 0x3fffffff)) return hipErrorInvalidConfiguration;
    // As many work-groups as the device holds at once, or one for each tile; the
    // same for every die.
    int64_t grid = STAGES > 2 ? tiles : (int64_t)a.cus * std::max(1, 4 * OCC / Shape::WAVES) / 8 * 8;
    if (grid >= tiles) grid = (tiles + 7) / 8 * 8;
    if (grid < 8) grid = 8;
    tile_i8_kernel<WM, WN, MF, NF, GLU, OCC, STAGES><<<dim3((unsigned)grid), dim3(Shape::T), 0, st>>>(a);
    return hipGetLastError();
}

// What a launch of a tile kernel takes, in microseconds, fitted to timings of 176
// dense shapes (17 to 8192 rows, 1000 to 16384 columns of 512 to 8192 codes) and
// 320 grouped ones (8 to 128 experts): `begin` for a tile's ends (`grouped` once,
// where rows are looked for) and `one` for a step of 128 codes while every tile
// has a compute unit for itself; `full` for a step once all places are taken, and
// in proportion between; `last`, how much a round that is only begun costs beyond
// its share, and less after many uneven ones; `part`, what an expert's last tile,
// which lacks rows, costs beside a full one.  The kernel taken is within 1.1 % of
// the best on average, and within 10 % in 481 of the 496.
struct TileCost {
    int bm, bn, places;  // work-groups that a compute unit holds
    double begin, grouped, one, full, last, part;
};
// DEEP: a step in flight for each of several stages.
constexpr TileCost DEEP_64{64, 64, 2, 4.4, 1.1, 0.245, 0.45, 0.14, 0.83}, DEEP_128{128, 64, 1, 4.8, 0.5, 0.25, 0.35, 0.66, 0.66};
constexpr TileCost COST_64{64, 64, 3, 3.45, 1.6, 0.5, 0.76, 0.3, 0.8}, COST_128{128, 128, 2, 4.4, 1.0, 0.74, 1.05, 0.59, 0.71};
constexpr TileCost COST_256{256, 256, 1, 7.4, 0.0, 1.48, 1.77, 0.52, 0.6};
constexpr TileCost DEEP_64_GATED{64, 64, 1, 4.8, 1.2, 0.21, 0.5, 0.63, 0.66}, COST_64_GATED{64, 64, 2, 3.1, 1.9, 0.75, 0.87, 0.15, 1.2};
constexpr TileCost COST_128_GATED{128, 64, 2, 3.6, 2.0, 0.8, 1.11, 0.15, 1.0}, COST_256_GATED{256, 128, 1, 7.4, 1.9, 0.6, 1.55, 0.38, 0.83};

double tile_time(const GemmI8Args& a, const TileCost& c, double met, bool one_each = false) {
    if (one_each && row_tiles(a, c.bm) * ((a.n + c.bn - 1) / c.bn) > ONE_EACH) return HUGE_VAL;
    const double rt = a.offsets ? std::max(met, (double)a.rows / c.bm + met * c.part) : (double)((a.rows + c.bm - 1) / c.bm);
    const double alone = rt * (double)((a.n + c.bn - 1) / c.bn) / a.cus, rounds = alone / c.places;
    const double steps = (a.k + BK - 1) / BK, look = a.offsets ? c.grouped : 0.0;
    if (rounds >= 1.0) {
        const double more = c.last * (std::ceil(rounds) - rounds) / (a.offsets ? std::floor(rounds) : 1.0);
        return look + (rounds + more) * (c.begin + steps * c.full);
    }
    const double shared = c.places == 1 ? rounds : std::max(0.0, (alone - 1.0) / (c.places - 1));
    return look + c.begin + steps * (c.one + (c.full - c.one) * shared);
}

template <bool GLU>
hipError_t launch_few(const GemmI8Args& a, double per, hipStream_t st) {
    if (a.offsets) {
        // A row or a few for each expert: many work-groups, each with two waves
        // for up to 1024 codes (128 experts, one row each, 2048 columns of 768:
        // 26 us against 32 with four), four beyond (768 columns of 2048, gated: 39
        // against 41 with two).  A second block of rows pays from about six rows on.
        if (a.k <= 1024) return per <= 6 ? launch_rows<2, 1, 1, GLU>(a, st) : launch_rows<2, 1, 2, GLU>(a, st);
        return per <= 6 ? launch_rows<4, 1, 1, GLU>(a, st) : launch_rows<4, 1, 2, GLU>(a, st);
    }
    // One matrix: all its rows in one work-group (16 MB of them), so weights are
    // read once.  Eight waves share K, four where K is short or the columns
    // alone fill the device (16384 columns of 4096, one row: 12.8 us against
    // 14.9; 1024 of 8192: 9.8 against 7.2).  Twice the columns where that still fills it.
    const bool many = a.n >= 32 * (int64_t)a.cus;
    const bool short_k = a.k <= 2048 || a.n >= 64 * (int64_t)a.cus;
    if (a.rows <= 16) return short_k ? launch_rows<4, 1, 1, GLU>(a, st) : launch_rows<8, 1, 1, GLU>(a, st);
    if (a.rows <= 32) {
        if (many) return launch_rows<4, 2, 2, GLU>(a, st);
        return short_k ? launch_rows<4, 1, 2, GLU>(a, st) : launch_rows<8, 1, 2, GLU>(a, st);
    }
    if constexpr (!GLU) {
        if (a.rows <= 48) return many ? launch_rows<8, 2, 3, false>(a, st) : launch_rows<8, 1, 3, false>(a, st);
    }
    // Blocks of 32 rows, where columns alone would leave most of the device idle
    // (96 rows, 1024 columns of 8192: 13.5 us against 30 in tiles of 64).
    const int64_t blocks = (a.rows + 31) / 32;
    return blocks * a.n <= 32 * (int64_t)a.cus ? launch_rows<8, 1, 2, GLU>(a, st) : launch_rows<8, 2, 2, GLU>(a, st);
}

template <bool GLU>
hipError_t launch_plan(const GemmI8Args& a, hipStream_t st) {
    const double size = (double)a.n * a.k;
    if (a.offsets) {
        // A row or a few for each expert: bound by the weights' bytes, the kernel
        // without LDS stages, up to where tiles are as fast (128 experts, gated, 768
        // of 2048: 4 rows each 56 us against 62, 16 each 100 against 78), and for some
        // more where all of it is little (8 experts, 8 rows each, 512 of 1024: 5.2
        // against 6.8).
        const double per = (double)a.rows / a.experts, blocks = std::max((double)a.experts, a.rows / 32.0);
        if (per <= (GLU ? 9.0 : 6.0) || (per <= 32.0 && blocks * size <= 8 << 20)) {
            // (Tiles take what is more than one launch of it.)
            const hipError_t e = launch_few<GLU>(a, per, st);
            if (e != hipErrorInvalidConfiguration) return e;
        }
    }
    // Experts that have rows: all but those that chance leaves out.
    const double met = a.offsets ? a.experts * (1.0 - std::exp(-(double)a.rows / a.experts)) : 1.0;
    const double d64 = tile_time(a, GLU ? DEEP_64_GATED : DEEP_64, met, true);
    const double t64 = tile_time(a, GLU ? COST_64_GATED : COST_64, met);
    const double t128 = tile_time(a, GLU ? COST_128_GATED : COST_128, met);
    const double t256 = tile_time(a, GLU ? COST_256_GATED : COST_256, met);
    double best = std::min(std::min(d64, t64), std::min(t128, t256));
    if constexpr (!GLU) best = std::min(best, tile_time(a, DEEP_128, met, true));
    if (!a.offsets && a.rows <= 128) {
        // The kernel without stages, fitted to 33 to 128 rows; always for up to 16.
        // (64 rows, 2048 columns of 2048: 6.0 us against 8.1 in tiles; 4096 of 4096:
        // 14.1 against 12.1.)
        const double blocks = a.rows <= 48 ? 1.0 : (double)((a.rows + 31) / 32);
        if (a.rows <= 16 || 3.0 + 0.8 * a.k / 1024 + 0.2e-6 * blocks * size * (GLU ? 2 : 1) < best) {
            const hipError_t e = launch_few<GLU>(a, 0.0, st);
            if (e != hipErrorInvalidConfiguration) return e;
        }
    }
    if constexpr (GLU) {
        if (d64 == best) return launch_tile<2, 2, 1, 1, true, 1, 3>(a, st);
        if (t64 == best) return launch_tile<2, 2, 1, 1, true, 2>(a, st);
        return t128 == best ? launch_tile<4, 2, 1, 1, true, 4>(a, st) : launch_tile<4, 4, 2, 1, true, 4>(a, st);
    } else {
        if (d64 == best) return launch_tile<2, 2, 1, 1, false, 2, 4>(a, st);
        if (t64 == best) return launch_tile<2, 2, 1, 1, false, 3>(a, st);
        if (t128 == best) return launch_tile<2, 4, 2, 1, false, 4>(a, st);
        return t256 == best ? launch_tile<4, 4, 2, 2, false, 4>(a, st) : launch_tile<4, 2, 1, 1, false, 2, 3>(a, st);
    }
}

}  // namespace

hipError_t launch_gemm_i8(const GemmI8Args& given, hipStream_t st) {
    // Outputs that the 256 MB of memory-side cache would not keep for their reader
    // only push weights and activations out of it: they are written past the caches
    // (8192 x 16384 of 2048, fp16, 256 MiB: 285 -> 258 us).  With a kernel behind
    // that reads the output once: 256 MiB 368 -> 360 us, 192 MiB 273 -> 269 and
    // 264 -> 264, but 128 MiB 173 -> 182.
    GemmI8Args a = given;
    a.past_caches = a.rows * a.n * (a.y16 ? 2 : 4) >= (int64_t)192 << 20;
    return a.w2 ? launch_plan<true>(a, st) : launch_plan<false>(a, st);
}

}  // namespace qmm
