// layer_device.h -- sums, minima and maxima over the lanes of a wave without
// LDS: the data-parallel primitives of a row of 16 lanes, and on gfx950 the
// swaps of rows and halves; addresses in LDS.
#pragma once

#include "qmm_device.h"

namespace qmm {

template <int CTRL>
__device__ __forceinline__ float dpp_move(float v) {
    const int x = __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true);
    return __builtin_bit_cast(float, x);
}

// f over the N lanes (2 to 64, a power of two) that share lane / N; every lane
// gets it.  Each stage combines what the stages before made equal in groups of
// 1, 2, 4, ... lanes, so a mirror serves as well as an exclusive or.
template <int N, class F>
__device__ __forceinline__ float over_lanes(float v, F f) {
    if constexpr (N >= 2) v = f(v, dpp_move<0xB1>(v));   // quad_perm [1, 0, 3, 2]
    if constexpr (N >= 4) v = f(v, dpp_move<0x4E>(v));   // quad_perm [2, 3, 0, 1]
    if constexpr (N >= 8) v = f(v, dpp_move<0x141>(v));  // row_half_mirror
    if constexpr (N >= 16) v = f(v, dpp_move<0x140>(v)); // row_mirror
    // With the same value in both operands a swap leaves every other row (or
    // one half) twice in each result.
    if constexpr (N >= 32) {
        const u32 x = __builtin_bit_cast(u32, v);
        const auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
        const u32 a = r[0], b = r[1];
        v = f(__builtin_bit_cast(float, a), __builtin_bit_cast(float, b));
    }
    if constexpr (N >= 64) {
        const u32 x = __builtin_bit_cast(u32, v);
        const auto r = __builtin_amdgcn_permlane32_swap(x, x, false, false);
        const u32 a = r[0], b = r[1];
        v = f(__builtin_bit_cast(float, a), __builtin_bit_cast(float, b));
    }
    return v;
}

// f over lanes l, l ^ 16, l ^ 32 and l ^ 48.
template <class F>
__device__ __forceinline__ float over_rows(float v, F f) {
    const u32 x = __builtin_bit_cast(u32, v);
    const auto r = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    const u32 a = r[0], b = r[1];
    const u32 y = __builtin_bit_cast(u32, f(__builtin_bit_cast(float, a), __builtin_bit_cast(float, b)));
    const auto q = __builtin_amdgcn_permlane16_swap(y, y, false, false);
    const u32 c = q[0], d = q[1];
    return f(__builtin_bit_cast(float, c), __builtin_bit_cast(float, d));
}

// f over lanes l and l ^ 32.
template <class F>
__device__ __forceinline__ float over_halves(float v, F f) {
    const u32 x = __builtin_bit_cast(u32, v);
    const auto r = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    const u32 a = r[0], b = r[1];
    return f(__builtin_bit_cast(float, a), __builtin_bit_cast(float, b));
}

// Where in LDS p points, as the direct loads take it.
__device__ __forceinline__ u32 lds_address(const void* p) {
    return (u32)(size_t)(const __attribute__((address_space(3))) char*)p;
}

__device__ __forceinline__ float add_f32(float a, float b) { return a + b; }

}  // namespace qmm
