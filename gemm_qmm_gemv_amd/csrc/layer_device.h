// layer_device.h -- sums, minima and maxima over the lanes of a wave without
// LDS: the data-parallel primitives of a row of 16 lanes, and on gfx950 the
// swaps of rows and halves; addresses in LDS and
// loads that go there directly.
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

// 16 bytes per lane from memory to LDS without passing through registers: lane
// i's land at `to` + 16 i.  An instruction of its own text, because the
// compiler waits for all loads before any later LDS read if it knows that
// this one writes LDS; here readers do, before the barrier they share.  m0
// holds the LDS address.  Scalar registers that a vector instruction wrote may
// be read by a memory instruction five wait states later, which the compiler
// sees to for its own instructions only: s_mov and s_nop make up five (the
// same times as with the one that m0 needs).  There is no register for the
// load to write, and the address registers are read when it is issued.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"  // m0 is a reserved register
__device__ __forceinline__ void load_to_lds(u32x4 rsrc, u32 offset, u32 to) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 3\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds"
                 :
                 : "v"(offset), "s"(rsrc), "s"(to)
                 : "memory", "m0");
}
#pragma clang diagnostic pop

__device__ __forceinline__ float add_f32(float a, float b) { return a + b; }

}  // namespace qmm
