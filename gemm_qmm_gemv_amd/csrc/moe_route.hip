// moe_route.hip -- a token's scores for the experts to its experts, their
// weights, and the rows grouped by expert that the experts' products take:
//   s = softmax(l) or sigmoid(l),  c = s + bias,
//   the top_groups groups of highest score stay (a group's score: the sum of
//   its group_best highest c), of their experts the top_k of highest c,
//   w = s[chosen] [/ sum over the chosen] * scale,
// in fp32 from the logits of the chosen, then a counting sort of the (token,
// expert) pairs by expert, within an expert by token.
//
// A choice hangs on the last bits of its scores, so it is made on numbers that
// never run together: without a bias the order of the scores is that of the
// logits, which are compared as they are; with one, and for groups by the sum of
// two, on scores in fp32 where they lie far enough apart for that, else in 64
// bits.  Keys are whole numbers in the order of the values, so that a place that
// is taken (or not there) has a key below all of them.
//
// Short batches are one chain of waits and lane moves: one token of 128 experts
// 4.2 us (an empty launch: 1.6), 37 of 256 in groups with a bias 7.8 and 4.6
// for the placing; a choice left open costs such a call 5 us more.  Long ones
// are bound by vector instructions (16384 tokens of 128: 10.2 us at 73 % busy,
// 256 in groups with a bias 41 us at 87 %; 262144 of 128: 134 us, 82 %); the
// placing waits for memory and LDS (7.6 us; for the longest 39, and 9 for the
// sums that it reads).
#include <algorithm>
#include <type_traits>

#include "layer_device.h"
#include "moe_kernels.h"

namespace qmm {
namespace {

constexpr float INF = __builtin_huge_valf();
// Tokens that one work-group routes and places in one launch: what it holds at
// once, with a wave or 16 lanes for each.
constexpr int ROUTE_ONE = 16, ROUTE_ONE_16 = 64;
// Up to this many tokens get a wave each.
constexpr int ROUTE_WAVES = 4096;
// Tokens that one work-group places.
constexpr int PLACE = 64;
// Rows of counts that are summed up for the second launch, if there are more
// than CHUNKED.
constexpr int CHUNK = 64, CHUNKED = 256;
// Up to this many of those sums, over chunks and experts, are added up by every
// work-group that places; more are made running ones in a launch of their own, so
// that a token costs the same however many there are (65536 tokens of 128 experts,
// 2048 sums: 54.7 us either way, of 256 84.6 -> 82.9; 2^20 of 1024: 5432 -> 3203).
constexpr int RUNNING = 2048;

__device__ __forceinline__ int order_key(float v) {
    const int b = __builtin_bit_cast(int, v + 0.f);  // -0 is 0
    return b ^ ((b >> 31) & 0x7fffffff);
}
__device__ __forceinline__ int64_t order_key(double v) {
    const int64_t b = __builtin_bit_cast(int64_t, v + 0.0);
    return b ^ ((b >> 63) & 0x7fffffffffffffffLL);
}
__device__ __forceinline__ float key_value(int k) { return __builtin_bit_cast(float, k ^ ((k >> 31) & 0x7fffffff)); }
template <class K>
__device__ constexpr K taken() {
    return sizeof(K) == 4 ? (K)0x80000000u : (K)0x8000000000000000ull;
}

// f over the N lanes that share lane / N, for values of 4 or 8 bytes.
template <int CTRL, class V>
__device__ __forceinline__ V lane_move(V v) {
    if constexpr (sizeof(V) == 4) {
        return __builtin_bit_cast(V, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
    } else {
        const u32x2 x = __builtin_bit_cast(u32x2, v);
        u32x2 r;
        r[0] = (u32)__builtin_amdgcn_mov_dpp((int)x[0], CTRL, 0xF, 0xF, true);
        r[1] = (u32)__builtin_amdgcn_mov_dpp((int)x[1], CTRL, 0xF, 0xF, true);
        return __builtin_bit_cast(V, r);
    }
}
// f of v in lanes l and l ^ 16 (HALVES: l ^ 32), in both.
template <bool HALVES, class V, class F>
__device__ __forceinline__ V across(V v, F f) {
    const auto swap = [](u32 x) {
        if constexpr (HALVES)
            return __builtin_amdgcn_permlane32_swap(x, x, false, false);
        else
            return __builtin_amdgcn_permlane16_swap(x, x, false, false);
    };
    if constexpr (sizeof(V) == 4) {
        const auto r = swap(__builtin_bit_cast(u32, v));
        const u32 a = r[0], b = r[1];
        return f(__builtin_bit_cast(V, a), __builtin_bit_cast(V, b));
    } else {
        const u32x2 x = __builtin_bit_cast(u32x2, v);
        const auto lo = swap(x[0]), hi = swap(x[1]);
        const u32x2 a = {(u32)lo[0], (u32)hi[0]}, b = {(u32)lo[1], (u32)hi[1]};
        return f(__builtin_bit_cast(V, a), __builtin_bit_cast(V, b));
    }
}
template <int N, class V, class F>
__device__ __forceinline__ V lanes(V v, F f) {
    static_assert(N == 16 || N == 64, "lanes of a token");
    v = f(v, lane_move<0xB1>(v));
    v = f(v, lane_move<0x4E>(v));
    v = f(v, lane_move<0x141>(v));
    v = f(v, lane_move<0x140>(v));
    if constexpr (N == 64) {
        v = across<false>(v, f);
        v = across<true>(v, f);
    }
    return v;
}
// v of the first lane for which `here` holds; none: `other`.  Lanes hold what
// lies behind each other, so the first is the lowest index.
template <int N, class V>
__device__ __forceinline__ V first_of(bool here, V v, V other) {
    static_assert(sizeof(V) == 4, "one register");
    if constexpr (N == 64) {
        const uint64_t who = __ballot(here);
        if (who == 0) return other;
        return __builtin_bit_cast(V, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), __ffsll((unsigned long long)who) - 1));
    } else {
        const u32 who = (u32)(__ballot(here) >> (threadIdx.x & 48)) & 0xffffu;
        const int from = (int)(threadIdx.x & 48) + __ffs(who) - 1;
        const int r = __builtin_amdgcn_ds_bpermute(4 * from, __builtin_bit_cast(int, v));
        return who ? __builtin_bit_cast(V, r) : other;
    }
}
struct Max {
    template <class V>
    __device__ V operator()(V a, V b) const { return a > b ? a : b; }
};
struct Min {
    template <class V>
    __device__ V operator()(V a, V b) const { return a < b ? a : b; }
};
struct Add {
    template <class V>
    __device__ V operator()(V a, V b) const { return a + b; }
};

// Logits e0 .. e0 + PER - 1 of a token, -inf behind the last expert.
template <int PER>
__device__ __forceinline__ void load_logits(const RouteArgs& a, int64_t token, int e0, float (&l)[PER]) {
#pragma unroll
    for (int i = 0; i < PER; ++i) l[i] = -INF;
    const auto take_from = [&](auto p) {
        if (a.vec && PER % 4 == 0) {
            typedef std::remove_cv_t<std::remove_reference_t<decltype(*p)>> F;
            typedef F vec __attribute__((ext_vector_type(4)));
#pragma unroll
            for (int i = 0; i < PER / 4 * 4; i += 4) {
                if (e0 + i >= a.experts) continue;  // their number is a multiple of 4
                const vec v = *reinterpret_cast<const vec*>(p + e0 + i);
#pragma unroll
                for (int j = 0; j < 4; ++j) l[i + j] = (float)v[j];
            }
        } else {
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (e0 + i < a.experts) l[i] = (float)p[e0 + i];
        }
    };
    if (a.f16)
        take_from(static_cast<const f16*>(a.logits) + token * a.stride);
    else
        take_from(static_cast<const float*>(a.logits) + token * a.stride);
}

// What one token's lanes know after its choice: lane j < top_k holds expert and
// weight of choice j.
struct Chosen {
    int id;
    float w;
};

// Whether two scores in fp32 (with a bias) are so far apart that those in 64 bits
// are in the same order: `near`, what the scores themselves may be off by, and
// 2^-24 of their size for the bias, and twice as much.
__device__ __forceinline__ bool apart(float high, float low, float near) {
    return high - low > near + 0x1p-22f * (fabsf(high) + fabsf(low));
}

// Between what a group's score in fp32 may lie in 64 bits: `near` for the scores
// in it, and for biases and their sum 2^-23 of the terms' size, which may be far
// above the sum's where they cancel, and twice as much.  `lowest`: the lowest
// term; -inf (a bias, or a NaN placed so) is that in 64 bits, too.
struct Range {
    float lo, hi;
};
__device__ __forceinline__ Range range_of(float score, float size, float lowest, float near) {
    if (lowest == -INF) return {-INF, -INF};
    const float off = near + 0x1p-22f * size;
    return off < INF ? Range{score - off, score + off} : Range{-INF, INF};
}

// Of the lanes' groups of keys the `count` highest, the lower index first among
// equals: lane j gets the index and the key of choice j.  Returns whether every
// key chosen is apart from the next (the first left out included), if asked.
template <int L, int PER, bool APART, class Key>
__device__ __forceinline__ bool take(Key (&key)[PER], int e0, int lane, int count, int& id, Key& value, float near = 0.f) {
    bool clear = true;
    float before = 0.f;
    for (int j = 0; j < count + (APART ? 1 : 0); ++j) {
        Key m = key[0];
#pragma unroll
        for (int i = 1; i < PER; ++i) m = key[i] > m ? key[i] : m;
        const Key best = lanes<L>(m, Max{});
        if constexpr (APART) {
            if (best != taken<Key>()) {
                const float v = key_value(best);
                if (j > 0) clear = clear && apart(before, v, near);
                before = v;
            }
            if (j == count) break;
        }
        int at = e0;
#pragma unroll
        for (int i = PER - 1; i > 0; --i)
            if (key[i] == best) at = e0 + i;
        if (key[0] == best) at = e0;
        const int e = first_of<L>(m == best, at, 0);
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (e - e0 == i) key[i] = taken<Key>();
        if (lane == j) {
            id = e;
            value = best;
        }
    }
    return clear;
}

// The two highest of v's values among this lane's, then among the lanes' that
// share a group.
struct TwoBest {
    template <class V>
    __device__ static void add(V& x, V& y, V a) {
        const V low = a < x ? a : x;
        y = y > low ? y : low;
        x = x > a ? x : a;
    }
};
template <int CTRL, class V>
__device__ __forceinline__ void join_two(V& x, V& y) {
    const V a = lane_move<CTRL>(x), b = lane_move<CTRL>(y);
    TwoBest::add(x, y, a);
    y = y > b ? y : b;
}

// Keys of experts outside the top_groups best groups become taken.  s: what is
// summed, if two are.  Returns whether every group that stays is above every other
// in 64 bits, too, if asked.
template <int L, int PER, bool APART, class Key, class V>
__device__ __forceinline__ bool keep_groups(const RouteArgs& a, Key (&key)[PER], const V (&s)[PER], int e0, int lane, float near = 0.f) {
    const int each = a.experts / a.groups;
    const V low = -(V)INF;
    Range range{0.f, 0.f};  // of that score, if asked
    using Mark = std::conditional_t<sizeof(Key) == 4 && sizeof(V) == 4, int, int64_t>;
    Mark mine = taken<Mark>();  // the score of the lane's group, in the first lane of it
    int group = lane;
    const int wide = each / PER;  // lanes of a group
    if (each % PER == 0 && wide <= 8 && (wide & (wide - 1)) == 0) {
        // Every lane's experts are of one group: all groups at once.
        group = e0 / each;
        if (a.group_best == 1) {
            Key k = key[0];
#pragma unroll
            for (int i = 1; i < PER; ++i) k = key[i] > k ? key[i] : k;
            if (wide >= 2) k = Max{}(k, lane_move<0xB1>(k));
            if (wide >= 4) k = Max{}(k, lane_move<0x4E>(k));
            if (wide >= 8) k = Max{}(k, lane_move<0x141>(k));
            mine = k;
            if constexpr (APART) range = range_of(key_value(k), fabsf(key_value(k)), key_value(k), 0.5f * near);
        } else {
            V x = low, y = low;
#pragma unroll
            for (int i = 0; i < PER; ++i) TwoBest::add(x, y, s[i]);
            if (wide >= 2) join_two<0xB1>(x, y);
            if (wide >= 4) join_two<0x4E>(x, y);
            if (wide >= 8) join_two<0x141>(x, y);
            V sum = x + y;
            if (sum != sum) sum = low;
            mine = order_key(sum);
            if constexpr (APART) range = range_of(sum, fabsf(x) + fabsf(y), y, near);
        }
        if (lane % wide != 0 || e0 >= a.experts) mine = taken<Mark>();
    } else {
        // One group after the other, over all lanes.
        for (int g = 0; g < a.groups; ++g) {
            const int lo = g * each, hi = lo + each;
            if (a.group_best == 1) {
                Key k = taken<Key>();
#pragma unroll
                for (int i = 0; i < PER; ++i)
                    if (e0 + i >= lo && e0 + i < hi && key[i] > k) k = key[i];
                k = lanes<L>(k, Max{});
                if (lane == g) {
                    mine = k;
                    if constexpr (APART) range = range_of(key_value(k), fabsf(key_value(k)), key_value(k), 0.5f * near);
                }
            } else {
                V x = low, y = low;
#pragma unroll
                for (int i = 0; i < PER; ++i)
                    if (e0 + i >= lo && e0 + i < hi) TwoBest::add(x, y, s[i]);
                const V first = lanes<L>(x, Max{});
                const int owner = first_of<L>(x == first, lane, L);
                const V second = lanes<L>(lane == owner ? y : x, Max{});
                V sum = first + second;
                if (sum != sum) sum = low;
                if (lane == g) {
                    mine = order_key(sum);
                    if constexpr (APART) range = range_of(sum, fabsf(first) + fabsf(second), second, near);
                }
            }
        }
    }
    // One bit for each group that stays.
    uint64_t stay = 0;
    const bool has = mine != taken<Mark>();
    for (int j = 0; j < a.top_groups; ++j) {
        const Mark m = lanes<L>(mine, Max{});
        const int owner = first_of<L>(mine == m, lane, 0), g = first_of<L>(mine == m, group, 0);
        stay |= 1ull << g;
        if (lane == owner) mine = taken<Mark>();
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = e0 + i;
        if (e < a.experts && !(stay >> (e / each) & 1)) key[i] = taken<Key>();
    }
    if constexpr (APART) {
        if (a.top_groups == a.groups) return true;
        // (The order among those that stay is of no account.  One whose score is far
        // from the border may be uncertain by more than one that is next to it.)
        const bool out = mine != taken<Mark>(), in = has && !out;
        const float lowest = lanes<L>(in ? range.lo : INF, Min{}), highest = lanes<L>(out ? range.hi : -INF, Max{});
        return near < INF && lowest > highest;  // near: NaN where the scores are
    }
    return true;
}

// The choice on scores in 64 bits.
template <int L, int PER, bool BIAS>
__device__ __forceinline__ int choose_exact(const RouteArgs& a, int64_t token, float top, int lane) {
    const int e0 = lane * PER;
    float l[PER];
    load_logits<PER>(a, token, e0, l);
#pragma unroll
    for (int i = 0; i < PER; ++i)
        if (l[i] != l[i]) l[i] = -INF;
    double s[PER];
    if (a.sigmoid) {
#pragma unroll
        for (int i = 0; i < PER; ++i) s[i] = 1.0 / (1.0 + exp(-(double)l[i]));
    } else {
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            s[i] = top == -INF ? 0.0 : l[i] == top ? 1.0 : exp((double)l[i] - (double)top);  // top may be +inf
            sum += s[i];
        }
        sum = lanes<L>(sum, Add{});
        const double r = sum > 0.0 ? 1.0 / sum : 0.0;
#pragma unroll
        for (int i = 0; i < PER; ++i) s[i] *= r;
    }
    int id = -1;
    if constexpr (BIAS) {
        int64_t key[PER], best = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            if (e0 + i < a.experts) s[i] += (double)a.bias[e0 + i];
            if (s[i] != s[i] || e0 + i >= a.experts) s[i] = -(double)INF;
            key[i] = e0 + i < a.experts ? order_key(s[i]) : taken<int64_t>();
        }
        if (a.groups > 1) keep_groups<L, PER, false>(a, key, s, e0, lane);
        take<L, PER, false>(key, e0, lane, a.top_k, id, best);
    } else {
        int key[PER], best = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            key[i] = e0 + i < a.experts ? order_key(l[i]) : taken<int>();
            if (e0 + i >= a.experts) s[i] = -(double)INF;
        }
        if (a.groups > 1) keep_groups<L, PER, false>(a, key, s, e0, lane);
        take<L, PER, false>(key, e0, lane, a.top_k, id, best);
    }
    return id;
}

// What a choice is made on.
enum Mode {
    LOGITS,  // the logits: their order is the scores'
    PAIRS,   // the same, in groups by the sum of their two best scores
    BIASED,  // scores and biases
};

// L lanes share a token; lane i of them holds experts i PER .. i PER + PER - 1.
template <int L, int PER, Mode MODE>
__device__ __forceinline__ Chosen choose(const RouteArgs& a, int64_t token, int lane) {
    const int e0 = lane * PER;
    float l[PER];
    load_logits<PER>(a, token, e0, l);
    // A NaN is placed as -inf and makes the token's weights NaN.
    int bad = 0;
    float top = -INF;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        if (l[i] != l[i]) {
            bad = 1;
            l[i] = -INF;
        }
        top = fmaxf(top, l[i]);
    }
    bad = lanes<L>(bad, Max{});
    top = lanes<L>(top, Max{});
    if (!a.sigmoid && top == INF) bad = 1;
    const bool empty = top == -INF;  // every score is zero

    constexpr bool BIAS = MODE == BIASED;
    int key[PER], best = 0;
    Chosen c{-1, 0.f};
    float sum_all = 0.f;
    if constexpr (MODE == LOGITS) {
#pragma unroll
        for (int i = 0; i < PER; ++i) key[i] = e0 + i < a.experts ? order_key(l[i]) : taken<int>();
        if (a.groups > 1) keep_groups<L, PER, false>(a, key, l, e0, lane);
        take<L, PER, false>(key, e0, lane, a.top_k, c.id, best);
    } else {
        // In fp32 first; where that leaves a choice open, in 64 bits.  A sigmoid
        // is good to 2^-22 (exponential and quotient), a softmax score p to 2^-19
        // p (and at most 22 additions); near is that of two, and twice as much.
        float s[PER], near = 0x1p-20f;
        if (a.sigmoid) {
#pragma unroll
            for (int i = 0; i < PER; ++i) s[i] = 1.f / (1.f + expf(-l[i]));
        } else {
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                s[i] = empty ? 0.f : expf(l[i] - top);
                sum += s[i];
            }
            sum_all = lanes<L>(sum, Add{});
            const float r = empty ? 0.f : 1.f / sum_all;
            near = 0x1p-17f * r;  // r is the largest score
#pragma unroll
            for (int i = 0; i < PER; ++i) s[i] *= r;
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            if constexpr (BIAS) {
                if (e0 + i < a.experts) s[i] += a.bias[e0 + i];
                if (s[i] != s[i]) s[i] = -INF;
                key[i] = order_key(s[i]);
            } else {
                key[i] = order_key(l[i]);
            }
            if (e0 + i >= a.experts) {
                s[i] = -INF;
                key[i] = taken<int>();
            }
        }
        bool clear = true;
        if (a.groups > 1) clear = keep_groups<L, PER, true>(a, key, s, e0, lane, near);
        clear = take<L, PER, BIAS>(key, e0, lane, a.top_k, c.id, best, near) && clear;
        if (__any(!clear)) {
            const int id = choose_exact<L, PER, BIAS>(a, token, top, lane);
            if (!clear) c.id = id;
        }
    }
    float chosen_l = -INF;
    if (lane < a.top_k) {
        const int64_t at = token * a.stride + c.id;
        chosen_l = a.f16 ? (float)static_cast<const f16*>(a.logits)[at] : static_cast<const float*>(a.logits)[at];
        if (chosen_l != chosen_l) chosen_l = -INF;
    }
    // Weights from the logits of the chosen, in fp32.
    float w = 0.f;
    if (a.sigmoid) {
        // Below 0 as e^l / (1 + e^l); where only ratios count, times what brings
        // the largest into range.
        float shift = 0.f;
        if (a.renorm) {
            shift = fminf(lanes<L>(lane < a.top_k ? chosen_l : -INF, Max{}), 0.f);
            if (shift == -INF) shift = 0.f;
        }
        if (lane < a.top_k)
            w = chosen_l > 0.f ? 1.f / (1.f + expf(-chosen_l)) : expf(chosen_l - shift) / (1.f + expf(chosen_l));
        if (a.renorm) {
            const float sum = lanes<L>(w, Add{});
            w = sum > 0.f ? w / sum : 0.f;
        }
    } else if (!empty) {
        // Where only ratios count, from the largest of the chosen.
        float from = top, sum;
        if (a.renorm) {
            from = lanes<L>(lane < a.top_k ? chosen_l : -INF, Max{});
            if (from == -INF) from = top;
        }
        if (lane < a.top_k) w = expf(chosen_l - from);
        if (a.renorm) {
            sum = lanes<L>(w, Add{});
        } else if constexpr (MODE != LOGITS) {
            sum = sum_all;
        } else {
            sum = 0.f;
#pragma unroll
            for (int i = 0; i < PER; ++i) sum += expf(l[i] - top);
            sum = lanes<L>(sum, Add{});
        }
        w = sum > 0.f ? w / sum : 0.f;
    }
    c.w = bad ? __builtin_nanf("") : w * a.scale;
    return c;
}

// Sums over the experts before, T of them at a time, in all threads of a
// work-group: to(e, sum before, own) for each expert, the sum of all returned.
template <class N, class To>
__device__ __forceinline__ int sums_before(int experts, int* part, N own, To to) {
    const int tid = threadIdx.x, threads = blockDim.x;
    int base = 0;
    for (int e0 = 0; e0 < experts; e0 += threads) {
        const int e = e0 + tid, n = e < experts ? own(e) : 0;
        int sum = n;
        for (int d = 1; d < 64; d *= 2) {
            const int before = __shfl_up(sum, d, 64);
            if ((tid & 63) >= d) sum += before;
        }
        if ((tid & 63) == 63) part[tid >> 6] = sum;
        __syncthreads();
        int before = base;
        for (int i = 0; i < threads / 64; ++i) {
            if (i < tid >> 6) before += part[i];
            base += part[i];
        }
        if (e < experts) to(e, before + sum - n, n);
        __syncthreads();
    }
    return base;
}

// Tokens of one work-group: few, so that waves do not wait for each other's
// instructions (37 tokens of 256 experts in groups: 12.6 us with 4, 13.3 with 8,
// 15.7 with 16; 4097 of 256: 18.4 with 32, 25.9 with 64), but no more than 256
// work-groups, as the second launch reads all rows of counts in each of its own
// (16384 tokens of 128: 17.3 us with 64, 21.9 with 16).
int block_tokens(int64_t tokens) {
    int block = 4;
    while (block < PLACE && (tokens + block - 1) / block > CHUNKED) block *= 2;
    return block;
}

// A work-group takes `block` tokens, blockDim / L of them at a time (ONE: it is
// the only one).  Ranks within an expert come from a mask per expert with a bit
// for each token: a token names an expert at most once.
template <int L, int PER, Mode MODE, bool ONE>
__global__ void __launch_bounds__(1024) route_kernel(RouteArgs a, int block) {
    extern __shared__ uint64_t mask[];  // [experts]; ONE: ids and weights of the pairs, offsets
    __shared__ int part[16];
    const int tid = threadIdx.x, threads = blockDim.x, lane = tid % L;
    int* const lds_id = reinterpret_cast<int*>(mask + a.experts);
    float* const lds_w = reinterpret_cast<float*>(lds_id + block * a.top_k);
    const int64_t first = (int64_t)blockIdx.x * block;
    const int here = (int)(a.tokens - first < block ? a.tokens - first : block);
    for (int e = tid; e < a.experts; e += threads) mask[e] = 0;
    __syncthreads();
    for (int t0 = 0; t0 < here; t0 += threads / L) {
        const int t = t0 + tid / L;
        if (L == 64 && t >= here) break;  // a whole wave
        const int64_t token = first + (t < here ? t : 0);
        Chosen c = choose<L, PER, MODE>(a, token, lane);
        if (t < here && lane < a.top_k) {
            if (a.keep && !a.keep[token]) c = Chosen{-1, 0.f};
            const int64_t pair = token * a.top_k + lane;
            a.ids[pair] = c.id;
            a.weights[pair] = c.w;
            if (ONE) {
                lds_id[t * a.top_k + lane] = c.id;
                lds_w[t * a.top_k + lane] = c.w;
            }
            if (c.id >= 0) atomicOr(reinterpret_cast<unsigned long long*>(mask + c.id), 1ull << t);
        }
    }
    if (!a.offsets) return;
    __syncthreads();
    if constexpr (ONE) {
        int* const off = reinterpret_cast<int*>(lds_w + block * a.top_k);
        const int all = sums_before(a.experts, part, [&](int e) { return (int)__popcll(mask[e]); },
                                    [&](int e, int before, int) {
                                        off[e] = before;
                                        a.offsets[e] = before;
                                    });
        if (tid == 0) a.offsets[a.experts] = all;
        for (int p = tid; p < here * a.top_k; p += threads) {
            const int e = lds_id[p], t = p / a.top_k;
            const int row = e < 0 ? -1 : off[e] + (int)__popcll(mask[e] & ((1ull << t) - 1));
            if (a.pair_row) a.pair_row[p] = row;
            if (row < 0) continue;
            if (a.pair_token) a.pair_token[row] = t;
            if (a.pair_weight) a.pair_weight[row] = lds_w[p];
        }
    } else {
        const int width = (a.experts + 15) & ~15;
        uint8_t* const counts = a.counts + (int64_t)blockIdx.x * width;
        for (int e = 4 * tid; e < width; e += 4 * threads) {
            u32 n = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (e + j < a.experts) n |= (u32)__popcll(mask[e + j]) << (8 * j);
            *reinterpret_cast<u32*>(counts + e) = n;
        }
    }
}

// Sums of CHUNK rows of counts, for every expert: 16 experts a thread, rows of
// them side by side.
__global__ void __launch_bounds__(256) route_sums_kernel(const uint8_t* counts, u32* sums, int width, int blocks) {
    extern __shared__ u32 all_of[];  // [width]
    const int tid = threadIdx.x, pieces = width / 16, side = 256 / pieces;
    const int row0 = (int)blockIdx.x * CHUNK, rows = blocks - row0 < CHUNK ? blocks - row0 : CHUNK;
    for (int e = tid; e < width; e += 256) all_of[e] = 0;
    __syncthreads();
    if (tid / pieces < side) {
        const int piece = tid % pieces;
        const u32x4* const p = reinterpret_cast<const u32x4*>(counts) + (int64_t)row0 * pieces + piece;
        for (int b = tid / pieces; b < rows; b += side) {
            const u32x4 v = p[(int64_t)b * pieces];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const u32 n = v[j / 4] >> (8 * (j % 4)) & 255u;
                if (n) atomicAdd(all_of + 16 * piece + j, n);
            }
        }
    }
    __syncthreads();
    for (int e = tid; e < width; e += 256) sums[(int64_t)blockIdx.x * width + e] = all_of[e];
}

// Those sums to running ones, each chunk's own included: a work-group for 64
// experts, a lane each, its 16 waves one behind the other along the chunks.
__global__ void __launch_bounds__(1024) route_running_kernel(u32* sums, int width, int chunks) {
    __shared__ u32 part[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, e = (int)blockIdx.x * 64 + lane;
    const int per = (chunks + 15) / 16, from = wave * per, to = from + per < chunks ? from + per : chunks;
    u32* const p = sums + e;
    u32 sum = 0;
    if (e < width) {
#pragma unroll 8
        for (int c = from; c < to; ++c) sum += p[(int64_t)c * width];
    }
    part[wave][lane] = sum;
    __syncthreads();
    if (e >= width) return;
    sum = 0;
    for (int w = 0; w < wave; ++w) sum += part[w][lane];
#pragma unroll 8
    for (int c = from; c < to; ++c) {
        sum += p[(int64_t)c * width];
        p[(int64_t)c * width] = sum;
    }
}

// Last launch where several work-groups routed: each takes PLACE tokens, adds up
// what the experts got before, and places its pairs.  Counts (`blocks` rows, of
// `block` tokens each) are read 16 experts a thread, rows of them side by side;
// where there are sums of CHUNK rows, those (where they are running ones, of the
// chunk before, the own and the last) and the rows of the own chunk.
__global__ void __launch_bounds__(256) route_place_kernel(RouteArgs a, int block, int blocks, const u32* sums, bool running) {
    extern __shared__ uint64_t mask[];  // [experts], then [2][width]: rows before this work-group, all rows
    __shared__ int part[4];
    const int tid = threadIdx.x, width = (a.experts + 15) & ~15, mine = blockIdx.x * (PLACE / block);
    int* const before = reinterpret_cast<int*>(mask + a.experts);
    int* const all = before + width;
    const int64_t first = (int64_t)blockIdx.x * PLACE;
    const int here = (int)(a.tokens - first < PLACE ? a.tokens - first : PLACE);
    const int pairs = here * a.top_k;
    for (int e = tid; e < a.experts; e += 256) mask[e] = 0;
    for (int e = tid; e < 2 * width; e += 256) before[e] = 0;
    __syncthreads();
    const int32_t* const ids = a.ids + first * a.top_k;
    for (int p = tid; p < pairs; p += 256) {
        const int e = ids[p];
        if (e >= 0) atomicOr(reinterpret_cast<unsigned long long*>(mask + e), 1ull << (p / a.top_k));
    }
    int from = 0, to = blocks;
    if (sums) {
        const int own = mine / CHUNK, chunks = (blocks + CHUNK - 1) / CHUNK;
        from = own * CHUNK;
        to = from + CHUNK < blocks ? from + CHUNK : blocks;
        for (int e = tid; running && e < width; e += 256) {
            const u32 n = own > 0 ? sums[(int64_t)(own - 1) * width + e] : 0;
            atomicAdd(before + e, (int)n);
            atomicAdd(all + e, (int)(sums[(int64_t)(chunks - 1) * width + e] - (sums[(int64_t)own * width + e] - n)));
        }
        for (int i = tid; !running && i < chunks * width; i += 256) {
            const int c = i / width, e = i % width, n = (int)sums[i];
            if (n == 0 || c == own) continue;
            atomicAdd(all + e, n);
            if (c < own) atomicAdd(before + e, n);
        }
    }
    const int pieces = width / 16, side = 256 / pieces;  // 1 to 64 pieces of a row, so 4 rows at a time at least
    const int piece = tid % pieces, row0 = tid / pieces;
    if (row0 < side) {
        // Sums of bytes, two in a register: a thread has at most a quarter of the
        // rows, and a row's counts are at most its tokens.
        static_assert(CHUNK <= CHUNKED && CHUNKED / 4 * PLACE < 1 << 16, "sums in 16 bits");
        u32 sum[8], low[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[j] = low[j] = 0;
        const auto add = [&](u32x4 v, bool earlier) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const u32 n = v[j / 2] >> (8 * (j % 2)) & 0x00ff00ffu;  // bytes j % 2 and j % 2 + 2
                sum[j] += n;
                low[j] += earlier ? n : 0;
            }
        };
        const u32x4* const counts = reinterpret_cast<const u32x4*>(a.counts) + piece;
        int b = from + row0;
        for (; b + 3 * side < to; b += 4 * side) {
            u32x4 v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = counts[(int64_t)(b + i * side) * pieces];
#pragma unroll
            for (int i = 0; i < 4; ++i) add(v[i], b + i * side < mine);
        }
        for (; b < to; b += side) add(counts[(int64_t)b * pieces], b < mine);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int e = 16 * piece + 4 * (j / 2) + j % 2;
            if (low[j] & 0xffff) atomicAdd(before + e, (int)(low[j] & 0xffff));
            if (low[j] >> 16) atomicAdd(before + e + 2, (int)(low[j] >> 16));
            if (sum[j] & 0xffff) atomicAdd(all + e, (int)(sum[j] & 0xffff));
            if (sum[j] >> 16) atomicAdd(all + e + 2, (int)(sum[j] >> 16));
        }
    }
    __syncthreads();
    const int rows = sums_before(a.experts, part, [&](int e) { return all[e]; },
                                 [&](int e, int at, int) {
                                     before[e] += at;
                                     if (blockIdx.x == 0) a.offsets[e] = at;
                                 });
    if (blockIdx.x == 0 && tid == 0) a.offsets[a.experts] = rows;
    for (int p = tid; p < pairs; p += 256) {
        const int e = ids[p], t = p / a.top_k;
        const int row = e < 0 ? -1 : before[e] + (int)__popcll(mask[e] & ((1ull << t) - 1));
        const int64_t pair = first * a.top_k + p;
        if (a.pair_row) a.pair_row[pair] = row;
        if (row < 0) continue;
        if (a.pair_token) a.pair_token[row] = (int32_t)(first + t);
        if (a.pair_weight) a.pair_weight[row] = a.weights[pair];
    }
}

int64_t count_bytes(int64_t blocks, int experts) { return blocks * ((experts + 15) & ~15); }

template <int L, int PER, Mode MODE>
hipError_t launch(const RouteArgs& a, hipStream_t st) {
    constexpr int AT_ONCE = 1024 / L;
    if (a.tokens <= AT_ONCE) {
        // Four waves at least, for what is done for each expert (one token of 256
        // experts: 5.1 us, 6.1 with one wave).
        const int threads = a.tokens * L < 256 ? 256 : (int)((a.tokens * L + 63) / 64 * 64);
        const size_t lds = (size_t)a.experts * 12 + (size_t)AT_ONCE * a.top_k * 8;
        route_kernel<L, PER, MODE, true><<<dim3(1), dim3(threads), lds, st>>>(a, AT_ONCE);
        return hipGetLastError();
    }
    const int block = block_tokens(a.tokens);
    const int64_t blocks = (a.tokens + block - 1) / block;
    route_kernel<L, PER, MODE, false><<<dim3((unsigned)blocks), dim3(block * L < 1024 ? block * L : 1024), (size_t)a.experts * 8, st>>>(a, block);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !a.offsets) return e;
    const int width = (a.experts + 15) & ~15;
    u32* sums = nullptr;
    const int chunks = (int)((blocks + CHUNK - 1) / CHUNK);
    const bool running = chunks * width > RUNNING;
    if (blocks > CHUNKED) {
        sums = reinterpret_cast<u32*>(a.counts + count_bytes(blocks, a.experts));
        route_sums_kernel<<<dim3((unsigned)chunks), dim3(256), (size_t)width * 4, st>>>(a.counts, sums, width, (int)blocks);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        if (running) {
            route_running_kernel<<<dim3((unsigned)((width + 63) / 64)), dim3(1024), 0, st>>>(sums, width, chunks);
            if ((e = hipGetLastError()) != hipSuccess) return e;
        }
    }
    const size_t place = (size_t)a.experts * 8 + (size_t)width * 8;
    route_place_kernel<<<dim3((unsigned)((a.tokens + PLACE - 1) / PLACE)), dim3(256), place, st>>>(a, block, (int)blocks, sums, running);
    return hipGetLastError();
}

template <int L, int PER>
hipError_t launch_mode(const RouteArgs& a, hipStream_t st) {
    if (a.bias) return launch<L, PER, BIASED>(a, st);
    if (a.groups > 1 && a.group_best == 2) return launch<L, PER, PAIRS>(a, st);
    return launch<L, PER, LOGITS>(a, st);
}

}  // namespace

size_t route_workspace(int64_t tokens, int experts) {
    if (tokens <= ROUTE_ONE) return 0;
    const int block = block_tokens(tokens);
    // (What does for these tokens does for fewer, which may have more rows of counts.)
    const int64_t fewer = tokens > 4 * CHUNKED ? CHUNKED : 0;
    const int64_t blocks = std::max((tokens + block - 1) / block, fewer);
    return (size_t)(count_bytes(blocks, experts) + (blocks > CHUNKED ? 4 * count_bytes((blocks + CHUNK - 1) / CHUNK, experts) : 0));
}

hipError_t launch_route(const RouteArgs& a, hipStream_t st) {
    // A wave for each token is the shortest way through (one token of 128
    // experts: 4.5 us against 6.3 with 16 lanes); four tokens to a wave take
    // fewer instructions in all and are quicker once the device is full (16384
    // tokens of 128 experts, ids only: 9.3 us against 13.7), and where they save
    // the second launch (64 experts: 64 tokens 7.7 us, 8.9 with a wave each; 128:
    // 48 tokens 8.9, 9.0, but 64 tokens 10.6, 9.1).
    const bool one = a.experts <= 128 && a.tokens > ROUTE_ONE && a.tokens <= (a.experts <= 64 ? ROUTE_ONE_16 : 48) && !a.bias && a.groups == 1;
    if ((a.tokens > ROUTE_WAVES || one) && a.top_k <= 16 && a.groups <= 16) {
        if (a.experts <= 64) return launch_mode<16, 4>(a, st);
        if (a.experts <= 128) return launch_mode<16, 8>(a, st);
        // 16 experts a lane only where the choice is on logits (16384 tokens of 256:
        // 25.5 us against 29.6); with scores beside them registers run out (with a
        // bias 44.6 against 38.8).
        if (a.experts <= 256 && !a.bias && (a.groups == 1 || a.group_best == 1)) return launch<16, 16, LOGITS>(a, st);
    }
    if (a.experts <= 64) return launch_mode<64, 1>(a, st);
    if (a.experts <= 128) return launch_mode<64, 2>(a, st);
    if (a.experts <= 256) return launch_mode<64, 4>(a, st);
    if (a.experts <= 512) return launch_mode<64, 8>(a, st);
    return launch_mode<64, 16>(a, st);
}

}  // namespace qmm
