// moe_route.hip -- a token's scores for the experts to its experts, their
// weights, and the rows grouped by expert that the experts' products take:
//   s = softmax(l) or sigmoid(l),  c = s + bias,
//   the top_groups groups of highest score stay (a group's score: the sum of
//   its group_best highest c), of their experts the top_k of highest c,
//   w = s[chosen] [/ sum over the chosen] * scale,
// then a counting sort of the (token, expert) pairs by expert, within an expert
// by token.
//
// A choice hangs on the last bits of its scores, so it is made on numbers that
// never run together: without a bias the order of the scores is that of the
// logits, which are compared as they are; with one, scores are formed in 64
// bits.  Keys are whole numbers in the order of the values, so that a place that
// is taken (or not there) has a key below all of them.
#include "layer_device.h"
#include "moe_kernels.h"

namespace qmm {
namespace {

constexpr float INF = __builtin_huge_valf();

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
template <class V>
__device__ __forceinline__ V lane_xor(V v, int mask) {
    if constexpr (sizeof(V) == 4) {
        return __builtin_bit_cast(V, __shfl_xor(__builtin_bit_cast(int, v), mask, 64));
    } else {
        const u32x2 x = __builtin_bit_cast(u32x2, v);
        u32x2 r;
        r[0] = (u32)__shfl_xor((int)x[0], mask, 64);
        r[1] = (u32)__shfl_xor((int)x[1], mask, 64);
        return __builtin_bit_cast(V, r);
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
        v = f(v, lane_xor(v, 16));
        v = f(v, lane_xor(v, 32));
    }
    return v;
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

// What one token's lanes know after its choice: lane j < top_k holds expert and
// weight of choice j.
struct Chosen {
    int id;
    float w;
};

// L lanes share a token; lane i of them holds experts i PER .. i PER + PER - 1.
template <int L, int PER, bool BIAS>
__device__ __forceinline__ Chosen choose(const RouteArgs& a, int64_t token, int lane) {
    using Key = std::conditional_t<BIAS, int64_t, int>;
    const int e0 = lane * PER;
    float l[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) l[i] = -INF;
    if (a.f16) {
        const f16* p = static_cast<const f16*>(a.logits) + token * a.stride;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (e0 + i < a.experts) l[i] = (float)p[e0 + i];
    } else {
        const float* p = static_cast<const float*>(a.logits) + token * a.stride;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (e0 + i < a.experts) l[i] = p[e0 + i];
    }
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

    const bool pairs = a.groups > 1 && a.group_best == 2;
    double s[PER];  // scores in 64 bits where a sum of them is compared
    if (BIAS || pairs) {
        if (a.sigmoid) {
#pragma unroll
            for (int i = 0; i < PER; ++i) s[i] = 1.0 / (1.0 + exp(-(double)l[i]));
        } else {
            double sum = 0.0;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                s[i] = empty ? 0.0 : l[i] == top ? 1.0 : exp((double)l[i] - (double)top);  // top may be +inf
                sum += s[i];
            }
            sum = lanes<L>(sum, Add{});
            const double r = empty ? 0.0 : 1.0 / sum;
#pragma unroll
            for (int i = 0; i < PER; ++i) s[i] *= r;
        }
        if constexpr (BIAS) {
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (e0 + i < a.experts) s[i] += (double)a.bias[e0 + i];
        }
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (s[i] != s[i]) s[i] = -(double)INF;
    }
    Key key[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        if constexpr (BIAS)
            key[i] = order_key(s[i]);
        else
            key[i] = order_key(l[i]);
        if (e0 + i >= a.experts) key[i] = taken<Key>();
    }
    if (a.groups > 1) {
        const int each = a.experts / a.groups;
        // Lane g holds the score of group g.
        int64_t mine = taken<int64_t>();
        for (int g = 0; g < a.groups; ++g) {
            const int lo = g * each, hi = lo + each;
            int64_t best;
            if (a.group_best == 1) {
                Key k = taken<Key>();
#pragma unroll
                for (int i = 0; i < PER; ++i)
                    if (e0 + i >= lo && e0 + i < hi && key[i] > k) k = key[i];
                best = lanes<L>(k, Max{});
            } else {
                // The two highest, lane by lane and then over the lanes.
                double x = -(double)INF, y = -(double)INF;
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    if (e0 + i < lo || e0 + i >= hi) continue;
                    y = fmax(y, fmin(x, s[i]));
                    x = fmax(x, s[i]);
                }
                const double first = lanes<L>(x, Max{});
                const int owner = lanes<L>(x == first ? lane : L, Min{});
                const double second = lanes<L>(lane == owner ? y : x, Max{});
                double sum = first + second;
                if (sum != sum) sum = -(double)INF;
                best = order_key(sum);
            }
            if (lane == g) mine = best;
        }
        // One bit for each group that stays.
        uint64_t stay = 0;
        for (int j = 0; j < a.top_groups; ++j) {
            const int64_t m = lanes<L>(mine, Max{});
            const int g = lanes<L>(mine == m ? lane : L, Min{});
            stay |= 1ull << g;
            if (lane == g) mine = taken<int64_t>();
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = e0 + i;
            if (e < a.experts && !(stay >> (e / each) & 1)) key[i] = taken<Key>();
        }
    }
    Chosen c{-1, 0.f};
    float chosen_l = -INF;
    for (int j = 0; j < a.top_k; ++j) {
        Key m = key[0];
        int at = e0;
#pragma unroll
        for (int i = 1; i < PER; ++i)
            if (key[i] > m) {
                m = key[i];
                at = e0 + i;
            }
        const Key best = lanes<L>(m, Max{});
        const int e = lanes<L>(m == best ? at : 0x7fffffff, Min{});
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (e0 + i == e) key[i] = taken<Key>();
        if (lane == j) {
            c.id = e;
            if constexpr (!BIAS) chosen_l = key_value(best);
        }
    }
    if constexpr (BIAS) {
        if (lane < a.top_k) {
            const int64_t at = token * a.stride + c.id;
            chosen_l = a.f16 ? (float)static_cast<const f16*>(a.logits)[at] : static_cast<const float*>(a.logits)[at];
        }
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
        if (lane < a.top_k) w = expf(chosen_l - top);
        float sum;
        if (a.renorm) {
            sum = lanes<L>(w, Add{});
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

// A work-group takes ROUTE_BLOCK tokens (ONE: all of them, in as many rounds)
// and T / L of them at a time.  Ranks within an expert come from a mask per
// expert with a bit for each token: a token names an expert at most once.
template <int T, int L, int PER, bool BIAS, bool ONE>
__global__ void __launch_bounds__(T) route_kernel(RouteArgs a) {
    extern __shared__ uint64_t mask[];  // [experts], then ids and weights of the block's pairs
    __shared__ int part[T / 64];
    constexpr int TOKENS = T / L;
    const int tid = threadIdx.x, lane = tid % L, slot = tid / L;
    int* const lds_id = reinterpret_cast<int*>(mask + a.experts);
    float* const lds_w = reinterpret_cast<float*>(lds_id + ROUTE_BLOCK * a.top_k);
    const int64_t first = (int64_t)blockIdx.x * ROUTE_BLOCK;
    const int here = (int)(a.tokens - first < ROUTE_BLOCK ? a.tokens - first : ROUTE_BLOCK);
    for (int e = tid; e < a.experts; e += T) mask[e] = 0;
    __syncthreads();
    for (int t = slot; t < ROUTE_BLOCK; t += TOKENS) {
        if (t - slot >= here) break;  // the same for all
        const bool live = t < here;
        const int64_t token = first + (live ? t : 0);
        Chosen c = choose<L, PER, BIAS>(a, token, lane);
        if (!live || lane >= a.top_k) continue;
        if (a.keep && !a.keep[token]) c = Chosen{-1, 0.f};
        const int64_t pair = token * a.top_k + lane;
        if (a.ids) a.ids[pair] = c.id;
        if (a.weights) a.weights[pair] = c.w;
        lds_id[t * a.top_k + lane] = c.id;
        lds_w[t * a.top_k + lane] = c.w;
        if (c.id >= 0) atomicOr(reinterpret_cast<unsigned long long*>(mask + c.id), 1ull << t);
    }
    if (!a.offsets) return;
    __syncthreads();
    const int pairs = here * a.top_k;
    if constexpr (ONE) {
        // Offsets: sums over the experts before, T of them at a time; the
        // masks' places take the offsets.
        int base = 0;
        int* const off = reinterpret_cast<int*>(lds_w + ROUTE_BLOCK * a.top_k);
        for (int e0 = 0; e0 < a.experts; e0 += T) {
            const int e = e0 + tid;
            const int n = e < a.experts ? __popcll(mask[e]) : 0;
            int sum = n;
            for (int d = 1; d < 64; d *= 2) {
                const int before = __shfl_up(sum, d, 64);
                if ((tid & 63) >= d) sum += before;
            }
            if ((tid & 63) == 63) part[tid >> 6] = sum;
            __syncthreads();
            int before = base;
            for (int i = 0; i < T / 64; ++i) {
                if (i < tid >> 6) before += part[i];
                base += part[i];
            }
            if (e < a.experts) {
                off[e] = before + sum - n;
                a.offsets[e] = before + sum - n;
            }
            __syncthreads();
        }
        if (tid == 0) a.offsets[a.experts] = base;
        for (int p = tid; p < pairs; p += T) {
            const int e = lds_id[p], t = p / a.top_k;
            const int row = e < 0 ? -1 : off[e] + __popcll(mask[e] & ((1ull << t) - 1));
            if (a.pair_row) a.pair_row[p] = row;
            if (row < 0) continue;
            if (a.pair_token) a.pair_token[row] = t;
            if (a.pair_weight) a.pair_weight[row] = lds_w[p];
        }
    } else {
        const int width = (a.experts + 7) & ~7;
        uint16_t* const counts = a.counts + (int64_t)blockIdx.x * width;
        for (int e = tid; e < width; e += T) counts[e] = e < a.experts ? (uint16_t)__popcll(mask[e]) : (uint16_t)0;
    }
}

// Second launch where several work-groups routed: each takes the tokens of one
// of them again, adds up what the experts got before, and places its pairs.
template <int T>
__global__ void __launch_bounds__(T) route_place_kernel(RouteArgs a, int blocks) {
    extern __shared__ uint64_t mask[];  // [experts], then [2][experts]: rows before this work-group, all rows
    __shared__ int part[T / 64];
    const int tid = threadIdx.x;
    int* const before = reinterpret_cast<int*>(mask + a.experts);
    const int width = (a.experts + 7) & ~7;
    const int64_t first = (int64_t)blockIdx.x * ROUTE_BLOCK;
    const int here = (int)(a.tokens - first < ROUTE_BLOCK ? a.tokens - first : ROUTE_BLOCK);
    const int pairs = here * a.top_k;
    for (int e = tid; e < a.experts; e += T) mask[e] = 0;
    __syncthreads();
    const int32_t* const ids = a.ids + first * a.top_k;
    for (int p = tid; p < pairs; p += T) {
        const int e = ids[p];
        if (e >= 0) atomicOr(reinterpret_cast<unsigned long long*>(mask + e), 1ull << (p / a.top_k));
    }
    int base = 0;
    for (int e0 = 0; e0 < a.experts; e0 += T) {
        const int e = e0 + tid;
        int mine = 0, all = 0;
        if (e < a.experts) {
            for (int b = 0; b < blocks; ++b) {
                const int n = a.counts[(int64_t)b * width + e];
                all += n;
                if (b < (int)blockIdx.x) mine += n;
            }
        }
        int sum = all;
        for (int d = 1; d < 64; d *= 2) {
            const int x = __shfl_up(sum, d, 64);
            if ((tid & 63) >= d) sum += x;
        }
        if ((tid & 63) == 63) part[tid >> 6] = sum;
        __syncthreads();
        int at = base;
        for (int i = 0; i < T / 64; ++i) {
            if (i < tid >> 6) at += part[i];
            base += part[i];
        }
        at += sum - all;
        if (e < a.experts) {
            before[e] = at + mine;
            if (blockIdx.x == 0) a.offsets[e] = at;
        }
        __syncthreads();
    }
    if (blockIdx.x == 0 && tid == 0) a.offsets[a.experts] = base;
    for (int p = tid; p < pairs; p += T) {
        const int e = ids[p], t = p / a.top_k;
        const int row = e < 0 ? -1 : before[e] + __popcll(mask[e] & ((1ull << t) - 1));
        const int64_t pair = first * a.top_k + p;
        if (a.pair_row) a.pair_row[pair] = row;
        if (row < 0) continue;
        if (a.pair_token) a.pair_token[row] = (int32_t)(first + t);
        if (a.pair_weight) a.pair_weight[row] = a.weights[pair];
    }
}

template <int T, int L, int PER, bool BIAS>
hipError_t launch(const RouteArgs& a, hipStream_t st) {
    const size_t lds = (size_t)a.experts * 12 + (size_t)ROUTE_BLOCK * a.top_k * 8;
    const int64_t blocks = (a.tokens + ROUTE_BLOCK - 1) / ROUTE_BLOCK;
    if (route_in_one(a.tokens)) {
        route_kernel<T, L, PER, BIAS, true><<<dim3(1), dim3(T), lds, st>>>(a);
        return hipGetLastError();
    }
    route_kernel<T, L, PER, BIAS, false><<<dim3((unsigned)blocks), dim3(T), lds, st>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !a.offsets) return e;
    route_place_kernel<256><<<dim3((unsigned)blocks), dim3(256), (size_t)a.experts * 12, st>>>(a, (int)blocks);
    return hipGetLastError();
}

template <int T, int L, int PER>
hipError_t launch_bias(const RouteArgs& a, hipStream_t st) {
    return a.bias ? launch<T, L, PER, true>(a, st) : launch<T, L, PER, false>(a, st);
}

}  // namespace

bool route_in_one(int64_t tokens) { return tokens <= ROUTE_BLOCK; }

size_t route_workspace(int64_t tokens, int experts) {
    if (route_in_one(tokens)) return 0;
    return (size_t)((tokens + ROUTE_BLOCK - 1) / ROUTE_BLOCK) * (size_t)((experts + 7) & ~7) * 2;
}

hipError_t launch_route(const RouteArgs& a, hipStream_t st) {
    if (a.top_k <= 16 && a.groups <= 16) {
        if (a.experts <= 64) return launch_bias<256, 16, 4>(a, st);
        if (a.experts <= 128) return launch_bias<256, 16, 8>(a, st);
        if (a.experts <= 256) return launch_bias<256, 16, 16>(a, st);
    }
    if (a.experts <= 128) return launch_bias<256, 64, 2>(a, st);
    if (a.experts <= 256) return launch_bias<256, 64, 4>(a, st);
    if (a.experts <= 512) return launch_bias<256, 64, 8>(a, st);
    return launch_bias<256, 64, 16>(a, st);
}

}  // namespace qmm
