// The router: each token's top-k experts and their weights from its logits.
//
// One warp a token.  Without bias and groups experts are chosen by their
// logits, which order as their scores do.  Otherwise by c = score + bias in fp32,
// whose rounding may turn two neighbours round: where two of the values that
// decide the choice lie closer than a bound of that rounding (score_reach, and
// below it) and do not come from the same logit and bias, the token is chosen
// once more by c in 64 bits (14 us; one of some 1900 tokens of 256 experts, sigmoid,
// bias in steps of 0.001, 4 of 8 groups; with a bias and 32 slots, whose 33rd candidate has
// no lane, every token).  32768 of those tokens: 79.9 us.
//
// The choice.  The K-th largest of the lanes' largest values bounds the K-th
// largest value from below, and few values reach it: they go to a list, whose
// members find their places by comparing themselves with one another.  The
// instructions bound the kernel for many tokens, about 400 for one of 256
// experts, 8 chosen (32768 fp32 tokens 15.2 us, 2.4 TB/s, and bf16 ones the same, 1.3 TB/s);
// K rounds of a warp's maximum over what is left took 29.6 us.
#include <algorithm>
#include <type_traits>

#include "route_common.cuh"

namespace epg {

namespace {

constexpr int kWarps = 4;
constexpr uint32_t kClosed = 0x007fffffu;      // key of -inf; a closed expert's is this or less

// Unsigned keys that order as the values do: NaN above all, then +inf, down to
// -inf.
__device__ __forceinline__ uint32_t key_of(float v) {
    const uint32_t b = __float_as_uint(v + 0.0f);    // -0 as +0, any NaN as the positive one
    return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ uint64_t key_of(double v) {
    const uint64_t b = static_cast<uint64_t>(__double_as_longlong(v + 0.0));
    return v != v ? ~0ull : v == -kInf ? 0ull : (b >> 63 ? ~b : b | (1ull << 63));
}
__device__ __forceinline__ uint32_t key_max(uint32_t k) { return __reduce_max_sync(0xffffffffu, k); }
__device__ __forceinline__ uint64_t key_max(uint64_t k) {
    const uint32_t hi = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(k >> 32));
    const uint32_t lo = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(k >> 32) == hi ? static_cast<uint32_t>(k) : 0u);
    return static_cast<uint64_t>(hi) << 32 | lo;
}
__device__ __forceinline__ float value_of(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

// How far a score s in fp32 may lie from the formula's, x its logit less the row's largest.  With u = 2^-24, in s: softmax
// |x| u by x's rounding and 4 u by expf's (2 units of the last place), for s itself and for the total, where the mean of |x|
// by the scores is at most ln E < 8; the total's additions, at most kPer - 1 in a lane and 5 between lanes; the division's u.
// Sigmoid, e = expf(-|l|): (4 (1 - s) + 2) u where s >= 1/2, (4 + 4 s + 2) u below: at most 8 s u, and at most 4 u.  (Down
// at the subnormal numbers a few of their steps; beyond |x| = 128 a score is 0.)
constexpr float kHalfStep = 5.9604645e-8f;     // u
template <int kPer>
__device__ __forceinline__ float score_reach(bool softmax, float s, float x) {
    return kHalfStep * (softmax ? s * (kPer + 24.0f + fminf(-x, 128.0f)) : fminf(9.0f * s, 4.5f)) + 1.2e-38f;
}
// The most of any score of a row: s (a - x) falls with -x, from the largest score on, 1 over the total.
template <int kPer>
__device__ __forceinline__ float row_reach(bool softmax, float total) {
    return score_reach<kPer>(softmax, softmax ? 1.0f / total : 1.0f, 0.0f);
}
// How far c = s + bias may: its own rounding besides.
__device__ __forceinline__ float sum_reach(float of_score, float c) { return of_score + kHalfStep * fabsf(c); }

// What a warp's choice needs in shared memory: the candidates in the order of their indices, and the chosen ones' places.
struct alignas(16) Lists {
    uint32_t key[36];        // (the last four: zeros behind 32, and where what is no candidate goes)
    int16_t expert[36];
    int16_t ranked[33];
};

// The K largest keys, equal ones by the lower index, one round a slot: lane k gets the k-th expert, or -1.
template <int kPer, typename Key>
__device__ __forceinline__ int choose_in_rounds(Key (&key)[kPer], int K, Key closed, int lane) {
    int mine = -1;
    for (int k = 0; k < K; ++k) {
        Key best = closed;
        int at = 0x7fffffff;
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            if (key[j] > best) {
                best = key[j];
                at = j * 32 + lane;
            }
        const Key top = key_max(best);
        if (top == closed) break;     // nothing is open any more
        const int e = __reduce_min_sync(0xffffffffu, best == top ? at : 0x7fffffff);
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            if (e == j * 32 + lane) key[j] = closed;
        if (lane == k) mine = e;
    }
    return mine;
}

// The same by a list: some lane for each of the K experts has its slot in *place and its key in *mine (the others'
// places are K or more).  Returns the expert; with `ranked`, list->ranked has the first K + 1 in order, -1 after the last.
template <int kPer>
__device__ __forceinline__ int choose(uint32_t (&key)[kPer], int K, bool ranked, Lists* list, int lane, int* place,
                                      uint32_t* mine) {
    const int wanted = K + (ranked ? 1 : 0);
    uint32_t best = key[0];
#pragma unroll
    for (int j = 1; j < kPer; ++j) best = max(best, key[j]);
    uint32_t least = 0;
#pragma unroll 4
    for (int k = 0; k < wanted; ++k) {
        least = __reduce_max_sync(0xffffffffu, best);
        best = best == least ? 0 : best;
    }
    least = max(least, kClosed + 1);      // (fewer lanes with open ones than wanted: all that are open)
    int n = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const unsigned there = __ballot_sync(0xffffffffu, key[j] >= least);
        const int at = key[j] >= least ? min(n + __popc(there & ((1u << lane) - 1)), 32) : 32;
        list->key[at] = key[j];
        list->expert[at] = static_cast<int16_t>(j * 32 + lane);
        n += __popc(there);
    }
    __syncwarp();
    int e = -1;
    if (n <= 32) {
        // larger ones come first, and equal ones before
        if (lane < 4) list->key[n + lane] = 0;
        __syncwarp();
        const uint32_t own = lane < n ? list->key[lane] : 0;
        int rank = __popc(__match_any_sync(0xffffffffu, own) & ((1u << lane) - 1));
        for (int i = 0; i < n; i += 4) {
            const uint4 k = *reinterpret_cast<const uint4*>(list->key + i);
            rank += (k.x > own) + (k.y > own) + (k.z > own) + (k.w > own);
        }
        *place = lane < n ? rank : wanted;
        *mine = own;
        e = lane < n ? list->expert[lane] : -1;
    } else {
        // many equal values, or few lanes with open ones
        uint32_t left[kPer];
#pragma unroll
        for (int j = 0; j < kPer; ++j) left[j] = key[j];
        e = choose_in_rounds(left, min(wanted, 32), kClosed, lane);
        *place = e >= 0 ? lane : wanted;
        uint32_t found = 0;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const uint32_t other = __shfl_sync(0xffffffffu, key[j], e & 31);
            if (e >= 0 && e / 32 == j) found = other;
        }
        *mine = found;
    }
    if (ranked) {
        if (lane <= K) list->ranked[lane] = -1;
        if (lane == 0) list->ranked[32] = -1;
        __syncwarp();
        if (e >= 0 && *place <= K) list->ranked[*place] = static_cast<int16_t>(e);
    }
    __syncwarp();
    return e;
}

// Closes the experts of all but the topk_groups best groups.  c is in shared memory by expert.
// With `close`, which says whether c's rounding may have made another choice: of_score, how far a score may be off.
template <typename V>
__device__ __forceinline__ void keep_groups(const RouteParams& p, V* c, int lane, float of_score, bool* close) {
    const int G = p.num_groups, size = p.E / G;
    // lanes of a group: a power of two
    int share = 1;
    while (share * 2 * G <= 32) share *= 2;
    const int g = lane / share, sub = lane & (share - 1), turns = (size + share - 1) / share;
    V first = -kInf, second = -kInf;
    if (g < G)
        for (int i = 0, at = g % turns; i < turns; ++i, at = at + 1 == turns ? 0 : at + 1) {     // (each group in another bank)
            const int e = at * share + sub;
            const V v = e < size ? c[g * size + e] : static_cast<V>(-kInf);
            if (v != v || v > first) {
                second = first;
                first = v;
            } else if (v > second) {
                second = v;
            }
        }
    for (int o = 1; o < share; o *= 2) {
        const V other = __shfl_xor_sync(0xffffffffu, first, o), next = __shfl_xor_sync(0xffffffffu, second, o);
        const bool higher = key_of(other) > key_of(first);
        const V rest = higher ? first : other, own = higher ? next : second;
        first = higher ? other : first;
        second = key_of(rest) > key_of(own) ? rest : own;
    }
    const bool open = g < G && first != static_cast<V>(-kInf);
    const V score = second != static_cast<V>(-kInf) ? first + second : first;
    // the best groups, one round each, equal ones by the lower index
    auto key = open && sub == 0 ? key_of(score) : decltype(key_of(score))(0);
    unsigned keep = 0;
    V worst = 0;
    for (int k = 0; k < p.topk_groups; ++k) {
        const auto top = key_max(key);
        if (top == 0) break;
        const int winner = __ffs(__ballot_sync(0xffffffffu, key == top)) - 1;
        if (lane == winner) key = 0;
        keep |= 1u << (winner / share);
        worst = __shfl_sync(0xffffffffu, score, winner);
    }
    const bool kept = g < G && (keep >> g & 1);
    if (close && sizeof(V) == 4) {
        // The last one kept against the best one dropped, by the most that any group's sum may be off: its two members'
        // scores, their c's and its own rounding.  (The members may be far larger than their sum, and another kept group's
        // sum, larger than the last one's, may be off by more.)
        const float one = static_cast<float>(first), two = second != static_cast<V>(-kInf) ? static_cast<float>(second) : 0.0f;
        const float off = 2.0f * of_score + kHalfStep * (fabsf(one) + fabsf(two) + fabsf(static_cast<float>(score)));
        const float reach = open && one != kInf ? off : 0.0f;      // (+inf is itself in any number of bits)
        const auto next = key_max(key);
        const int other = next == 0 ? -1 : __ffs(__ballot_sync(0xffffffffu, key == next)) - 1;
        const float b = __shfl_sync(0xffffffffu, static_cast<float>(score), other & 31), a = static_cast<float>(worst);
        if (!(a - b > 2.0f * warp_max(reach)) && other >= 0) *close = true;
    }
    if (g < G && !kept)
        for (int i = sub; i < size; i += share) c[g * size + i] = -kInf;
    __syncwarp();
}

// The choice by c in 64 bits: lane k gets the k-th expert, or -1.
template <int kPer>
__device__ __noinline__ int choose_by_doubles(const RouteParams& p, const float (&l)[kPer], const float (&c)[kPer],
                                              bool all, float largest, double* mem, int lane) {
    const bool softmax = p.score == EP_SCORE_SOFTMAX;
    double total = 0.0;
    if (softmax) {
#pragma unroll 1
        for (int j = 0; j < kPer; ++j)
            if (l[j] != -kInf) total += exp(static_cast<double>(l[j]) - largest);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    }
    double c64[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int e = j * 32 + lane;
        const double d = l[j];
        c64[j] = -kInf;
        if (e < p.E && l[j] != -kInf && (all || c[j] != -kInf)) {
            const double s = softmax ? exp(d - largest) / total : 1.0 / (1.0 + exp(-d));
            c64[j] = s + (p.bias ? static_cast<double>(p.bias[e]) : 0.0);
        }
    }
    if (all) {
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            if (j * 32 + lane < p.E) mem[j * 32 + lane] = c64[j];
        __syncwarp();
        keep_groups(p, mem, lane, 0.0f, static_cast<bool*>(nullptr));
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            if (j * 32 + lane < p.E) c64[j] = mem[j * 32 + lane];
        __syncwarp();
    }
    uint64_t key[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) key[j] = c64[j] == -kInf ? 0ull : key_of(p.bias ? c64[j] : static_cast<double>(l[j]));
    return choose_in_rounds(key, p.K, uint64_t{0}, lane);
}

template <typename L, int kPer, bool kFull, bool kByScore>
__global__ void __launch_bounds__(kWarps * 32) route_kernel(const RouteParams p) {
    extern __shared__ double smem[];     // [kWarps][E] where groups are kept
    __shared__ Lists lists[kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    Lists* const list = &lists[warp];
    const bool softmax = p.score == EP_SCORE_SOFTMAX;
    pdl_wait();
    pdl_launch_dependents();
    constexpr bool kAhead = kPer <= 16;      // the next row is asked for before this one's work
    const int step = gridDim.x * kWarps, first = blockIdx.x * kWarps + warp;
    const L* const logits = static_cast<const L*>(p.logits);
    float ahead[kPer];
    if (kAhead && first < p.T) load_row<kPer, kFull>(logits + first * p.row_stride, p.E, lane, ahead);
    for (int t = first; t < p.T; t += step) {
        const int64_t out = static_cast<int64_t>(t) * p.K;
        const L* const row = logits + t * p.row_stride;
        float l[kPer];
        if constexpr (kAhead) {
#pragma unroll
            for (int j = 0; j < kPer; ++j) l[j] = ahead[j];
            if (t < p.T - step) load_row<kPer, kFull>(row + step * p.row_stride, p.E, lane, ahead);
        } else {
            load_row<kPer, kFull>(row, p.E, lane, l);
        }
        if (p.token_mask && p.token_mask[t] == 0) {
            if (lane < p.K) {
                p.topk_idx[out + lane] = -1;
                p.topk_weights[out + lane] = 0.0f;
            }
            continue;
        }
        float largest = 0.0f, total = 0.0f;
        if (softmax && (kByScore || !p.normalize)) {
            largest = l[0];
#pragma unroll
            for (int j = 1; j < kPer; ++j) largest = fmaxf(largest, l[j]);
            largest = warp_max(largest);
#pragma unroll
            for (int j = 0; j < kPer; ++j) total += expf(l[j] - largest);
            total = warp_sum(total);
        }
        uint32_t key[kPer], mine;
        int e, place;
        if constexpr (!kByScore) {
#pragma unroll
            for (int j = 0; j < kPer; ++j) key[j] = key_of(l[j]);
            e = choose(key, p.K, false, list, lane, &place, &mine);
        } else {
            bool close = false;
            float c[kPer];
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                const int expert = j * 32 + lane;
                const float s = softmax ? expf(l[j] - largest) / total : sigmoid_shifted(l[j], 0.0f);
                c[j] = l[j] == -kInf ? -kInf : s + (p.bias && expert < p.E ? p.bias[expert] : 0.0f);
            }
            const bool grouped = p.topk_groups < p.num_groups;
            double* const mem = smem + static_cast<size_t>(warp) * p.E;
            if (grouped) {
                float* const m = reinterpret_cast<float*>(mem);
#pragma unroll
                for (int j = 0; j < kPer; ++j)
                    if (j * 32 + lane < p.E) m[j * 32 + lane] = c[j];
                __syncwarp();
                keep_groups(p, m, lane, row_reach<kPer>(softmax, total), &close);
#pragma unroll
                for (int j = 0; j < kPer; ++j)
                    if (j * 32 + lane < p.E) c[j] = m[j * 32 + lane];
                __syncwarp();
            }
            // without a bias the choice among the kept ones goes by the logits
#pragma unroll
            for (int j = 0; j < kPer; ++j) key[j] = c[j] == -kInf ? 0u : key_of(p.bias ? c[j] : l[j]);
            e = choose(key, p.K, true, list, lane, &place, &mine);
            if (p.bias) {
                // Neighbours of the first K + 1 that fp32 may have turned round: lane k the k-th and the next.  (Two values
                // that it has turned round lie within both their reaches, so of the neighbours between them a pair does, or
                // all are alike.)
                bool near = false, beyond = false;
                float la = 0.0f, ba = 0.0f, ca = 0.0f, ra = 0.0f;
                const auto sum = [&](float logit, float b, float* reach) {
                    const float s = softmax ? expf(logit - largest) / total : sigmoid_shifted(logit, 0.0f);
                    *reach = sum_reach(score_reach<kPer>(softmax, s, logit - largest), s + b);
                    return s + b;
                };
                const int a = lane < p.K ? list->ranked[lane] : -1, b = lane < p.K ? list->ranked[lane + 1] : -1;
                if (a >= 0 && b >= 0 && EP_IN(a, p.E) && EP_IN(b, p.E)) {
                    const float lb = to_float(row[b]), bb = p.bias[b];
                    la = to_float(row[a]);
                    ba = p.bias[a];
                    float rb;
                    ca = sum(la, ba, &ra);
                    const float cb = sum(lb, bb, &rb);
                    const bool same = la == lb && ba == bb;
                    near = ca - cb <= ra + rb && !same;
                    // Behind the last slot's, one that is not listed may come before it: where the next one is of the same logit
                    // and bias, or fp32 knows the other's score less well than the next one's.
                    beyond = lane == p.K - 1 && (same || ca - cb <= ra + sum_reach(row_reach<kPer>(softmax, total), ca));
                }
                if (__any_sync(0xffffffffu, beyond && !near)) {
                    la = __shfl_sync(0xffffffffu, la, p.K - 1);
                    ba = __shfl_sync(0xffffffffu, ba, p.K - 1);
                    ca = __shfl_sync(0xffffffffu, ca, p.K - 1);
                    ra = __shfl_sync(0xffffffffu, ra, p.K - 1);
#pragma unroll
                    for (int j = 0; j < kPer; ++j) {
                        if (c[j] == -kInf || c[j] > ca || (l[j] == la && p.bias[j * 32 + lane] == ba)) continue;
                        float r;
                        const float other = sum(l[j], p.bias[j * 32 + lane], &r);
                        near |= ca - other <= ra + r;
                    }
                }
                close |= __any_sync(0xffffffffu, near) || p.K == 32;     // (the 33rd has no lane)
            }
            if (close) {
                // one logit and one bias everywhere (a router before its first step) is a tie in any number of bits
                const float first_l = __shfl_sync(0xffffffffu, l[0], 0), first_b = p.bias ? p.bias[0] : 0.0f;
                bool differs = false;
#pragma unroll
                for (int j = 0; j < kPer; ++j) {
                    const int expert = j * 32 + lane;
                    if (expert < p.E) differs |= l[j] != first_l || (p.bias && p.bias[expert] != first_b);
                }
                close = __any_sync(0xffffffffu, differs);
            }
            if (close) {
                e = choose_by_doubles(p, l, c, grouped, largest, mem, lane);
                place = e >= 0 ? lane : p.K;
            }
        }
        // weights, by the lane that has a slot
        const bool there = e >= 0 && place < p.K && EP_IN(e, p.E) && EP_IN(place, p.K);
        const float v = !there ? -kInf : kByScore ? to_float(row[e]) : value_of(mine);
        float w;
        if (p.normalize) {
            const float top = warp_max(v);
            float s = 0.0f, rest;
            if (there)
                s = softmax ? exp2_approx((v - top) * kLog2E)
                            : shift_of(top) == 0.0f ? sigmoid_fast(v, &rest) : sigmoid_shifted(v, shift_of(top));
            w = s * (p.scale * reciprocal_approx(warp_sum(s)));
        } else {
            w = (softmax ? expf(v - largest) / total : sigmoid_shifted(v, 0.0f)) * p.scale;
        }
        const int filled = __popc(__ballot_sync(0xffffffffu, there));
        if (there) {
            p.topk_idx[out + place] = e;
            p.topk_weights[out + place] = w;
        }
        if (lane >= filled && lane < p.K && EP_IN(out + lane, static_cast<int64_t>(p.T) * p.K)) {
            p.topk_idx[out + lane] = -1;
            p.topk_weights[out + lane] = 0.0f;
        }
    }
}

}  // namespace

cudaError_t launch_route(const RouteParams& p, cudaStream_t stream) {
    return with_row_type(p.dtype, p.E, [&](auto* type, auto per, auto full) {
        using L = std::remove_const_t<std::remove_pointer_t<decltype(type)>>;
        const bool grouped = p.topk_groups < p.num_groups;
        const size_t smem = grouped ? static_cast<size_t>(kWarps) * p.E * 8 : 0;
        constexpr int kPer = decltype(per)::value;
        constexpr bool kFull = decltype(full)::value;
        const auto kernel = p.bias || grouped ? route_kernel<L, kPer, kFull, true> : route_kernel<L, kPer, kFull, false>;
        // Beyond what a kernel may have unasked, its own arrays among it: the most that any call asks for, so that a call
        // of another thread does not take it back before the launch.
        if (smem + kWarps * sizeof(Lists) > 48 * 1024) {
            const cudaError_t e =
                cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kWarps * EP_MAX_EXPERTS * 8);
            if (e != cudaSuccess) return e;
        }
        // (many tokens: warps that go on to another token have asked for its row)
        const int blocks = std::min((p.T + kWarps - 1) / kWarps, device_info().num_sms * 16);
        return launch_pdl(kernel, dim3(blocks), dim3(kWarps * 32), smem, stream, p);
    });
}

}  // namespace epg
