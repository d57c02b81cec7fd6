// The router: each token's top-k experts and their weights from its logits.
//
// One warp a token.  Without bias and groups experts are chosen by their
// logits, which order as their scores do.  Otherwise by c = score + bias in fp32,
// whose rounding may turn two neighbours round: where two of the values that
// decide the choice lie closer than that rounding reaches and do not come
// from the same logit and bias, the token is chosen once more by c in 64 bits.
#include <type_traits>

#include "route_common.cuh"

namespace epg {

namespace {

constexpr int kWarps = 4;

// Unsigned keys that order as the values do: NaN above all, then +inf, down to
// -inf; 0 (below every value) is left for closed experts.
__device__ __forceinline__ uint32_t key_of(float v) {
    const uint32_t b = __float_as_uint(v + 0.0f);    // -0 as +0
    return v != v ? 0xffffffffu : (b & 0x80000000u ? ~b : b | 0x80000000u);
}
__device__ __forceinline__ uint64_t key_of(double v) {
    const uint64_t b = static_cast<uint64_t>(__double_as_longlong(v + 0.0));
    return v != v ? ~0ull : (b >> 63 ? ~b : b | (1ull << 63));
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

// How far c in fp32 may lie from c: the score is good to a few units of the last place, the sum to half a one.
__device__ __forceinline__ float reach(float c) { return 5e-7f * fmaxf(1.0f, fabsf(c)); }

template <typename L, int kPer, bool kByScore>
struct Chooser {
    const RouteParams& p;
    const L* row;
    int lane;
    float l[kPer];

    // The K largest keys, equal ones by the lower index: lane k gets the k-th expert, or -1.
    // margin: the least distance between neighbours of the first K + 1 that are not the same inputs.
    template <typename Key>
    __device__ __forceinline__ int choose(Key (&key)[kPer], bool* close) {
        int mine = -1;
        Key before = 0;
        int chosen_before = -1;
        for (int k = 0; k <= p.K; ++k) {
            if (k == p.K && !(kByScore && sizeof(Key) == 4)) break;
            Key best = 0;
            int at = 0x7fffffff;
#pragma unroll
            for (int j = 0; j < kPer; ++j)
                if (key[j] > best) {
                    best = key[j];
                    at = j * 32 + lane;
                }
            const Key top = key_max(best);
            if (top == 0) break;     // nothing is open any more
            const int e = __reduce_min_sync(0xffffffffu, best == top ? at : 0x7fffffff);
            if constexpr (kByScore && sizeof(Key) == 4) {
                if (k > 0) {
                    const float a = value_of(before), b = value_of(top);
                    if (a - b <= reach(a) + reach(b) && before != 0xffffffffu && !same_inputs(chosen_before, e)) *close = true;
                }
            }
            if (k == p.K) break;
#pragma unroll
            for (int j = 0; j < kPer; ++j)
                if (e == j * 32 + lane) key[j] = 0;
            if (lane == k) mine = e;
            before = top;
            chosen_before = e;
        }
        return mine;
    }
    __device__ __forceinline__ bool same_inputs(int a, int b) const {
        return to_float(row[a]) == to_float(row[b]) && (!p.bias || p.bias[a] == p.bias[b]);
    }

    // Closes the experts of all but the topk_groups best groups.  `c` is in shared memory by expert.
    template <typename V>
    __device__ __forceinline__ void keep_groups(V* c, bool* close) {
        const int G = p.num_groups, size = p.E / G;
        V score = 0;
        bool open = false;
        if (lane < G) {
            V first = -kInf, second = -kInf;
            for (int i = 0; i < size; ++i) {
                const V v = c[lane * size + i];
                if (v != v || v > first) {
                    second = first;
                    first = v;
                } else if (v > second) {
                    second = v;
                }
            }
            open = first != -kInf;
            score = second != -kInf ? first + second : first;
        }
        // rank among the groups, equal ones by the lower index; closed groups come last
        int rank = 0;
        V below = -kInf;
        for (int g = 0; g < G; ++g) {
            const V other = __shfl_sync(0xffffffffu, score, g);
            const bool other_open = __shfl_sync(0xffffffffu, open ? 1 : 0, g) != 0;
            if (!other_open || g == lane) continue;
            const bool higher = key_of(other) > key_of(score) || (key_of(other) == key_of(score) && g < lane);
            if (!open || higher) ++rank;
            else if (other > below) below = other;
        }
        const bool kept = lane < G && open && rank < p.topk_groups;
        if (close && sizeof(V) == 4) {
            // the last one kept against the first one dropped
            const bool last = kept && rank == p.topk_groups - 1 && below != static_cast<V>(-kInf);
            const float a = static_cast<float>(score), b = static_cast<float>(below);
            if (__any_sync(0xffffffffu, last && !(a - b > 2.0f * (reach(a) + reach(b))))) *close = true;
        }
        if (lane < G && !kept)
            for (int i = 0; i < size; ++i) c[lane * size + i] = -kInf;
        __syncwarp();
    }
};

template <typename L, int kPer, bool kByScore>
__global__ void __launch_bounds__(kWarps * 32) route_kernel(const RouteParams p) {
    extern __shared__ double smem[];     // [kWarps][E] where groups are kept
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    pdl_wait();
    pdl_launch_dependents();
    for (int t = blockIdx.x * kWarps + warp; t < p.T; t += gridDim.x * kWarps) {
        const int64_t out = static_cast<int64_t>(t) * p.K;
        if (p.token_mask && p.token_mask[t] == 0) {
            if (lane < p.K) {
                p.topk_idx[out + lane] = -1;
                p.topk_weights[out + lane] = 0.0f;
            }
            continue;
        }
        const L* row = static_cast<const L*>(p.logits) + t * p.row_stride;
        Chooser<L, kPer, kByScore> ch{p, row, lane};
        load_row(row, p.E, lane, ch.l);
        float largest = -kInf;
#pragma unroll
        for (int j = 0; j < kPer; ++j) largest = fmaxf(largest, ch.l[j]);
        const bool softmax = p.score == EP_SCORE_SOFTMAX;
        float total = 0.0f;
        if (softmax) {
            largest = warp_max(largest);
            if (kByScore || !p.normalize) {
#pragma unroll
                for (int j = 0; j < kPer; ++j) total += expf(ch.l[j] - largest);
                total = warp_sum(total);
            }
        }
        uint32_t key[kPer];
        int mine;
        if constexpr (!kByScore) {
#pragma unroll
            for (int j = 0; j < kPer; ++j) key[j] = ch.l[j] == -kInf ? 0u : key_of(ch.l[j]);
            mine = ch.choose(key, nullptr);
        } else {
            bool close = false;
            float c[kPer];
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                const int e = j * 32 + lane;
                const float s = softmax ? expf(ch.l[j] - largest) / total : sigmoid_shifted(ch.l[j], 0.0f);
                c[j] = ch.l[j] == -kInf ? -kInf : s + (p.bias && e < p.E ? p.bias[e] : 0.0f);
            }
            const bool grouped = p.topk_groups < p.num_groups;
            if (grouped) {
                float* const mem = reinterpret_cast<float*>(smem + static_cast<size_t>(warp) * p.E);
#pragma unroll
                for (int j = 0; j < kPer; ++j)
                    if (j * 32 + lane < p.E) mem[j * 32 + lane] = c[j];
                __syncwarp();
                ch.keep_groups(mem, &close);
#pragma unroll
                for (int j = 0; j < kPer; ++j)
                    if (j * 32 + lane < p.E) c[j] = mem[j * 32 + lane];
                __syncwarp();
            }
            // without a bias the choice among the kept ones goes by the logits
#pragma unroll
            for (int j = 0; j < kPer; ++j) key[j] = c[j] == -kInf ? 0u : key_of(p.bias ? c[j] : ch.l[j]);
            bool near = false;
            mine = ch.choose(key, &near);
            if (close || (p.bias && near)) {
                double total64 = 0.0;
                if (softmax) {
#pragma unroll 1
                    for (int j = 0; j < kPer; ++j)
                        if (ch.l[j] != -kInf) total64 += exp(static_cast<double>(ch.l[j]) - largest);
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) total64 += __shfl_xor_sync(0xffffffffu, total64, o);
                }
                uint64_t key64[kPer];
                double c64[kPer];
#pragma unroll
                for (int j = 0; j < kPer; ++j) {
                    const int e = j * 32 + lane;
                    const double d = ch.l[j];
                    c64[j] = -kInf;
                    if (c[j] != -kInf || (grouped && ch.l[j] != -kInf)) {
                        const double s = softmax ? exp(d - largest) / total64 : 1.0 / (1.0 + exp(-d));
                        c64[j] = s + (p.bias && e < p.E ? static_cast<double>(p.bias[e]) : 0.0);
                    }
                }
                if (grouped) {
                    double* const mem = smem + static_cast<size_t>(warp) * p.E;
#pragma unroll
                    for (int j = 0; j < kPer; ++j)
                        if (j * 32 + lane < p.E) mem[j * 32 + lane] = c64[j];
                    __syncwarp();
                    ch.keep_groups(mem, nullptr);
#pragma unroll
                    for (int j = 0; j < kPer; ++j)
                        if (j * 32 + lane < p.E) c64[j] = mem[j * 32 + lane];
                    __syncwarp();
                }
#pragma unroll
                for (int j = 0; j < kPer; ++j)
                    key64[j] = c64[j] == -kInf ? 0ull : key_of(p.bias ? c64[j] : static_cast<double>(ch.l[j]));
                mine = ch.choose(key64, nullptr);
            }
        }
        // weights, by the lane of each slot
        const bool there = lane < p.K && mine >= 0;
        const float l = there ? to_float(row[mine]) : -kInf;
        float w;
        if (p.normalize) {
            const float top = warp_max(l);
            const float s = softmax ? (there ? expf(l - top) : 0.0f) : (there ? sigmoid_shifted(l, shift_of(top)) : 0.0f);
            const float sum = warp_sum(s);
            w = there ? s / sum * p.scale : 0.0f;
        } else {
            w = there ? (softmax ? expf(l - largest) / total : sigmoid_shifted(l, 0.0f)) * p.scale : 0.0f;
        }
        if (lane < p.K) {
            p.topk_idx[out + lane] = mine;
            p.topk_weights[out + lane] = w;
        }
    }
}

}  // namespace

cudaError_t launch_route(const RouteParams& p, cudaStream_t stream) {
    return with_row_type(p.dtype, p.E, [&](auto* type, auto per) {
        using L = std::remove_const_t<std::remove_pointer_t<decltype(type)>>;
        const bool grouped = p.topk_groups < p.num_groups;
        const size_t smem = grouped ? static_cast<size_t>(kWarps) * p.E * 8 : 0;
        const auto kernel = p.bias || grouped ? route_kernel<L, decltype(per)::value, true> : route_kernel<L, decltype(per)::value, false>;
        if (smem > 48 * 1024) {
            const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
            if (e != cudaSuccess) return e;
        }
        const int blocks = (p.T + kWarps - 1) / kWarps;
        return launch_pdl(kernel, dim3(blocks), dim3(kWarps * 32), smem, stream, p);
    });
}

}  // namespace epg
