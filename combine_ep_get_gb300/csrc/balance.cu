// The balance loss over the router's scores, and the gradient of the logits
// through the loss and through the weights of the chosen experts.
//
// With p the normalised scores of a token (softmax, or sigmoid over their sum),
// a sequence of n tokens has counts c_i and sums P_i of p_i over its tokens;
// its part of the loss is sum_i load_i P_i, load_i = coeff E c_i / (S K n^2), which
// is also the loss's derivative by each of its tokens' p_i.  Two kernels: the
// first adds scores and counts over tiles of tokens, cut where a sequence
// ends; the second adds the pieces of each sequence, eight experts a CTA and a
// fixed share of the pieces a thread, and its last CTA the sequences' parts.
// Every sum runs in an order that only the sizes decide.
//
// 32768 tokens of 256 experts, 8 chosen, inputs from memory: the loss 13.4 us for bf16 logits (1.5
// TB/s), the gradient through both 20 us for fp32 ones (3.5 TB/s): instructions
// of exponentials and sums bound both, and the loads and stores of 2 or 4
// bytes a lane.
#include <algorithm>
#include <type_traits>

#include "route_common.cuh"

namespace epg {

namespace {

constexpr int kThreads = kBalanceWarps * 32;

// exp(l - base) by the hardware's 2^x.
__device__ __forceinline__ float exp_below(float l, float base) { return exp2_approx((l - base) * kLog2E); }

__device__ __forceinline__ int clamped(int v, int n) { return v < 0 ? 0 : v > n ? n : v; }

// Scores of a row before they are divided by their sum, for a sigmoid 1 - score too; false for a row whose logits are
// all -inf.  *base: a softmax's q is exp(l - base) (the difference first: a product of either, rounded, is off by more
// than the exponent's range where logits are large), a sigmoid's is shifted by it.  Exponentials and reciprocals are
// the hardware's (sigmoid_fast): exact ones took half of the kernels' instructions.
template <bool kSoftmax, int kPer>
__device__ __forceinline__ bool scores_of(const float (&l)[kPer], float (&q)[kPer], float (&rest)[kPer], float* base) {
    float largest = l[0], any = 0.0f;      // any: NaN if one is
#pragma unroll
    for (int j = 0; j < kPer; ++j) largest = fmaxf(largest, l[j]);
    largest = warp_max(largest);
    if (largest == -kInf) {      // (a NaN is something, and stays one)
#pragma unroll
        for (int j = 0; j < kPer; ++j) any += l[j];
        if (!__any_sync(0xffffffffu, any != any)) return false;
    }
    *base = kSoftmax ? largest : shift_of(largest);
    if (kSoftmax) {
#pragma unroll
        for (int j = 0; j < kPer; ++j) q[j] = exp_below(l[j], *base);
    } else if (*base == 0.0f) {
#pragma unroll
        for (int j = 0; j < kPer; ++j) q[j] = sigmoid_fast(l[j], &rest[j]);
    } else {
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            q[j] = sigmoid_shifted(l[j], *base);
            rest[j] = sigmoid_shifted(-l[j], 0.0f);
        }
    }
    return true;
}

// What a token's work needs from memory, asked for while the token before is worked on.
template <typename L, int kPer, bool kFull>
struct Ahead {
    float l[kPer];
    int64_t named;      // the lane's slot
    float g;            // its derivative (the gradient)
    bool there;
    template <class P>
    __device__ __forceinline__ void ask(const P& p, int t, int lane, const int64_t* idx, const float* d_weights) {
        load_row<kPer, kFull>(static_cast<const L*>(p.logits) + t * p.row_stride, p.E, lane, l);
        there = !p.token_mask || p.token_mask[t] != 0;
        named = -1;
        g = 0.0f;
        if (lane < p.K) {
            const int64_t at = static_cast<int64_t>(t) * p.K + lane;
            if (idx) named = idx[at];
            if (d_weights) g = d_weights[at];
        }
    }
};

template <typename L, int kPer, bool kFull, bool kSoftmax>
__global__ void __launch_bounds__(kThreads) balance_sums_kernel(const BalanceParams p) {
    extern __shared__ float smem[];      // [kBalanceWarps][E] sums, [E] counts, tokens
    int* const count = reinterpret_cast<int*>(smem + kBalanceWarps * p.E);
    int* const tokens = count + p.E;
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    pdl_wait();
    pdl_launch_dependents();
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.arrived = 0;
    const int begin = blockIdx.x * p.tile_tokens, end = min(p.T, begin + p.tile_tokens);
    int q = warp_sequence_of(p.seq_offset, p.S, begin, lane);
    for (int at = begin; at < end;) {
        int stop = end;
        if (p.seq_offset) {
            if (q < p.S && p.seq_offset[q + 1] <= at) q = warp_sequence_of(p.seq_offset, p.S, at, lane);
            while (q < p.S && p.seq_offset[q + 1] <= at) ++q;      // (offsets that do not ascend: go on all the same)
            if (q >= p.S) break;
            stop = min(end, p.seq_offset[q + 1]);
            if (q < 0) {        // before the first sequence
                at = stop;
                continue;
            }
        }
        Ahead<L, kPer, kFull> ahead;
        if (at + warp < stop) ahead.ask(p, at + warp, lane, p.topk_idx, nullptr);
        for (int e = threadIdx.x; e < p.E; e += kThreads) count[e] = 0;
        if (threadIdx.x == 0) *tokens = 0;
        __syncthreads();
        float sum[kPer];
        int live = 0;
#pragma unroll
        for (int j = 0; j < kPer; ++j) sum[j] = 0.0f;
        for (int t = at + warp; t < stop; t += kBalanceWarps) {
            const Ahead<L, kPer, kFull> now = ahead;
            if (t + kBalanceWarps < stop) ahead.ask(p, t + kBalanceWarps, lane, p.topk_idx, nullptr);
            float s[kPer], rest[kPer], base;
            if (!now.there || !scores_of<kSoftmax>(now.l, s, rest, &base)) continue;
            float all = 0.0f;
#pragma unroll
            for (int j = 0; j < kPer; ++j) all += s[j];
            all = reciprocal_approx(warp_sum(all));
            ++live;
#pragma unroll
            for (int j = 0; j < kPer; ++j) sum[j] = fmaf(s[j], all, sum[j]);
            if (now.named >= 0 && now.named < p.E)
                atomicAdd(&count[now.named], 1);
            else if (now.named != -1)
                atomicOr(p.status, EP_ERR_INVALID_INDEX);
        }
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            if (kFull || j * 32 + lane < p.E) smem[warp * p.E + j * 32 + lane] = sum[j];
        if (lane == 0) atomicAdd(tokens, live);
        __syncthreads();
        const int64_t piece = blockIdx.x + q;
        if (EP_IN(piece, p.tiles + p.S)) {
            for (int e = threadIdx.x; e < p.E; e += kThreads) {
                float all = 0.0f;
#pragma unroll
                for (int w = 0; w < kBalanceWarps; ++w) all += smem[w * p.E + e];
                p.part[piece * p.E + e] = make_int2(__float_as_int(all), count[e]);
            }
            if (threadIdx.x == 0) p.part_tokens[piece] = *tokens;
        }
        __syncthreads();
        at = stop;
    }
}

// A CTA adds a sequence's pieces for eight experts: 32 bytes of scores' sums and as many of counts a piece, 128
// pieces at a time (32 experts a CTA, 32 pieces at a time, left it waiting for ten pieces one after another).
constexpr int kLossThreads = 1024, kLossWarps = kLossThreads / 32;

__global__ void __launch_bounds__(kLossThreads) balance_loss_kernel(const BalanceParams p) {
    __shared__ float sums[kLossWarps][kBalanceChunk];
    __shared__ int counts[kLossWarps][kBalanceChunk], live[kLossWarps];
    __shared__ bool last;
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, in_chunk = lane % kBalanceChunk;
    const int chunks = (p.E + kBalanceChunk - 1) / kBalanceChunk;
    const int q = blockIdx.x / chunks, e = blockIdx.x % chunks * kBalanceChunk + in_chunk;
    pdl_wait();
    pdl_launch_dependents();
    int first = 0, end = p.T;
    if (p.seq_offset) {
        const int a = p.seq_offset[q], b = p.seq_offset[q + 1];
        if ((a < 0 || a > b || b > p.T) && threadIdx.x == 0) atomicOr(p.status, EP_ERR_INVALID_INDEX);
        first = clamped(a, p.T);
        end = clamped(b, p.T);
    }
    const int tile0 = first / p.tile_tokens, tile1 = end > first ? (end - 1) / p.tile_tokens + 1 : tile0;
    float sum = 0.0f;
    int count = 0, n = 0;
#pragma unroll 4
    for (int tile = tile0 + threadIdx.x / kBalanceChunk; tile < tile1; tile += kLossThreads / kBalanceChunk) {
        const int64_t piece = tile + q;
        if (!EP_IN(piece, p.tiles + p.S)) continue;
        if (e < p.E) {
            const int2 part = p.part[piece * p.E + e];
            sum += __int_as_float(part.x);
            count += part.y;
        }
        if (in_chunk == 0) n += p.part_tokens[piece];
    }
    n = __reduce_add_sync(0xffffffffu, n);
#pragma unroll
    for (int o = kBalanceChunk; o < 32; o *= 2) {
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
        count += __shfl_xor_sync(0xffffffffu, count, o);
    }
    if (lane < kBalanceChunk) {
        sums[warp][lane] = sum;
        counts[warp][lane] = count;
    }
    if (lane == 0) live[warp] = n;
    __syncthreads();
    if (warp == 0) {
        sum = 0.0f;
        count = 0;
#pragma unroll
        for (int i = 0; i < kLossWarps; i += 32 / kBalanceChunk) {
            sum += sums[i + lane / kBalanceChunk][in_chunk];
            count += counts[i + lane / kBalanceChunk][in_chunk];
        }
#pragma unroll
        for (int o = kBalanceChunk; o < 32; o *= 2) {
            sum += __shfl_xor_sync(0xffffffffu, sum, o);
            count += __shfl_xor_sync(0xffffffffu, count, o);
        }
        n = __reduce_add_sync(0xffffffffu, live[lane]);
        const float tokens = static_cast<float>(n);
        const float load = n > 0 ? p.coeff * p.E / (static_cast<float>(p.S) * p.K) * (count / tokens) / tokens : 0.0f;
        const bool mine = lane < kBalanceChunk && e < p.E;
        if (mine && EP_IN(q, p.S)) {
            p.load[static_cast<int64_t>(q) * p.E + e] = load;
            if (p.counts) p.counts[static_cast<int64_t>(q) * p.E + e] = count;
        }
        const float loss = warp_sum(mine && n > 0 ? load * sum : 0.0f);
        if (lane == 0) {
            if (EP_IN(blockIdx.x, static_cast<int64_t>(p.S) * chunks)) p.part_loss[blockIdx.x] = loss;
            __threadfence();
            last = atomicAdd(p.arrived, 1u) == gridDim.x - 1;
        }
    }
    __syncthreads();
    if (!last) return;
    // shares of the parts by thread, then by warp
    __threadfence();
    float all = 0.0f;
    for (unsigned i = threadIdx.x; i < gridDim.x; i += kLossThreads) all += __ldcg(p.part_loss + i);
    all = warp_sum(all);
    if (lane == 0) sums[warp][0] = all;
    __syncthreads();
    if (warp == 0) {
        all = warp_sum(sums[lane][0]);
        if (lane == 0) *p.loss = all;
    }
}

template <typename L, int kPer, bool kFull, bool kSoftmax>
__global__ void __launch_bounds__(kThreads) route_backward_kernel(const RouteBackwardParams p) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    pdl_wait();
    pdl_launch_dependents();
    const float d_loss = p.load ? *p.d_loss : 0.0f;
    const int step = gridDim.x * kBalanceWarps, first = blockIdx.x * kBalanceWarps + warp;
    const int64_t* const idx = p.d_topk_weights ? p.topk_idx : nullptr;
    Ahead<L, kPer, kFull> ahead;
    float load[kPer];
    int load_of = -1;        // the sequence whose derivatives `load` holds
#pragma unroll
    for (int j = 0; j < kPer; ++j) load[j] = 0.0f;
    if (first < p.T) ahead.ask(p, first, lane, idx, p.d_topk_weights);
    for (int t = first; t < p.T; t += step) {
        const L* const row = static_cast<const L*>(p.logits) + t * p.row_stride;
        L* const out = static_cast<L*>(p.d_logits) + t * p.d_row_stride;
        const Ahead<L, kPer, kFull> now = ahead;
        if (t < p.T - step) ahead.ask(p, t + step, lane, idx, p.d_topk_weights);
        // the token's slots, a lane each, with their experts' logits
        int e = -1;
        float v = -kInf;
        if (now.there && now.named >= 0 && now.named < p.E) {
            e = static_cast<int>(now.named);
            if (EP_IN(t, p.T)) v = to_float(row[e]);
        } else if (now.there && now.named != -1) {
            atomicOr(p.status, EP_ERR_INVALID_INDEX);
        }
        const float g = v == -kInf ? 0.0f : now.g * p.scale;      // (whatever stands in a slot of no expert)
        __syncwarp();      // d_logits may be the logits: the slots' are read before another lane writes the row
        float s[kPer], rest[kPer], base;
        if (!now.there || !scores_of<kSoftmax>(now.l, s, rest, &base)) {
#pragma unroll
            for (int j = 0; j < kPer; ++j)
                if (kFull || j * 32 + lane < p.E) from_float(out + j * 32 + lane, 0.0f);
            continue;
        }
        // The loss's mean derivative, over the scores' sum.
        const int q = p.load ? warp_sequence_of(p.seq_offset, p.S, t, lane) : -1;
        const bool in_loss = q >= 0 && q < p.S && EP_IN(q, p.S);
        if (q != load_of) {
            load_of = q;
#pragma unroll
            for (int j = 0; j < kPer; ++j)
                load[j] = in_loss && (kFull || j * 32 + lane < p.E)
                              ? p.load[static_cast<int64_t>(q) * p.E + j * 32 + lane] * d_loss : 0.0f;
        }
        float inverse = 0.0f, mean = 0.0f;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            inverse += s[j];
            mean = fmaf(load[j], s[j], mean);
        }
        warp_sums(inverse, mean);
        inverse = reciprocal_approx(inverse);
        mean *= inverse;
        // Through the weights: the slots' lanes know their experts' whole derivative, and store it after the row's.
        float r = 0.0f;
        if (p.d_topk_weights) {
            if (p.normalize) {
                const float top = warp_max(v);
                const float u = v == -kInf ? 0.0f : kSoftmax ? exp_below(v, top) : sigmoid_shifted(v, shift_of(top));
                float sum = u, weighted = u * g;
                warp_sums(sum, weighted);
                const float over = reciprocal_approx(sum);
                r = u == 0.0f ? 0.0f : u * over * (g - weighted * over);
            } else if (v != -kInf) {
                r = (kSoftmax ? exp_below(v, base) * inverse : sigmoid_shifted(v, 0.0f)) * g;
            }
            if (kSoftmax && !p.normalize) mean += warp_sum(r);      // every expert loses its share of the chosen ones' sum
            if (!kSoftmax && e >= 0) r *= sigmoid_shifted(-v, 0.0f);
        }
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const float d = s[j] * inverse * (load[j] - mean);
            if (kFull || j * 32 + lane < p.E) from_float(out + j * 32 + lane, kSoftmax || !in_loss ? d : d * rest[j]);
        }
        if (p.d_topk_weights) {
            // an expert that is named twice gets both parts, in the order of the slots, from the first one's lane
            const unsigned same = __match_any_sync(0xffffffffu, e >= 0 ? e : -1 - lane);
            if (__any_sync(0xffffffffu, same & (same - 1))) {
                float sum = 0.0f;
                for (int k = 0; k < p.K; ++k) {
                    const float other = __shfl_sync(0xffffffffu, r, k);
                    if (same >> k & 1) sum += other;
                }
                r = sum;
            }
            __syncwarp();     // after the row's stores
            if (e >= 0 && (same & ((1u << lane) - 1)) == 0 && EP_IN(t, p.T) && EP_IN(e, p.E)) {
                const float a = in_loss ? p.load[static_cast<int64_t>(q) * p.E + e] * d_loss : 0.0f;
                float own = 0.0f;
                if (v == -kInf) {
                    own = 0.0f;
                } else if (kSoftmax) {
                    own = exp_below(v, base) * inverse * (a - mean);
                } else if (in_loss) {
                    float rest_e;
                    const float s_e = base == 0.0f ? sigmoid_fast(v, &rest_e) : sigmoid_shifted(v, base);
                    if (base != 0.0f) rest_e = sigmoid_shifted(-v, 0.0f);
                    own = s_e * inverse * (a - mean) * rest_e;
                }
                from_float(out + e, own + r);
            }
        }
    }
}

}  // namespace

cudaError_t launch_balance_loss(const BalanceParams& p, cudaStream_t stream) {
    const cudaError_t e = with_row_type(p.dtype, p.E, [&](auto* type, auto per, auto full) {
        using L = std::remove_const_t<std::remove_pointer_t<decltype(type)>>;
        constexpr int kPer = decltype(per)::value;
        constexpr bool kFull = decltype(full)::value;
        const auto kernel = p.score == EP_SCORE_SOFTMAX ? balance_sums_kernel<L, kPer, kFull, true>
                                                        : balance_sums_kernel<L, kPer, kFull, false>;
        const auto smem_of = [](int experts) { return (kBalanceWarps + 1) * experts * 4 + 16; };
        const size_t smem = smem_of(p.E);
        if (smem > 48 * 1024) {      // (the most that any call asks for: another thread's does not take it back)
            const cudaError_t err =
                cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_of(EP_MAX_EXPERTS));
            if (err != cudaSuccess) return err;
        }
        return launch_pdl(kernel, dim3(p.tiles > 0 ? p.tiles : 1), dim3(kThreads), smem, stream, p);
    });
    if (e != cudaSuccess) return e;
    const int chunks = (p.E + kBalanceChunk - 1) / kBalanceChunk;
    return launch_pdl(balance_loss_kernel, dim3(static_cast<unsigned>(p.S) * chunks), dim3(kLossThreads), 0, stream, p);
}

cudaError_t launch_route_backward(const RouteBackwardParams& p, cudaStream_t stream) {
    return with_row_type(p.dtype, p.E, [&](auto* type, auto per, auto full) {
        using L = std::remove_const_t<std::remove_pointer_t<decltype(type)>>;
        constexpr int kPer = decltype(per)::value;
        constexpr bool kFull = decltype(full)::value;
        const auto kernel = p.score == EP_SCORE_SOFTMAX ? route_backward_kernel<L, kPer, kFull, true>
                                                        : route_backward_kernel<L, kPer, kFull, false>;
        // (many tokens: warps that go on to another token have asked for its row)
        const int blocks = std::min((p.T + kBalanceWarps - 1) / kBalanceWarps, device_info().num_sms * 8);
        return launch_pdl(kernel, dim3(blocks), dim3(kThreads), 0, stream, p);
    });
}

}  // namespace epg
