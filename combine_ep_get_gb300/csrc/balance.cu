// The balance loss over the router's scores, and the gradient of the logits
// through the loss and through the weights of the chosen experts.
//
// With p the normalised scores of a token (softmax, or sigmoid over their sum),
// a sequence of n tokens has counts c_i and sums P_i of p_i over its tokens;
// its part of the loss is sum_i load_i P_i, load_i = coeff E c_i / (S K n^2), which
// is also the loss's derivative by each of its tokens' p_i.  Two kernels: the
// first adds scores and counts over tiles of tokens, cut where a sequence
// ends; the second adds the pieces of each sequence in their order, 32 experts
// a CTA, and its last CTA the sequences' parts.  Every sum runs in an order
// that only the sizes decide.
#include <algorithm>
#include <type_traits>

#include "route_common.cuh"

namespace epg {

namespace {

constexpr int kThreads = kBalanceWarps * 32;

__device__ __forceinline__ int clamped(int v, int n) { return v < 0 ? 0 : v > n ? n : v; }

// Scores of a row as parts of their sum, for a sigmoid 1 - score too; false for a row whose logits are all -inf.
// *base and *inverse: a softmax's q is 2^(log2(e) l - base) * inverse; a sigmoid's base is its shift.  Exponentials and reciprocals are the hardware's
// (sigmoid_fast): exact ones took half of the kernels' instructions.
template <int kPer>
__device__ __forceinline__ bool normalised_scores(const float (&l)[kPer], int score, float (&q)[kPer], float (&rest)[kPer],
                                                  float* base, float* inverse) {
    float largest = l[0];
    bool nan = l[0] != l[0];
#pragma unroll
    for (int j = 1; j < kPer; ++j) {
        largest = fmaxf(largest, l[j]);
        nan |= l[j] != l[j];
    }
    largest = warp_max(largest);
    // (a NaN is something, and stays one)
    if (largest == -kInf && !__any_sync(0xffffffffu, nan)) return false;
    float sum = 0.0f;
    *base = score == EP_SCORE_SOFTMAX ? largest * kLog2E : shift_of(largest);
    if (score == EP_SCORE_SOFTMAX) {
#pragma unroll
        for (int j = 0; j < kPer; ++j) sum += q[j] = exp2_approx(fmaf(l[j], kLog2E, -*base));
    } else if (*base == 0.0f) {
#pragma unroll
        for (int j = 0; j < kPer; ++j) sum += q[j] = sigmoid_fast(l[j], &rest[j]);
    } else {
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            sum += q[j] = sigmoid_shifted(l[j], *base);
            rest[j] = sigmoid_shifted(-l[j], 0.0f);
        }
    }
    *inverse = 1.0f / warp_sum(sum);
#pragma unroll
    for (int j = 0; j < kPer; ++j) q[j] *= *inverse;
    return true;
}

template <typename L, int kPer>
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
            while (q < p.S && p.seq_offset[q + 1] <= at) ++q;
            if (q >= p.S) break;
            stop = min(end, p.seq_offset[q + 1]);
            if (q < 0) {        // before the first sequence
                at = stop;
                continue;
            }
        }
        for (int e = threadIdx.x; e < p.E; e += kThreads) count[e] = 0;
        if (threadIdx.x == 0) *tokens = 0;
        __syncthreads();
        float sum[kPer];
        int live = 0;
#pragma unroll
        for (int j = 0; j < kPer; ++j) sum[j] = 0.0f;
        constexpr bool kAhead = kPer <= 16;      // the next row is asked for before this one's work
        const L* const logits = static_cast<const L*>(p.logits);
        float ahead[kPer];
        if (kAhead && at + warp < stop) load_row(logits + (at + warp) * p.row_stride, p.E, lane, ahead);
        for (int t = at + warp; t < stop; t += kBalanceWarps) {
            float l[kPer], s[kPer], rest[kPer], base, inverse;
            if constexpr (kAhead) {
#pragma unroll
                for (int j = 0; j < kPer; ++j) l[j] = ahead[j];
                if (t + kBalanceWarps < stop) load_row(logits + (t + kBalanceWarps) * p.row_stride, p.E, lane, ahead);
            } else {
                load_row(logits + t * p.row_stride, p.E, lane, l);
            }
            if (p.token_mask && p.token_mask[t] == 0) continue;
            if (!normalised_scores(l, p.score, s, rest, &base, &inverse)) continue;
            ++live;
#pragma unroll
            for (int j = 0; j < kPer; ++j) sum[j] += s[j];
            if (lane < p.K) {
                const int64_t e = p.topk_idx[static_cast<int64_t>(t) * p.K + lane];
                if (e >= 0 && e < p.E)
                    atomicAdd(&count[e], 1);
                else if (e != -1)
                    atomicOr(p.status, EP_ERR_INVALID_INDEX);
            }
        }
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            if (j * 32 + lane < p.E) smem[warp * p.E + j * 32 + lane] = sum[j];
        if (lane == 0) atomicAdd(tokens, live);
        __syncthreads();
        const int64_t piece = blockIdx.x + q;
        if (EP_IN(piece, p.tiles + p.S)) {
            for (int e = threadIdx.x; e < p.E; e += kThreads) {
                float all = 0.0f;
#pragma unroll
                for (int w = 0; w < kBalanceWarps; ++w) all += smem[w * p.E + e];
                p.part_sum[piece * p.E + e] = all;
                p.part_count[piece * p.E + e] = count[e];
            }
            if (threadIdx.x == 0) p.part_tokens[piece] = *tokens;
        }
        __syncthreads();
        at = stop;
    }
}

constexpr int kParts = 32;       // shares of a sequence's pieces, one warp each

__global__ void __launch_bounds__(kParts * 32) balance_loss_kernel(const BalanceParams p) {
    __shared__ float sums[kParts][33];
    __shared__ int counts[kParts][33], live[kParts];
    __shared__ bool last;
    const int lane = threadIdx.x & 31, part = threadIdx.x / 32;
    const int chunks = (p.E + kBalanceChunk - 1) / kBalanceChunk;
    const int q = blockIdx.x / chunks, e = blockIdx.x % chunks * kBalanceChunk + lane;
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
    for (int tile = tile0 + part; tile < tile1; tile += kParts) {
        const int64_t piece = tile + q;
        if (!EP_IN(piece, p.tiles + p.S)) continue;
        if (e < p.E) {
            sum += p.part_sum[piece * p.E + e];
            count += p.part_count[piece * p.E + e];
        }
        n += p.part_tokens[piece];
    }
    sums[part][lane] = sum;
    counts[part][lane] = count;
    if (lane == 0) live[part] = n;
    __syncthreads();
    if (part == 0) {
        sum = 0.0f;
        count = n = 0;
        for (int i = 0; i < kParts; ++i) {
            sum += sums[i][lane];
            count += counts[i][lane];
            n += live[i];
        }
        const float tokens = static_cast<float>(n);
        const float load = n > 0 ? p.coeff * p.E / (static_cast<float>(p.S) * p.K) * (count / tokens) / tokens : 0.0f;
        if (e < p.E) {
            p.load[static_cast<int64_t>(q) * p.E + e] = load;
            if (p.counts) p.counts[static_cast<int64_t>(q) * p.E + e] = count;
        }
        const float loss = warp_sum(e < p.E && n > 0 ? load * sum : 0.0f);
        if (lane == 0) {
            p.part_loss[blockIdx.x] = loss;
            __threadfence();
            last = atomicAdd(p.arrived, 1u) == gridDim.x - 1;
        }
    }
    __syncthreads();
    if (!last) return;
    // shares of the parts by thread, then by warp
    __threadfence();
    float all = 0.0f;
    for (unsigned i = threadIdx.x; i < gridDim.x; i += kParts * 32) all += __ldcg(p.part_loss + i);
    all = warp_sum(all);
    if (lane == 0) sums[part][0] = all;
    __syncthreads();
    if (part == 0) {
        all = warp_sum(sums[lane][0]);
        if (lane == 0) *p.loss = all;
    }
}

template <typename L, int kPer>
__global__ void __launch_bounds__(kThreads) route_backward_kernel(const RouteBackwardParams p) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    pdl_wait();
    pdl_launch_dependents();
    const bool softmax = p.score == EP_SCORE_SOFTMAX;
    const float d_loss = p.load ? *p.d_loss : 0.0f;
    constexpr bool kAhead = kPer <= 16;      // the next row is asked for before this one's work
    const int step = gridDim.x * kBalanceWarps, first = blockIdx.x * kBalanceWarps + warp;
    const L* const logits = static_cast<const L*>(p.logits);
    float ahead[kPer], load[kPer];
    int load_of = -1;        // the sequence whose derivatives `load` holds
#pragma unroll
    for (int j = 0; j < kPer; ++j) load[j] = 0.0f;
    if (kAhead && first < p.T) load_row(logits + first * p.row_stride, p.E, lane, ahead);
    for (int t = first; t < p.T; t += step) {
        const L* const row = logits + t * p.row_stride;
        L* const out = static_cast<L*>(p.d_logits) + t * p.d_row_stride;
        float l[kPer], s[kPer], rest[kPer], d[kPer], base, inverse;
        if constexpr (kAhead) {
#pragma unroll
            for (int j = 0; j < kPer; ++j) l[j] = ahead[j];
            if (t < p.T - step) load_row(row + step * p.row_stride, p.E, lane, ahead);
        } else {
            load_row(row, p.E, lane, l);
        }
        // the token's slots, a lane each, with their experts' logits
        int e = -1;
        float g = 0.0f, v = -kInf;
        if (p.d_topk_weights && lane < p.K) {
            const int64_t at = static_cast<int64_t>(t) * p.K + lane, named = p.topk_idx[at];
            if (named >= 0 && named < p.E) {
                e = static_cast<int>(named);
                g = p.d_topk_weights[at] * p.scale;
                v = to_float(row[e]);
            } else if (named != -1) {
                atomicOr(p.status, EP_ERR_INVALID_INDEX);
            }
        }
        if ((p.token_mask && p.token_mask[t] == 0) || !normalised_scores(l, p.score, s, rest, &base, &inverse)) {
#pragma unroll
            for (int j = 0; j < kPer; ++j)
                if (j * 32 + lane < p.E) from_float(out + j * 32 + lane, 0.0f);
            continue;
        }
        // through the loss
        float mean = 0.0f;
        const int q = p.load ? warp_sequence_of(p.seq_offset, p.S, t, lane) : -1;
        const bool in_loss = q >= 0 && q < p.S;
        if (in_loss) {
            if (q != load_of) {
                load_of = q;
#pragma unroll
                for (int j = 0; j < kPer; ++j)
                    load[j] = j * 32 + lane < p.E ? p.load[static_cast<int64_t>(q) * p.E + j * 32 + lane] * d_loss : 0.0f;
            }
#pragma unroll
            for (int j = 0; j < kPer; ++j) mean += load[j] * s[j];
            mean = warp_sum(mean);
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                d[j] = s[j] * (load[j] - mean);
                if (!softmax) d[j] *= rest[j];
            }
        } else {
#pragma unroll
            for (int j = 0; j < kPer; ++j) d[j] = 0.0f;
        }
        // Through the weights: the slots' lanes know their experts' whole derivative, and store it after the row's.
        float r = 0.0f;
        if (p.d_topk_weights) {
            const float top = warp_max(v);
            if (p.normalize) {
                const float u = v == -kInf ? 0.0f : softmax ? exp2_approx((v - top) * kLog2E) : sigmoid_shifted(v, shift_of(top));
                const float sum = warp_sum(u), part = u == 0.0f ? 0.0f : u / sum;
                r = part * (g - warp_sum(part * g));
            } else if (v != -kInf) {
                r = (softmax ? exp2_approx(fmaf(v, kLog2E, -base)) * inverse : sigmoid_shifted(v, 0.0f)) * g;
            }
            if (softmax && !p.normalize) {
                // every expert loses its share of the chosen ones' sum
                const float spread = warp_sum(r);
                mean += spread;
#pragma unroll
                for (int j = 0; j < kPer; ++j) d[j] -= s[j] * spread;
            }
            if (!softmax && e >= 0) r *= sigmoid_shifted(-v, 0.0f);
        }
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            if (j * 32 + lane < p.E) from_float(out + j * 32 + lane, d[j]);
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
            if (e >= 0 && (same & ((1u << lane) - 1)) == 0) {
                float own = 0.0f;
                if (v == -kInf) {
                    own = 0.0f;
                } else if (softmax) {
                    const float s_e = exp2_approx(fmaf(v, kLog2E, -base)) * inverse;
                    own = s_e * ((in_loss ? p.load[static_cast<int64_t>(q) * p.E + e] * d_loss : 0.0f) - mean);
                } else if (in_loss) {
                    float rest_e;
                    const float s_e = (base == 0.0f ? sigmoid_fast(v, &rest_e) : sigmoid_shifted(v, base)) * inverse;
                    if (base != 0.0f) rest_e = sigmoid_shifted(-v, 0.0f);
                    own = s_e * (p.load[static_cast<int64_t>(q) * p.E + e] * d_loss - mean) * rest_e;
                }
                from_float(out + e, own + r);
            }
        }
    }
}

}  // namespace

cudaError_t launch_balance_loss(const BalanceParams& p, cudaStream_t stream) {
    const cudaError_t e = with_row_type(p.dtype, p.E, [&](auto* type, auto per) {
        using L = std::remove_const_t<std::remove_pointer_t<decltype(type)>>;
        const auto kernel = balance_sums_kernel<L, decltype(per)::value>;
        const size_t smem = static_cast<size_t>(kBalanceWarps + 1) * p.E * 4 + 16;
        if (smem > 48 * 1024) {
            const cudaError_t err =
                cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
            if (err != cudaSuccess) return err;
        }
        return launch_pdl(kernel, dim3(p.tiles > 0 ? p.tiles : 1), dim3(kThreads), smem, stream, p);
    });
    if (e != cudaSuccess) return e;
    const int chunks = (p.E + kBalanceChunk - 1) / kBalanceChunk;
    return launch_pdl(balance_loss_kernel, dim3(static_cast<unsigned>(p.S) * chunks), dim3(kParts * 32), 0, stream, p);
}

cudaError_t launch_route_backward(const RouteBackwardParams& p, cudaStream_t stream) {
    return with_row_type(p.dtype, p.E, [&](auto* type, auto per) {
        using L = std::remove_const_t<std::remove_pointer_t<decltype(type)>>;
        const auto kernel = route_backward_kernel<L, decltype(per)::value>;
        // (many tokens: warps that go on to another token have asked for its row)
        const int blocks = std::min((p.T + kBalanceWarps - 1) / kBalanceWarps, device_info().num_sms * 8);
        return launch_pdl(kernel, dim3(blocks), dim3(kThreads), 0, stream, p);
    });
}

}  // namespace epg
