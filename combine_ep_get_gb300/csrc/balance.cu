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
#include <type_traits>

#include "route_common.cuh"

namespace epg {

namespace {

constexpr int kThreads = kBalanceWarps * 32;

__device__ __forceinline__ int clamped(int v, int n) { return v < 0 ? 0 : v > n ? n : v; }

// Scores of a row as parts of their sum, with the largest logit and (softmax)
// the sum of exponentials; false for a row whose logits are all -inf.
template <int kPer>
__device__ __forceinline__ bool normalised_scores(const float (&l)[kPer], int score, float (&q)[kPer], float& largest,
                                                  float& sum) {
    largest = -kInf;
    bool any = false;      // (a NaN is something, and stays one)
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        largest = fmaxf(largest, l[j]);
        any |= l[j] != -kInf;
    }
    if (!__any_sync(0xffffffffu, any)) return false;
    largest = warp_max(largest);
    sum = 0.0f;
    if (score == EP_SCORE_SOFTMAX) {
#pragma unroll
        for (int j = 0; j < kPer; ++j) sum += q[j] = expf(l[j] - largest);
    } else {
        const float shift = shift_of(largest);
#pragma unroll
        for (int j = 0; j < kPer; ++j) sum += q[j] = sigmoid_shifted(l[j], shift);
    }
    sum = warp_sum(sum);
#pragma unroll
    for (int j = 0; j < kPer; ++j) q[j] /= sum;
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
    int q = p.seq_offset ? sequence_of(p.seq_offset, p.S, begin) : 0;
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
        for (int t = at + warp; t < stop; t += kBalanceWarps) {
            if (p.token_mask && p.token_mask[t] == 0) continue;
            float l[kPer], s[kPer], largest, all;
            load_row(static_cast<const L*>(p.logits) + t * p.row_stride, p.E, lane, l);
            if (!normalised_scores(l, p.score, s, largest, all)) continue;
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
    extern __shared__ float smem[];      // [kBalanceWarps][E]: the chosen experts' parts of a row
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    float* const chosen = smem + warp * p.E;
    pdl_wait();
    pdl_launch_dependents();
    const bool softmax = p.score == EP_SCORE_SOFTMAX;
    const float d_loss = p.load ? *p.d_loss : 0.0f;
    for (int e = lane; e < p.E; e += 32) chosen[e] = 0.0f;
    __syncwarp();
    for (int t = blockIdx.x * kBalanceWarps + warp; t < p.T; t += gridDim.x * kBalanceWarps) {
        L* const out = static_cast<L*>(p.d_logits) + t * p.d_row_stride;
        const L* const row = static_cast<const L*>(p.logits) + t * p.row_stride;
        float l[kPer], s[kPer], d[kPer], largest = 0.0f, total = 1.0f;
        bool live = !p.token_mask || p.token_mask[t] != 0;
        if (live) {
            load_row(row, p.E, lane, l);
            live = normalised_scores(l, p.score, s, largest, total);
        }
        if (!live) {
#pragma unroll
            for (int j = 0; j < kPer; ++j)
                if (j * 32 + lane < p.E) from_float(out + j * 32 + lane, 0.0f);
            continue;
        }
        // through the loss
#pragma unroll
        for (int j = 0; j < kPer; ++j) d[j] = 0.0f;
        const int q = p.load ? sequence_of(p.seq_offset, p.S, t) : -1;
        if (q >= 0 && q < p.S) {
            float mean = 0.0f;
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                const int e = j * 32 + lane;
                if (e < p.E) d[j] = p.load[static_cast<int64_t>(q) * p.E + e] * d_loss;
                mean += d[j] * s[j];
            }
            mean = warp_sum(mean);
#pragma unroll
            for (int j = 0; j < kPer; ++j) d[j] = s[j] * (d[j] - mean);
        }
        // through the weights, by the lane of each slot
        float spread = 0.0f;      // softmax without normalisation: every expert's share of the chosen ones' sum
        if (p.d_topk_weights) {
            int e = -1;
            float g = 0.0f, v = -kInf;
            if (lane < p.K) {
                const int64_t at = static_cast<int64_t>(t) * p.K + lane;
                const int64_t named = p.topk_idx[at];
                if (named >= 0 && named < p.E) {
                    e = static_cast<int>(named);
                    g = p.d_topk_weights[at] * p.scale;
                    v = to_float(row[e]);
                } else if (named != -1) {
                    atomicOr(p.status, EP_ERR_INVALID_INDEX);
                }
            }
            const float top = warp_max(v);
            float r = 0.0f;
            if (p.normalize) {
                const float u = v == -kInf ? 0.0f : softmax ? expf(v - top) : sigmoid_shifted(v, shift_of(top));
                const float sum = warp_sum(u), part = u == 0.0f ? 0.0f : u / sum;
                r = part * (g - warp_sum(part * g));
            } else if (softmax) {
                r = v == -kInf ? 0.0f : expf(v - largest) / total * g;
                spread = warp_sum(r);
            } else if (v != -kInf) {
                r = sigmoid_shifted(v, 0.0f) * g;
            }
            if (!softmax && e >= 0) r *= sigmoid_shifted(-v, 0.0f);
            // an expert that is named twice gets both parts, in the order of the slots
            float sum = 0.0f;
            bool first = true;
            for (int k = 0; k < p.K; ++k) {
                const int ek = __shfl_sync(0xffffffffu, e, k);
                const float rk = __shfl_sync(0xffffffffu, r, k);
                if (ek == e) {
                    sum += rk;
                    if (k < lane) first = false;
                }
            }
            if (e >= 0 && first) chosen[e] = sum;
            __syncwarp();
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                const int ej = j * 32 + lane;
                if (ej < p.E) {
                    const float c = chosen[ej];
                    d[j] = softmax ? d[j] + c - s[j] * spread : sigmoid_shifted(-l[j], 0.0f) * d[j] + c;
                    if (c != 0.0f || c != c) chosen[ej] = 0.0f;
                }
            }
            __syncwarp();
        } else if (!softmax) {
#pragma unroll
            for (int j = 0; j < kPer; ++j) d[j] *= sigmoid_shifted(-l[j], 0.0f);
        }
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            if (j * 32 + lane < p.E) from_float(out + j * 32 + lane, d[j]);
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
        const size_t smem = static_cast<size_t>(kBalanceWarps) * p.E * 4;
        if (smem > 48 * 1024) {
            const cudaError_t err =
                cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
            if (err != cudaSuccess) return err;
        }
        const int blocks = (p.T + kBalanceWarps - 1) / kBalanceWarps;
        return launch_pdl(kernel, dim3(blocks), dim3(kThreads), smem, stream, p);
    });
}

}  // namespace epg
