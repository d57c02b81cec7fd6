// The experts' products with 4-bit weights and group scales.
//
// z[row, f] = sum over groups of scale[group, f] * sum over the group's k of (u[f, k] - zero[group, f]) x[row, k]
//
// A warp takes one feature (a pair of them for SWIGLU) and up to eight rows of
// one expert; its lanes share the sum.
#include "experts_w4.cuh"

namespace epg {

namespace {

constexpr int kWarps = 8, kRows = 8;

enum Mode { kProduct, kFewUp, kFewDown };

struct Args {
    const __nv_bfloat16* x;
    Weights4 w;
    const float* bias;
    int K, N, Nw, E, act;        // depth, features out, features of the weights
    // product
    const float* row_weight;
    const __nv_bfloat16* residual;
    int64_t rows;
    const int32_t* expert_offset;
    const int32_t* counts;
    // few tokens
    const int64_t* topk_idx;
    int T, topk;
    __nv_bfloat16* y;            // product: [rows][N]; up: h [T * topk][N]
    float* part;                 // down: [T * topk][N]
    int32_t* status;
};

__device__ __forceinline__ float scale_at(const Weights4& w, const void* from, int64_t i) {
    return w.sf_fp32 ? static_cast<const float*>(from)[i] : __bfloat162float(static_cast<const __nv_bfloat16*>(from)[i]);
}
__device__ __forceinline__ float code_value(uint32_t u, int format) {
    if (format == EP_W4_INT) return static_cast<float>(u);
    const uint32_t e = (u >> 1) & 3u, m = u & 1u;
    const float v = e == 0 ? 0.5f * m : (1.0f + 0.5f * m) * static_cast<float>(1u << (e - 1));
    return u & 8u ? -v : v;
}

template <Mode kMode>
__global__ void __launch_bounds__(kWarps * 32) experts_w4_kernel(const Args p) {
    extern __shared__ int smem[];     // [E] tile_end, first, count; few: list and expert of the entries
    int* const tile_end = smem;
    int* const first = tile_end + p.E;
    int* const count = first + p.E;
    int16_t* const list = reinterpret_cast<int16_t*>(count + p.E);
    __shared__ int warp_sum_mem[kWarps];
    __shared__ int64_t warp_rows[kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    constexpr int kThreads = kWarps * 32;
    pdl_wait();
    pdl_launch_dependents();
    if (kMode == kProduct) {
        expert_blocks<kThreads>(p.expert_offset, p.counts, p.E, p.rows, first, count, warp_rows, p.status);
    } else {
        const int entries = p.T * p.topk;
        for (int e = threadIdx.x; e < p.E; e += kThreads) count[e] = 0;
        __syncthreads();
        for (int i = threadIdx.x; i < entries; i += kThreads) {
            const int64_t e = p.topk_idx[i];
            if (e >= 0 && e < p.E)
                atomicAdd(&count[e], 1);
            else if (e != -1 && kMode == kFewUp && blockIdx.x == 0)
                atomicOr(p.status, EP_ERR_INVALID_INDEX);
        }
        __syncthreads();
        scan_experts<kThreads>(p.E, first, warp_sum_mem, [&](int e) { return count[e]; });
        // first[e] is where e's entries end; filled from the last one down, in
        // the order of (token, slot), it becomes where they begin: every CTA
        // has to give a tile the same rows
        if (warp == 0)
            for (int i0 = (entries - 1) / 32 * 32; i0 >= 0; i0 -= 32) {
                const int i = i0 + lane;
                const int64_t named = i < entries ? p.topk_idx[i] : -1;
                const int e = named >= 0 && named < p.E ? static_cast<int>(named) : -1;
                const unsigned same = __match_any_sync(0xffffffffu, e);
                if (e >= 0) list[first[e] - __popc(same >> lane)] = static_cast<int16_t>(i);
                __syncwarp();
                if (e >= 0 && (same >> lane) == 1u) first[e] -= __popc(same);
                __syncwarp();
            }
        __syncthreads();
    }
    scan_experts<kThreads>(p.E, tile_end, warp_sum_mem, [&](int e) { return (count[e] + kRows - 1) / kRows; });
    const int feature_tiles = (p.N + kWarps - 1) / kWarps;
    const int64_t tiles = static_cast<int64_t>(tile_end[p.E - 1]) * feature_tiles;
    for (int64_t g = blockIdx.x; g < tiles; g += gridDim.x) {
        const int row_tile = static_cast<int>(g / feature_tiles), f = static_cast<int>(g % feature_tiles) * kWarps + warp;
        int lo = 0, hi = p.E - 1;      // the expert: the first with tile_end > row_tile
        while (lo < hi) {
            const int mid = (lo + hi) / 2;
            if (tile_end[mid] > row_tile)
                hi = mid;
            else
                lo = mid + 1;
        }
        const int e = lo, r0 = (row_tile - (e > 0 ? tile_end[e - 1] : 0)) * kRows, n = min(kRows, count[e] - r0);
        if (f >= p.N) continue;
        int64_t out_row[kRows], x_row[kRows];
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const int at = first[e] + r0 + (r < n ? r : 0);
            out_row[r] = kMode == kProduct ? at : list[at];
            x_row[r] = kMode == kFewUp ? out_row[r] / p.topk : out_row[r];
        }
        const bool gated = p.act == EP_ACT_SWIGLU;
        float z[2][kRows];
        for (int half = 0; half < (gated ? 2 : 1); ++half) {
            const int feature = f + half * p.N;
            const uint32_t* const w = reinterpret_cast<const uint32_t*>(
                p.w.w + (static_cast<int64_t>(e) * p.Nw + feature) * (p.K / 2));
            const int groups = p.K / p.w.group;
            float acc[kRows] = {};
            for (int k = lane * 8; k < p.K; k += 256) {
                const uint32_t word = w[k / 8];
                const int64_t at = (static_cast<int64_t>(e) * groups + k / p.w.group) * p.Nw + feature;
                const float s = scale_at(p.w, p.w.sf, at);
                const float zero = p.w.format != EP_W4_INT ? 0.0f : p.w.zero ? scale_at(p.w, p.w.zero, at) : 8.0f;
                float v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = (code_value((word >> (4 * i)) & 15u, p.w.format) - zero) * s;
#pragma unroll
                for (int r = 0; r < kRows; ++r) {
                    if (r >= n) break;
                    const __nv_bfloat16* const x = p.x + x_row[r] * p.K + k;
#pragma unroll
                    for (int i = 0; i < 8; ++i) acc[r] = fmaf(v[i], __bfloat162float(x[i]), acc[r]);
                }
            }
            const float b = p.bias ? p.bias[static_cast<int64_t>(e) * p.Nw + feature] : 0.0f;
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                float sum = acc[r];
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                z[half][r] = sum + b;
            }
        }
        if (lane != 0) continue;
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            if (r >= n) break;
            const float a = gated ? silu(z[0][r]) * z[1][r] : activate(z[0][r], p.act);
            const int64_t at = out_row[r] * p.N + f;
            if (kMode == kProduct) {
                float v = a;
                if (p.row_weight) v *= p.row_weight[out_row[r]];
                if (p.residual) v += __bfloat162float(p.residual[at]);
                p.y[at] = __float2bfloat16_rn(v);
            } else if (kMode == kFewUp) {
                p.y[at] = __float2bfloat16_rn(a);
            } else {
                p.part[at] = a;
            }
        }
    }
}

// out[t] = residual[t] + sum over k ascending of weight * part[t, k]
__global__ void __launch_bounds__(256) few_sum_kernel(const FewTokensW4Params p) {
    pdl_wait();
    pdl_launch_dependents();
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= static_cast<int64_t>(p.T) * p.H) return;
    const int t = static_cast<int>(i / p.H), f = static_cast<int>(i % p.H);
    float sum = 0.0f;
    for (int k = 0; k < p.K; ++k) {
        const int64_t e = p.topk_idx[t * p.K + k];
        if (e >= 0 && e < p.E) sum = fmaf(p.topk_weights[t * p.K + k], p.part[(static_cast<int64_t>(t) * p.K + k) * p.H + f], sum);
    }
    if (p.residual) sum += __bfloat162float(p.residual[i]);
    p.out[i] = __float2bfloat16_rn(sum);
}

template <Mode kMode>
cudaError_t launch(const Args& a, int64_t tiles_bound, cudaStream_t stream) {
    const size_t smem = static_cast<size_t>(a.E) * 12 + static_cast<size_t>(a.T) * a.topk * 2;
    const int64_t blocks = std::max<int64_t>(1, std::min<int64_t>(tiles_bound, device_info().num_sms * 8));
    return launch_pdl(experts_w4_kernel<kMode>, dim3(static_cast<unsigned>(blocks)), dim3(kWarps * 32), smem, stream, a);
}

}  // namespace

cudaError_t launch_expert_gemm_w4(const ExpertGemmW4Params& p, cudaStream_t stream) {
    Args a{};
    a.x = p.x;
    a.w = p.w;
    a.bias = p.bias;
    a.K = p.K;
    a.N = p.N;
    a.Nw = p.Nw;
    a.E = p.E;
    a.act = p.act;
    a.row_weight = p.row_weight;
    a.residual = p.residual;
    a.rows = p.rows;
    a.expert_offset = p.expert_offset;
    a.counts = p.counts;
    a.y = p.y;
    a.status = p.status;
    return launch<kProduct>(a, (p.rows / kRows + p.E) * ((p.N + kWarps - 1) / kWarps), stream);
}

cudaError_t launch_few_tokens_w4(const FewTokensW4Params& p, cudaStream_t stream) {
    Args a{};
    a.x = p.x;
    a.w = p.up;
    a.bias = p.bias_up;
    a.K = p.H;
    a.N = p.I;
    a.Nw = p.Nw;
    a.E = p.E;
    a.act = p.act;
    a.topk_idx = p.topk_idx;
    a.T = p.T;
    a.topk = p.K;
    a.y = p.h;
    a.status = p.status;
    const int64_t row_tiles = p.T * p.K / kRows + std::min(p.E, p.T * p.K);
    cudaError_t e = launch<kFewUp>(a, row_tiles * ((p.I + kWarps - 1) / kWarps), stream);
    if (e != cudaSuccess) return e;
    a.x = p.h;
    a.w = p.down;
    a.bias = p.bias_down;
    a.K = p.I;
    a.N = a.Nw = p.H;
    a.act = EP_ACT_NONE;
    a.y = nullptr;
    a.part = p.part;
    e = launch<kFewDown>(a, row_tiles * ((p.H + kWarps - 1) / kWarps), stream);
    if (e != cudaSuccess) return e;
    const int64_t outs = static_cast<int64_t>(p.T) * p.H;
    return launch_pdl(few_sum_kernel, dim3(static_cast<unsigned>((outs + 255) / 256)), dim3(256), 0, stream, p);
}

}  // namespace epg
