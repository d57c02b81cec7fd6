// Parameter blocks and launchers of the experts' operators (experts*.cu).
#pragma once

#include <atomic>

#include <cuda_bf16.h>

#include "ep_internal.cuh"

namespace epg {

constexpr int kMaxExpertDim = 1 << 20;

struct ExpertGemmParams {
    const uint8_t* x;            // [rows][K] bf16 or E4M3 codes
    const float* x_sf;           // FP8: element (d, b) at d * sf_row + b * sf_block
    int64_t sf_row, sf_block;
    const uint8_t* w;            // [E][Nw][K]
    const float* w_sf;           // FP8: [E][Nw / 128][K / 128]
    const float* bias;           // [E][Nw] or null
    const float* row_weight;     // [rows] or null
    const __nv_bfloat16* residual;   // [rows][N] or null
    int64_t rows;
    int K, N, Nw, E, act;
    const int32_t* expert_offset;    // [E]
    const int32_t* counts;           // [E]
    __nv_bfloat16* y;            // [rows][N]
    __nv_bfloat16* z;            // [rows][Nw] or null
    int32_t* status;
};

struct ExpertBackwardParams {
    const __nv_bfloat16* dy;     // [rows][N]
    const __nv_bfloat16* x;      // [rows][K]
    const __nv_bfloat16* w;      // [E][Nw][K]
    const __nv_bfloat16* z;      // [rows][Nw]
    const float* row_weight;     // [rows] or null
    int64_t rows;
    int K, N, Nw, E, act;
    const int32_t* expert_offset;
    const int32_t* counts;
    __nv_bfloat16* dx;           // [rows][K] or null
    __nv_bfloat16* dw;           // [E][Nw][K] or null
    float* dbias;                // [E][Nw] or null
    float* d_row_weight;         // [rows] or null
    __nv_bfloat16* dz;           // workspace [rows][Nw]
    float* bias_part;            // workspace [row tiles][Nw]: sums of dz over a tile's rows
    float* weight_part;          // workspace [strips][rows]: sums of dy * a over a strip's columns
    int* blocks_fit;             // workspace: expert_blocks' answer, for the kernel that adds the partial sums
    int32_t* status;
};

struct FewTokensParams {
    const __nv_bfloat16* x;      // [T][H]
    const int64_t* topk_idx;     // [T][K]
    const float* topk_weights;   // [T][K]
    const __nv_bfloat16* w_up;   // [E][Nw][H]
    const float* bias_up;        // [E][Nw] or null
    const __nv_bfloat16* w_down; // [E][H][I]
    const float* bias_down;      // [E][H] or null
    const __nv_bfloat16* residual;   // [T][H] or null
    int T, H, I, Nw, K, E, act;
    __nv_bfloat16* h;            // workspace [T * K][I], expert by expert
    float* part;                 // workspace [T * K][H]
    uint32_t* done;              // workspace [H / 128, rounded up][T]
    __nv_bfloat16* out;          // [T][H]
    int32_t* status;
};

cudaError_t launch_expert_backward(const ExpertBackwardParams& p, cudaStream_t stream);
cudaError_t launch_few_tokens(const FewTokensParams& p, cudaStream_t stream);
// The parts of these on the tensor cores.
cudaError_t launch_expert_gemm_fp8(const ExpertGemmParams& p, cudaStream_t stream);
cudaError_t launch_expert_gemm_bf16(const ExpertGemmParams& p, cudaStream_t stream);
cudaError_t launch_input_grad(const ExpertBackwardParams& p, const __nv_bfloat16* dz, bool wait_late,
                              cudaStream_t stream);
cudaError_t launch_weight_grad(const ExpertBackwardParams& p, const __nv_bfloat16* dz, bool wait_late,
                               cudaStream_t stream);

// Lets a kernel use all the shared memory a block may have, once for a device
// (`done` is the kernel's own; a second thread that does it too does no harm).
constexpr int kMaxDevices = 64;
inline cudaError_t allow_all_smem(const void* kernel, std::atomic<bool>* done) {
    const DeviceInfo& info = device_info();
    const bool known = info.device >= 0 && info.device < kMaxDevices;
    if (known && done[info.device].load(std::memory_order_acquire)) return cudaSuccess;
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, info.max_smem_optin);
    if (e == cudaSuccess && known) done[info.device].store(true, std::memory_order_release);
    return e;
}

// Reads before the wait.  Three of the experts' kernels read before their
// griddepcontrol.wait: the few-token layer's down kernel (topk_idx, w_down) and
// both products of the gradients where another kernel of the call stands
// between them and dz's (dz, x, w, the blocks).  All of it was complete before
// that kernel, whose threads wait before they let the next one start (or, for
// the second product, before they let the first one start): what a wait has
// seen end is in L2.  There the early reads go, by tensor maps or __ldcg, never
// through an L1 that an earlier launch may have filled.  What the kernel just
// before writes (h, the sums) is read after the wait or not at all, and every
// kernel waits before it ends, so a kernel that waits for the last one of a
// call waits for all of them.  (With every wait at the start: gradients of
// 5005 rows over 40 experts 90.9 -> 97.8 us, one token's layer 116.6 -> 120.4.)

// launch_pdl with clusters of `cluster` CTAs.
template <typename... KArgs, typename... Args>
cudaError_t launch_experts(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                           int cluster, Args&&... args) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    if (debug_enabled()) debug_launch(reinterpret_cast<const void*>(kernel), grid, block, smem, cluster);
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// Workspace carve-ups shared by the size queries and the calls.
constexpr int kBackwardTileRows = 32;   // rows of one partial column sum of dz
constexpr int kBackwardStrip = 256;     // columns of one partial row sum
struct BackwardWorkspace {
    size_t off_dz, off_part, off_weight, off_fit, total;
};
inline BackwardWorkspace backward_workspace(int64_t rows, int N, int Nw, int E) {
    const auto up = [](size_t v) { return (v + 255) / 256 * 256; };
    const size_t tiles = static_cast<size_t>(rows) / kBackwardTileRows + E;
    BackwardWorkspace b;
    b.off_dz = 0;
    b.off_part = up(static_cast<size_t>(rows) * Nw * 2);
    b.off_weight = b.off_part + up(tiles * Nw * 4);
    b.off_fit = b.off_weight + up((static_cast<size_t>(N) + kBackwardStrip - 1) / kBackwardStrip * rows * 4);
    b.total = b.off_fit + 256;
    return b;
}
struct FewWorkspace {
    size_t off_h, off_part, off_done, total;
};
inline FewWorkspace few_workspace(int T, int K, int H, int I) {
    const auto up = [](size_t v) { return (v + 255) / 256 * 256; };
    FewWorkspace f;
    f.off_h = 0;
    f.off_part = up(static_cast<size_t>(T) * K * I * 2);
    f.off_done = f.off_part + up(static_cast<size_t>(T) * K * H * 4);
    f.total = f.off_done + up((static_cast<size_t>(H) + 127) / 128 * T * 4) + 256;
    return f;
}

// The activation of a pre-activation z (the gated one takes gate and up).
// 2^x and 1/x as the hardware gives them, to 2^-22 of the result and one unit in
// the last place, subnormals as zero.  An activation rounded to bf16 does not
// see it.  The fp32 gradients hardly do: their error is that of their sums
// (dbias and d_row_weight of 512 rows x 512 against 64 bits, SILU 0.92e-7 and
// 1.0e-7 where exact functions give 0.92e-7 and 0.93e-7, GELU 1.3e-7 and 1.1e-7
// against 0.87e-7 and 0.91e-7).  Of its own value silu is off by up to 4e-7 at z =
// -5 and 8e-7 at -12 (exact functions: 1.9e-7).  The exact forms' branches and
// scalings cost the epilogues and the activation's backward pass more than
// their memory (GELU, 17004 rows x 1296: 42 against 36 us).
__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float reciprocal_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
constexpr float kLog2E = 1.4426950408889634f;
__device__ __forceinline__ float sigmoid(float z) { return reciprocal_approx(1.0f + exp2_approx(-kLog2E * z)); }
__device__ __forceinline__ float silu(float z) { return z * sigmoid(z); }
// The normal distribution function: erf by Abramowitz and Stegun, Handbook of
// Mathematical Functions, 7.1.26 (off by at most 1.5e-7, the size of fp32's
// own error in 1 + erf), whose exponential the density takes too.  Far down the
// tail the fit is what is left: GELU is off by 0.05% of its value at z = -4,
// 0.16% at -5, 0.36% at -6 and 3% at -12 (fp32's 1 + erf: 0.07%, 6%, all of it),
// where bf16 rounds to 0.39%; by 2.1e-7 at most anywhere below 1.
__device__ __forceinline__ float normal_cdf(float z, float* density) {
    const float e = exp2_approx(-0.5f * kLog2E * z * z);   // exp(-x^2), x = |z| / sqrt(2)
    const float t = reciprocal_approx(fmaf(0.3275911f * 0.70710678f, fabsf(z), 1.0f));
    const float poly = t * fmaf(t, fmaf(t, fmaf(t, fmaf(t, 1.061405429f, -1.453152027f), 1.421413741f), -0.284496736f),
                                0.254829592f);
    const float upper = 0.5f * poly * e;     // 1 - Phi(|z|)
    *density = 0.39894228f * e;
    return z < 0.0f ? upper : 1.0f - upper;
}
__device__ __forceinline__ float activate(float z, int act) {
    switch (act) {
        case EP_ACT_RELU: return z < 0.0f ? 0.0f : z;   // NaN stays
        case EP_ACT_GELU: {
            float density;
            return z * normal_cdf(z, &density);
        }
        case EP_ACT_SILU: return silu(z);
        default: return z;
    }
}
// The activation of n values; which one it is is asked once.
template <int N>
__device__ __forceinline__ void activate_all(float (&v)[N], int act) {
    switch (act) {
        case EP_ACT_RELU:
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = activate(v[i], EP_ACT_RELU);
            break;
        case EP_ACT_GELU:
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = activate(v[i], EP_ACT_GELU);
            break;
        case EP_ACT_SILU:
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = activate(v[i], EP_ACT_SILU);
            break;
        default: break;
    }
}

// Rows of expert e that lie inside the arrays; the rest is skipped and flagged.
// kEarly: a read that may come before the wait.
template <bool kEarly = false>
__device__ __forceinline__ int expert_rows(const int32_t* offset, const int32_t* counts, int e, int64_t rows,
                                           int64_t* first, int32_t* status) {
    const int64_t o = kEarly ? __ldcg(offset + e) : offset[e], c = kEarly ? __ldcg(counts + e) : counts[e];
    *first = o;
    if (c <= 0) return 0;
    if (o < 0 || o >= rows) {
        atomicOr(status, EP_ERR_CAPACITY);
        return 0;
    }
    if (o + c > rows) {
        atomicOr(status, EP_ERR_CAPACITY);
        return static_cast<int>(rows - o);
    }
    return static_cast<int>(c);
}

// Sum over a warp of values below 2^42 each: 16 bits and the rest.
__device__ __forceinline__ int64_t warp_sum64(int64_t v) {
    const int64_t low = __reduce_add_sync(0xffffffffu, static_cast<unsigned>(v) & 0xffffu);
    return (static_cast<int64_t>(__reduce_add_sync(0xffffffffu, static_cast<unsigned>(v >> 16))) << 16) + low;
}

// The experts' blocks into shared memory, by all threads of a block of
// kThreads.  Blocks whose rows add up to more than there are overlap, and may
// have more row tiles than the workspace and the grids are sized for (rows /
// tile + E): they are flagged and count as empty; the answer is then false.
template <int kThreads>
__device__ __forceinline__ bool expert_blocks(const int32_t* offset, const int32_t* counts, int E, int64_t rows,
                                              int* first, int* count, int64_t* warp_rows, int32_t* status) {
    int64_t mine = 0;
    for (int e = threadIdx.x; e < E; e += kThreads) {
        int64_t at;
        const int n = expert_rows<true>(offset, counts, e, rows, &at, status);
        first[e] = static_cast<int>(at);
        count[e] = n;
        mine += n;
    }
    // (few instructions: a short call's time is fetching them)
    const int64_t warps_sum = warp_sum64(mine);
    const int lane = threadIdx.x & 31;
    if (lane == 0) warp_rows[threadIdx.x / 32] = warps_sum;
    __syncthreads();
    if (warp_sum64(lane < kThreads / 32 ? warp_rows[lane] : 0) <= rows) return true;
    for (int e = threadIdx.x; e < E; e += kThreads) count[e] = 0;
    if (threadIdx.x == 0) atomicOr(status, EP_ERR_CAPACITY);
    __syncthreads();
    return false;
}

// Inclusive scan of f(e) over the experts into out[e], by all threads of a
// block of kThreads; warp_sum has a word for each warp.
template <int kThreads, class F>
__device__ __forceinline__ void scan_experts(int E, int* out, int* warp_sum, F f) {
    const int each = (E + kThreads - 1) / kThreads, e0 = threadIdx.x * each;
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    int sum = 0;
    for (int i = 0; i < each; ++i)
        if (e0 + i < E) sum += f(e0 + i);
    const int incl = warp_inclusive_scan(sum);
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    int run = incl - sum;
    for (int w = 0; w < warp; ++w) run += warp_sum[w];
    for (int i = 0; i < each; ++i)
        if (e0 + i < E) {
            run += f(e0 + i);
            out[e0 + i] = run;
        }
    __syncthreads();
}

}  // namespace epg
