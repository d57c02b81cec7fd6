// Parameter blocks and launchers of the experts with 4-bit weights (experts_w4.cu).
#pragma once

#include "experts.cuh"

namespace epg {

// One product's weights: codes [E][Nw][K / 2], scales and zero points [E][K / group][Nw].
struct Weights4 {
    const uint8_t* w;
    const void* sf;
    const void* zero;            // null: 8 (int), or the FP4 type
    int sf_fp32;                 // scales and zero points are fp32, else bf16
    int format;                  // EP_W4_INT or EP_W4_FP
    int group;
};

struct ExpertGemmW4Params {
    const __nv_bfloat16* x;      // [rows][K]
    Weights4 w;
    const float* bias;           // [E][Nw] or null
    const float* row_weight;     // [rows] or null
    const __nv_bfloat16* residual;   // [rows][N] or null
    int64_t rows;
    int K, N, Nw, E, act;
    const int32_t* expert_offset;    // [E]
    const int32_t* counts;           // [E]
    __nv_bfloat16* y;            // [rows][N]
    int32_t* status;
};

struct FewTokensW4Params {
    const __nv_bfloat16* x;      // [T][H]
    const int64_t* topk_idx;     // [T][K]
    const float* topk_weights;   // [T][K]
    Weights4 up;                 // [E][Nw][H]
    const float* bias_up;        // [E][Nw] or null
    Weights4 down;               // [E][H][I]
    const float* bias_down;      // [E][H] or null
    const __nv_bfloat16* residual;   // [T][H] or null
    int T, H, I, Nw, K, E, act;
    // Workspace [T * K][I], by entry.  bf16, as the down product's MMA takes its rows and the formula says: the one
    // rounding between the products, 0.16% of a token's norm beside the output's own 0.17%.
    __nv_bfloat16* h;
    float* part;                 // workspace [T * K][H]
    __nv_bfloat16* out;          // [T][H]
    int32_t* status;
};

cudaError_t launch_expert_gemm_w4(const ExpertGemmW4Params& p, cudaStream_t stream);
cudaError_t launch_few_tokens_w4(const FewTokensW4Params& p, cudaStream_t stream);

struct FewW4Workspace {
    size_t off_h, off_part, total;
};
inline FewW4Workspace few_w4_workspace(int T, int K, int H, int I) {
    const auto up = [](size_t v) { return (v + 255) / 256 * 256; };
    FewW4Workspace f;
    f.off_h = 0;
    f.off_part = up(static_cast<size_t>(T) * K * I * 2);
    f.total = f.off_part + up(static_cast<size_t>(T) * K * H * 4) + 256;
    return f;
}

}  // namespace epg
