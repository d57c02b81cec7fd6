// Parameter blocks and launchers of the router's operators (route.cu,
// balance.cu): the choice of experts, the balance loss and their gradient.
#pragma once

#include "ep_internal.cuh"

namespace epg {

struct RouteParams {
    const void* logits;          // [T][E], rows row_stride elements apart
    int dtype;                   // EP_BF16, EP_FP16 or EP_FP32
    int64_t row_stride;
    const float* bias;           // [E] or null
    const uint8_t* token_mask;   // [T] or null
    int T, E, K, score, num_groups, topk_groups, normalize;
    float scale;
    int64_t* topk_idx;           // [T][K]
    float* topk_weights;         // [T][K]
    int32_t* status;
};

struct BalanceParams {
    const void* logits;
    int dtype;
    int64_t row_stride;
    const int64_t* topk_idx;     // [T][K]
    const uint8_t* token_mask;   // [T] or null
    const int32_t* seq_offset;   // [S + 1] or null
    int T, E, K, S, score;
    float coeff;
    float* loss;                 // [1]
    float* load;                 // [S][E]
    int32_t* counts;             // [S][E] or null
    // workspace: one piece is one tile's tokens of one sequence, numbered tile + sequence
    int2* part;                  // [tiles + S][E] sums of scores (their bits), entries naming each expert
    int32_t* part_tokens;        // [tiles + S] tokens that count
    float* part_loss;            // [S][chunks of experts]
    uint32_t* arrived;           // [1]
    int tile_tokens, tiles;
    int32_t* status;
};

struct RouteBackwardParams {
    const void* logits;
    int dtype;
    int64_t row_stride;
    const int64_t* topk_idx;     // [T][K]
    const uint8_t* token_mask;   // [T] or null
    const float* d_topk_weights; // [T][K] or null
    const float* load;           // [S][E] or null
    const float* d_loss;         // [1], with load
    const int32_t* seq_offset;   // [S + 1] or null
    int T, E, K, S, score, normalize;
    float scale;
    void* d_logits;              // [T][E], rows d_row_stride elements apart
    int64_t d_row_stride;
    int32_t* status;
};

cudaError_t launch_route(const RouteParams& p, cudaStream_t stream);
cudaError_t launch_balance_loss(const BalanceParams& p, cudaStream_t stream);
cudaError_t launch_route_backward(const RouteBackwardParams& p, cudaStream_t stream);

// Workspace carve-up shared by the size query and the call.
constexpr int kBalanceWarps = 8;
constexpr int kBalanceChunk = 8;        // experts of one CTA of the second kernel
constexpr int kBalanceTiles = 512;      // at most (304: 15.1 us for 32768 tokens, 608: 13.7, 512: 12.8)
struct BalanceWorkspace {
    int tile_tokens, tiles;
    size_t off_part, off_tokens, off_loss, off_arrived, total;
};
inline BalanceWorkspace balance_workspace(int T, int E, int S) {
    const auto up = [](size_t v) { return (v + 255) / 256 * 256; };
    BalanceWorkspace b;
    const int each = (T + kBalanceTiles - 1) / kBalanceTiles;
    b.tile_tokens = each < 2 * kBalanceWarps ? 2 * kBalanceWarps : (each + kBalanceWarps - 1) / kBalanceWarps * kBalanceWarps;
    b.tiles = T > 0 ? (T + b.tile_tokens - 1) / b.tile_tokens : 0;
    const size_t pieces = static_cast<size_t>(b.tiles) + S, chunks = (static_cast<size_t>(E) + kBalanceChunk - 1) / kBalanceChunk;
    b.off_part = 0;
    b.off_tokens = up(pieces * E * 8);
    b.off_loss = b.off_tokens + up(pieces * 4);
    b.off_arrived = b.off_loss + up(static_cast<size_t>(S) * chunks * 4);
    b.total = b.off_arrived + 256;
    return b;
}

}  // namespace epg
