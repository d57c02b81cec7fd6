// C ABI of libep_get.so: host-side argument checks, parameter blocks and
// launches.  Declarations and the full contract are in include/ep_get.h.
#include <algorithm>
#include <atomic>
#include <chrono>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <cxxabi.h>
#include <mutex>
#include <string>

#include "ep_internal.cuh"
#include "experts.cuh"
#include "experts_w4.cuh"
#include "route.cuh"

namespace epg {

bool debug_enabled() {
    static const bool on = [] {
        const char* v = std::getenv("EP_GET_DEBUG");
        return v != nullptr && v[0] != '\0' && std::strcmp(v, "0") != 0;
    }();
    return on;
}

void debug_log(const char* fmt, ...) {
    char line[512];
    va_list ap;
    va_start(ap, fmt);
    std::vsnprintf(line, sizeof(line), fmt, ap);
    va_end(ap);
    std::fprintf(stderr, "[ep_get] %s\n", line);
}

void debug_launch(const void* kernel, dim3 grid, dim3 block, size_t smem, int cluster) {
    const char* name = nullptr;
    if (cudaFuncGetName(&name, kernel) != cudaSuccess || name == nullptr) {
        cudaGetLastError();
        name = "?";
    }
    int st = 0;
    char* readable = abi::__cxa_demangle(name, nullptr, nullptr, &st);
    debug_log("launch %s grid (%u, %u, %u) block (%u, %u, %u) smem %zu cluster %d",
              (st == 0 && readable) ? readable : name, grid.x, grid.y, grid.z, block.x, block.y, block.z, smem,
              cluster);
    std::free(readable);
}

// A status a host check returns, logged (with the check's line) when it is an error.
ep_status_t debug_ret(const char* fn, int line, ep_status_t s) {
    if (s != EP_OK && debug_enabled()) debug_log("%s: %s (api.cu:%d)", fn, ep_status_string(s), line);
    return s;
}

const DeviceInfo& device_info() {
    constexpr int kMaxDevices = 64;
    static std::mutex mu;
    static DeviceInfo infos[kMaxDevices];
    static bool have[kMaxDevices] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) dev = 0;
    std::lock_guard<std::mutex> lock(mu);
    if (!have[dev]) {
        DeviceInfo d{dev, 0, 0};
        cudaDeviceGetAttribute(&d.num_sms, cudaDevAttrMultiProcessorCount, dev);
        cudaDeviceGetAttribute(&d.max_smem_optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
        if (d.num_sms < 1) d.num_sms = 1;
        infos[dev] = d;
        have[dev] = true;
    }
    return infos[dev];
}

}  // namespace epg

#define EP_RET(s) ::epg::debug_ret(__func__, __LINE__, (s))

namespace {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool ok_ptr(const void* p) { return p != nullptr && aligned16(p); }

// Shape checks shared by the three calls.
ep_status_t check_shape(int T, int K, int E, int R) {
    if (T < 0 || K < 1 || E < 1 || R < 1) return EP_RET(EP_ERR_INVALID_ARG);
    if (K > EP_MAX_TOPK || R > EP_MAX_RANKS || E > EP_MAX_EXPERTS) return EP_RET(EP_ERR_UNSUPPORTED);
    if (E % R != 0) return EP_RET(EP_ERR_INVALID_ARG);
    if (E / R > EP_MAX_EXPERTS_PER_RANK) return EP_RET(EP_ERR_UNSUPPORTED);
    if (static_cast<int64_t>(T) * R > INT32_MAX || static_cast<int64_t>(T) * K > INT32_MAX)
        return EP_RET(EP_ERR_UNSUPPORTED);
    return EP_OK;
}

}  // namespace

extern "C" {

int ep_abi_version(void) { return 8; }

int ep_bounds_checked(void) { return EP_GET_CHECKED ? 1 : 0; }

size_t ep_layout_workspace_bytes(int num_tokens, int num_topk, int num_experts, int num_ranks,
                                 int ranks_per_node) {
    (void)num_topk;
    if (num_tokens < 0 || num_experts < 1 || num_ranks < 1) return 16;
    const int nodes = ranks_per_node > 0 ? num_ranks / ranks_per_node : 0;
    return epg::layout_workspace(num_tokens, num_experts, num_ranks, nodes).total;
}

int ep_theoretical_num_sms(int hidden, int num_topk, int num_experts, int num_ranks, int out_dtype,
                           int is_combine, double hbm_gbs, double sm_read_gbs, double sm_write_gbs,
                           int prefer_overlap_with_compute, int device_sms) {
    const bool fp8 = out_dtype == EP_FP8_E4M3;
    if (out_dtype != EP_BF16 && !fp8) return 0;
    if (hidden <= 0 || hidden % (fp8 ? 128 : 8) != 0) return 0;
    if (num_ranks < 1 || num_experts < num_ranks || num_experts % num_ranks != 0) return 0;
    if (num_topk < 1 || num_topk > EP_MAX_TOPK || num_topk > num_experts) return 0;
    if (!(hbm_gbs > 0.0) || !(sm_read_gbs > 0.0) || !(sm_write_gbs > 0.0) || device_sms < 1) return 0;
    // C(E - E/R, K) / C(E, K) = prod_{i<K} (E - E/R - i) / (E - i): the chance
    // that none of K distinct uniform experts lives on a given rank.
    const int others = num_experts - num_experts / num_ranks;
    double miss = 1.0;
    for (int i = 0; i < num_topk; ++i)
        miss *= others - i > 0 ? static_cast<double>(others - i) / (num_experts - i) : 0.0;
    const double g = num_ranks * (1.0 - miss);
    const double h = static_cast<double>(hidden);
    const double row = fp8 ? h + 4.0 * (h / 128.0) : 2.0 * h;
    const double read = is_combine ? g * 2.0 * h : 2.0 * h;
    const double write = is_combine ? 2.0 * h : g * row;
    const double per_byte = hbm_gbs / (read + write);
    const double n = std::max(per_byte * read / sm_read_gbs, per_byte * write / sm_write_gbs);
    int sms = std::max(4, static_cast<int>(std::ceil(n * 1.25)));
    sms += sms & 1;
    if (!prefer_overlap_with_compute) sms = std::max(sms, 64);
    return std::min(sms, device_sms);
}

int64_t ep_recv_capacity_bound(int num_tokens, int num_topk, int num_ranks) {
    if (num_tokens <= 0 || num_topk <= 0 || num_ranks <= 0) return 0;
    return static_cast<int64_t>(num_tokens) * (num_topk < num_ranks ? num_topk : num_ranks);
}

}  // extern "C"

namespace epg {

ep_status_t layout_params(const int64_t* topk_idx, int T, int K, int E, int R, int ranks_per_node,
                          int expert_alignment, const ep_layout_t* out, void* workspace, size_t ws_bytes,
                          int32_t* d_status, bool check_workspace, LayoutParams& p) {
    if (!out || !d_status) return EP_RET(EP_ERR_INVALID_ARG);
    ep_status_t s = check_shape(T, K, E, R);
    if (s != EP_OK) return s;
    if (ranks_per_node < 0 || (ranks_per_node > 0 && R % ranks_per_node != 0))
        return EP_RET(EP_ERR_INVALID_ARG);
    if (expert_alignment < 1) return EP_RET(EP_ERR_INVALID_ARG);
    if (!ok_ptr(out->num_tokens_per_rank) || !ok_ptr(out->num_tokens_per_expert) ||
        !ok_ptr(out->rank_offset) || !ok_ptr(out->expert_offset))
        return EP_RET(EP_ERR_INVALID_ARG);
    if (T > 0 && (!ok_ptr(topk_idx) || !ok_ptr(out->is_token_in_rank) || !ok_ptr(out->dst_row)))
        return EP_RET(EP_ERR_INVALID_ARG);
    if (out->num_tokens_per_node && !aligned16(out->num_tokens_per_node)) return EP_RET(EP_ERR_INVALID_ARG);
    if (out->src_dst_count && (!aligned16(out->src_dst_count) || T % R != 0)) return EP_RET(EP_ERR_INVALID_ARG);
    if (out->token_offset && !aligned16(out->token_offset)) return EP_RET(EP_ERR_INVALID_ARG);
    if (out->expanded_row && !aligned16(out->expanded_row)) return EP_RET(EP_ERR_INVALID_ARG);
    // node rows: node_offset and node_row together (node_row may be NULL, an
    // empty array, when there are no tokens)
    if (out->node_row && !out->node_offset) return EP_RET(EP_ERR_INVALID_ARG);
    if (out->node_offset && !out->node_row && T > 0) return EP_RET(EP_ERR_INVALID_ARG);
    if (out->node_offset && (ranks_per_node <= 0 || !ok_ptr(out->num_tokens_per_node) ||
                             !aligned16(out->node_row) || !aligned16(out->node_offset)))
        return EP_RET(EP_ERR_INVALID_ARG);
    const int nodes_ws = ranks_per_node > 0 ? R / ranks_per_node : 0;
    const epg::LayoutWorkspace w = epg::layout_workspace(T, E, R, nodes_ws);
    if (!check_workspace) return EP_OK;
    if (!ok_ptr(workspace) || ws_bytes < w.total) return EP_RET(EP_ERR_INVALID_ARG);

    p = epg::LayoutParams{};
    p.topk_idx = topk_idx;
    p.T = T;
    p.K = K;
    p.E = E;
    p.R = R;
    p.experts_per_rank = E / R;
    p.ranks_per_node = ranks_per_node;
    p.num_nodes = (ranks_per_node > 0 && out->num_tokens_per_node) ? R / ranks_per_node : 0;
    p.alignment = expert_alignment;
    p.num_tiles = (T + epg::kTileTokens - 1) / epg::kTileTokens;
    p.num_tokens_per_rank = out->num_tokens_per_rank;
    p.num_tokens_per_node = out->num_tokens_per_node;
    p.num_tokens_per_expert = out->num_tokens_per_expert;
    p.is_token_in_rank = out->is_token_in_rank;
    p.rank_offset = out->rank_offset;
    p.expert_offset = out->expert_offset;
    p.dst_row = out->dst_row;
    p.src_dst_count = out->src_dst_count;
    p.token_offset = out->token_offset;
    p.expanded_row = T > 0 ? out->expanded_row : nullptr;
    p.node_offset = out->node_offset;
    p.node_row = T > 0 ? out->node_row : nullptr;
    char* ws = static_cast<char*>(workspace);
    p.ws_rank = reinterpret_cast<int32_t*>(ws + w.off_rank);
    p.ws_expert = reinterpret_cast<int32_t*>(ws + w.off_expert);
    p.ws_node = reinterpret_cast<int32_t*>(ws + w.off_node);
    p.ws_bitmap = reinterpret_cast<uint32_t*>(ws + w.off_bitmap);
    p.status = d_status;
    return EP_OK;
}

}  // namespace epg

extern "C" {

ep_status_t ep_get_layout(const int64_t* topk_idx, int T, int K, int E, int R, int ranks_per_node,
                          int expert_alignment, const ep_layout_t* out, void* workspace,
                          size_t ws_bytes, int32_t* d_status, void* cuda_stream) {
    EP_DEBUG("ep_get_layout: T=%d K=%d E=%d R=%d ranks_per_node=%d alignment=%d%s%s",
             T, K, E, R, ranks_per_node, expert_alignment, out && out->expanded_row ? " expanded_row" : "",
             out && out->node_row ? " node_row" : "");
    epg::LayoutParams p{};
    const ep_status_t s = epg::layout_params(topk_idx, T, K, E, R, ranks_per_node, expert_alignment, out, workspace,
                                             ws_bytes, d_status, true, p);
    if (s != EP_OK) return s;
    const cudaStream_t stream = static_cast<cudaStream_t>(cuda_stream);
    if (epg::launch_layout(p, stream) != cudaSuccess) return EP_RET(EP_ERR_CUDA);
    // no tokens: the node-row kernels are not launched, node_offset is all zero
    if (T == 0 && out->node_offset &&
        cudaMemsetAsync(out->node_offset, 0, sizeof(int32_t) * (R / ranks_per_node + 1), stream) != cudaSuccess)
        return EP_RET(EP_ERR_CUDA);
    return EP_OK;
}

}  // extern "C"

namespace {

// A tag for the rows-ready signal, distinct for every call of the process:
// the splitmix64 output function (Steele, Lea and Flood, "Fast splittable
// pseudorandom number generators", 2014), a bijection of 64-bit words,
// applied to a per-process offset plus an odd multiple of the call count.
uint64_t next_rows_tag() {
    static std::atomic<uint64_t> calls{0};
    static const uint64_t salt =
        static_cast<uint64_t>(std::chrono::steady_clock::now().time_since_epoch().count()) ^
        static_cast<uint64_t>(reinterpret_cast<uintptr_t>(&calls));
    uint64_t z = salt + 0x9e3779b97f4a7c15ull * (calls.fetch_add(1, std::memory_order_relaxed) + 1);
    z = (z ^ (z >> 30)) * 0xbf58476d1ce4e5b9ull;
    z = (z ^ (z >> 27)) * 0x94d049bb133111ebull;
    z ^= z >> 31;
    return z != 0 ? z : 1;
}

// Shared by ep_dispatch and ep_layout_and_dispatch.  self_layout (few
// tokens, ep_layout_and_dispatch): no layout kernel has run; the dispatch
// kernel computes the rows itself and writes the layout arrays of `lp`.
ep_status_t dispatch_impl(const void* x, const int64_t* topk_idx, const float* topk_weights, int T, int H, int K,
                          int E, int R, const ep_layout_t* layout, int out_dtype, int64_t recv_capacity,
                          void* recv_x, float* recv_sf, int sf_col_major, int32_t* recv_topk_idx,
                          float* recv_topk_weights, int32_t* recv_src_idx, int num_sms, int32_t* d_status,
                          void* cuda_stream, const epg::LayoutParams* self_layout,
                          const epg::RowsSignal* rows = nullptr) {
    if (!layout || !d_status || num_sms < 0) return EP_RET(EP_ERR_INVALID_ARG);
    ep_status_t s = check_shape(T, K, E, R);
    if (s != EP_OK) return s;
    if (H < 1) return EP_RET(EP_ERR_INVALID_ARG);
    if (out_dtype == EP_BF16) {
        if (H % 8 != 0) return EP_RET(EP_ERR_INVALID_ARG);
    } else if (out_dtype == EP_FP8_E4M3) {
        if (H % 128 != 0) return EP_RET(EP_ERR_INVALID_ARG);
        if (H > 65536) return EP_RET(EP_ERR_UNSUPPORTED);
    } else {
        return EP_RET(EP_ERR_INVALID_ARG);
    }
    if (recv_capacity < 0 || recv_capacity > INT32_MAX) return EP_RET(EP_ERR_INVALID_ARG);
    if (static_cast<int64_t>(H) * 2 > UINT32_MAX / 2) return EP_RET(EP_ERR_UNSUPPORTED);
    if (T > 0 && (!ok_ptr(x) || !ok_ptr(topk_idx) || !ok_ptr(layout->dst_row)))
        return EP_RET(EP_ERR_INVALID_ARG);
    if (recv_capacity > 0 && !ok_ptr(recv_x)) return EP_RET(EP_ERR_INVALID_ARG);
    if (out_dtype == EP_FP8_E4M3 && recv_capacity > 0 && !ok_ptr(recv_sf)) return EP_RET(EP_ERR_INVALID_ARG);
    if (recv_topk_weights && T > 0 && !ok_ptr(topk_weights)) return EP_RET(EP_ERR_INVALID_ARG);
    if ((recv_topk_idx && !aligned16(recv_topk_idx)) ||
        (recv_topk_weights && !aligned16(recv_topk_weights)) ||
        (recv_src_idx && !aligned16(recv_src_idx)))
        return EP_RET(EP_ERR_INVALID_ARG);
    if (T == 0) return EP_OK;

    epg::DispatchParams p{};
    p.x = static_cast<const uint8_t*>(x);
    p.topk_idx = topk_idx;
    p.topk_weights = topk_weights;
    p.dst_row = layout->dst_row;
    p.token_offset = layout->token_offset;
    p.T = T;
    p.H = H;
    p.K = K;
    p.E = E;
    p.R = R;
    p.experts_per_rank = E / R;
    p.capacity = recv_capacity;
    p.recv_x = static_cast<uint8_t*>(recv_x);
    p.recv_sf = recv_sf;
    p.sf_col_major = sf_col_major ? 1 : 0;
    p.sf_stride = (recv_capacity + 3) / 4 * 4;
    p.recv_topk_idx = recv_topk_idx;
    p.recv_topk_weights = recv_topk_weights;
    p.recv_src_idx = recv_src_idx;
    p.num_sms = num_sms;
    p.status = d_status;
    if (self_layout) {
        p.self_route = 1;
        p.l_num_tokens_per_rank = self_layout->num_tokens_per_rank;
        p.l_num_tokens_per_node = self_layout->num_nodes > 0 ? self_layout->num_tokens_per_node : nullptr;
        p.l_num_tokens_per_expert = self_layout->num_tokens_per_expert;
        p.l_is_token_in_rank = self_layout->is_token_in_rank;
        p.l_rank_offset = self_layout->rank_offset;
        p.l_expert_offset = self_layout->expert_offset;
        p.l_dst_row = self_layout->dst_row;
        p.l_src_dst_count = self_layout->src_dst_count;
        p.l_token_offset = self_layout->token_offset;
        p.l_alignment = self_layout->alignment;
        p.l_ranks_per_node = self_layout->ranks_per_node;
        p.l_num_nodes = self_layout->num_nodes;
    }
    if (rows && rows->slots) {
        p.rows_ready = rows->slots;
        p.rows_tag = rows->tag;
        p.rows_tokens = rows->tokens;
        p.rows_slots = rows->count;
    }
    cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
    const cudaError_t e = out_dtype == EP_BF16 ? epg::launch_dispatch_bf16(p, st)
                                               : epg::launch_dispatch_fp8(p, st);
    return e == cudaSuccess ? EP_OK : EP_RET(EP_ERR_CUDA);
}

}  // namespace

extern "C" {

ep_status_t ep_dispatch(const void* x, const int64_t* topk_idx, const float* topk_weights, int T,
                        int H, int K, int E, int R, const ep_layout_t* layout, int out_dtype,
                        int64_t recv_capacity, void* recv_x, float* recv_sf, int sf_col_major,
                        int32_t* recv_topk_idx, float* recv_topk_weights, int32_t* recv_src_idx,
                        int num_sms, int32_t* d_status, void* cuda_stream) {
    EP_DEBUG("ep_dispatch: T=%d H=%d K=%d E=%d R=%d %s capacity=%lld sf_col_major=%d num_sms=%d",
             T, H, K, E, R, out_dtype == EP_FP8_E4M3 ? "fp8" : "bf16", static_cast<long long>(recv_capacity),
             sf_col_major, num_sms);
    return dispatch_impl(x, topk_idx, topk_weights, T, H, K, E, R, layout, out_dtype, recv_capacity, recv_x, recv_sf,
                         sf_col_major, recv_topk_idx, recv_topk_weights, recv_src_idx, num_sms, d_status, cuda_stream,
                         nullptr);
}

ep_status_t ep_layout_and_dispatch(const void* x, const int64_t* topk_idx, const float* topk_weights, int T, int H,
                                   int K, int E, int R, int ranks_per_node, int expert_alignment,
                                   const ep_layout_t* layout, void* workspace, size_t ws_bytes, int out_dtype,
                                   int64_t recv_capacity, void* recv_x, float* recv_sf, int sf_col_major,
                                   int32_t* recv_topk_idx, float* recv_topk_weights, int32_t* recv_src_idx,
                                   int32_t* d_status, void* cuda_stream) {
    EP_DEBUG("ep_layout_and_dispatch: T=%d H=%d K=%d E=%d R=%d ranks_per_node=%d alignment=%d %s capacity=%lld",
             T, H, K, E, R, ranks_per_node, expert_alignment, out_dtype == EP_FP8_E4M3 ? "fp8" : "bf16",
             static_cast<long long>(recv_capacity));
    // the dispatch's host checks first, so that a rejected call launches nothing
    if (!layout || !d_status) return EP_RET(EP_ERR_INVALID_ARG);
    ep_status_t s = check_shape(T, K, E, R);
    if (s != EP_OK) return s;
    if (H < 1 || (out_dtype != EP_BF16 && out_dtype != EP_FP8_E4M3)) return EP_RET(EP_ERR_INVALID_ARG);
    if (H % (out_dtype == EP_BF16 ? 8 : 128) != 0) return EP_RET(EP_ERR_INVALID_ARG);
    if (out_dtype == EP_FP8_E4M3 && H > 65536) return EP_RET(EP_ERR_UNSUPPORTED);
    if (recv_capacity < 0 || recv_capacity > INT32_MAX) return EP_RET(EP_ERR_INVALID_ARG);
    if (static_cast<int64_t>(H) * 2 > UINT32_MAX / 2) return EP_RET(EP_ERR_UNSUPPORTED);
    if (T > 0 && (!ok_ptr(x) || !ok_ptr(topk_idx))) return EP_RET(EP_ERR_INVALID_ARG);
    if (recv_capacity > 0 && !ok_ptr(recv_x)) return EP_RET(EP_ERR_INVALID_ARG);
    if (out_dtype == EP_FP8_E4M3 && recv_capacity > 0 && !ok_ptr(recv_sf)) return EP_RET(EP_ERR_INVALID_ARG);
    if (recv_topk_weights && T > 0 && !ok_ptr(topk_weights)) return EP_RET(EP_ERR_INVALID_ARG);
    if ((recv_topk_idx && !aligned16(recv_topk_idx)) || (recv_topk_weights && !aligned16(recv_topk_weights)) ||
        (recv_src_idx && !aligned16(recv_src_idx)))
        return EP_RET(EP_ERR_INVALID_ARG);
    epg::LayoutParams lp{};
    s = epg::layout_params(topk_idx, T, K, E, R, ranks_per_node, expert_alignment, layout, workspace, ws_bytes,
                           d_status, true, lp);
    if (s != EP_OK) return s;
    // Few tokens: one kernel; its CTAs derive the rows themselves and write
    // the layout (expanded rows and node rows need the layout kernel).
    const bool one_kernel = T >= 1 && T <= epg::kSelfRouteMaxTokens && R <= 32 && K <= epg::kSelfRouteMaxTopk &&
                            E <= epg::kSelfRouteMaxExperts && !lp.expanded_row && !lp.node_row && !lp.node_offset;
    // Otherwise the layout kernel, and the dispatch waits for the rows-ready
    // signal of the cluster layout (where the dispatch kernel is one of the
    // two that read it) instead of the layout kernel's completion.
    epg::RowsSignal rows{};
    if (!one_kernel && T > 0 && epg::dispatch_reads_rows_signal(out_dtype == EP_FP8_E4M3) &&
        (reinterpret_cast<uintptr_t>(workspace) & 127u) == 0) {
        rows.slots = static_cast<uint64_t*>(workspace);
        rows.tag = next_rows_tag();
        rows.bytes = ws_bytes;
    }
    if (!one_kernel) {
        if (epg::launch_layout(lp, static_cast<cudaStream_t>(cuda_stream), &rows) != cudaSuccess)
            return EP_RET(EP_ERR_CUDA);
        if (T == 0 && layout->node_offset &&
            cudaMemsetAsync(layout->node_offset, 0, sizeof(int32_t) * (R / ranks_per_node + 1),
                            static_cast<cudaStream_t>(cuda_stream)) != cudaSuccess)
            return EP_RET(EP_ERR_CUDA);
    }
    return dispatch_impl(x, topk_idx, topk_weights, T, H, K, E, R, layout, out_dtype, recv_capacity, recv_x, recv_sf,
                         sf_col_major, recv_topk_idx, recv_topk_weights, recv_src_idx, 0, d_status, cuda_stream,
                         one_kernel ? &lp : nullptr, &rows);
}

ep_status_t ep_dispatch_hierarchical(const void* x, const int64_t* topk_idx, const float* topk_weights, int T,
                                     int H, int K, int E, int R, int rpn, const ep_layout_t* layout,
                                     int out_dtype, int64_t node_capacity, void* node_x, float* node_sf,
                                     int32_t* node_src_idx, int64_t recv_capacity, void* recv_x, float* recv_sf,
                                     int sf_col_major, int32_t* recv_topk_idx, float* recv_topk_weights,
                                     int32_t* recv_src_idx, int32_t* d_status, void* cuda_stream) {
    EP_DEBUG("ep_dispatch_hierarchical: T=%d H=%d K=%d E=%d R=%d ranks_per_node=%d %s node_capacity=%lld capacity=%lld",
             T, H, K, E, R, rpn, out_dtype == EP_FP8_E4M3 ? "fp8" : "bf16", static_cast<long long>(node_capacity),
             static_cast<long long>(recv_capacity));
    if (!layout || !d_status) return EP_RET(EP_ERR_INVALID_ARG);
    ep_status_t s = check_shape(T, K, E, R);
    if (s != EP_OK) return s;
    if (rpn < 1 || R % rpn != 0) return EP_RET(EP_ERR_INVALID_ARG);
    const bool fp8 = out_dtype == EP_FP8_E4M3;
    if (H < 1) return EP_RET(EP_ERR_INVALID_ARG);
    if (out_dtype == EP_BF16) {
        if (H % 8 != 0) return EP_RET(EP_ERR_INVALID_ARG);
    } else if (fp8) {
        if (H % 128 != 0) return EP_RET(EP_ERR_INVALID_ARG);
        if (H > 65536) return EP_RET(EP_ERR_UNSUPPORTED);
    } else {
        return EP_RET(EP_ERR_INVALID_ARG);
    }
    if (recv_capacity < 0 || recv_capacity > INT32_MAX) return EP_RET(EP_ERR_INVALID_ARG);
    if (node_capacity < 0 || node_capacity > INT32_MAX) return EP_RET(EP_ERR_INVALID_ARG);
    if (static_cast<int64_t>(H) * 2 > UINT32_MAX / 2) return EP_RET(EP_ERR_UNSUPPORTED);
    if (T > 0 && (!ok_ptr(x) || !ok_ptr(topk_idx) || !ok_ptr(layout->dst_row) || !ok_ptr(layout->node_row)))
        return EP_RET(EP_ERR_INVALID_ARG);
    if (node_capacity > 0 && (!ok_ptr(node_x) || (fp8 && !ok_ptr(node_sf)))) return EP_RET(EP_ERR_INVALID_ARG);
    if (node_src_idx && !aligned16(node_src_idx)) return EP_RET(EP_ERR_INVALID_ARG);
    if (recv_capacity > 0 && !ok_ptr(recv_x)) return EP_RET(EP_ERR_INVALID_ARG);
    if (fp8 && recv_capacity > 0 && !ok_ptr(recv_sf)) return EP_RET(EP_ERR_INVALID_ARG);
    if (recv_topk_weights && T > 0 && !ok_ptr(topk_weights)) return EP_RET(EP_ERR_INVALID_ARG);
    if ((recv_topk_idx && !aligned16(recv_topk_idx)) || (recv_topk_weights && !aligned16(recv_topk_weights)) ||
        (recv_src_idx && !aligned16(recv_src_idx)))
        return EP_RET(EP_ERR_INVALID_ARG);
    if (T == 0) return EP_OK;
    const int nodes = R / rpn;
    cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);

    // stage 1: the ordinary dispatch with the node table as destinations
    epg::DispatchParams p{};
    p.x = static_cast<const uint8_t*>(x);
    p.topk_idx = topk_idx;
    p.topk_weights = topk_weights;
    p.dst_row = layout->node_row;
    p.T = T;
    p.H = H;
    p.K = K;
    p.E = E;
    p.R = nodes;
    p.experts_per_rank = E / R;
    p.capacity = node_capacity;
    p.recv_x = static_cast<uint8_t*>(node_x);
    p.recv_sf = node_sf;
    p.sf_col_major = 0;
    p.sf_stride = node_capacity;
    p.recv_src_idx = node_src_idx;
    p.status = d_status;
    cudaError_t e = fp8 ? epg::launch_dispatch_fp8(p, st) : epg::launch_dispatch_bf16(p, st);
    if (e != cudaSuccess) return EP_RET(EP_ERR_CUDA);

    // stage 2: node rows to the ranks of their node
    epg::HierParams h{};
    h.node_x = static_cast<const uint8_t*>(node_x);
    h.node_sf = node_sf;
    h.topk_idx = topk_idx;
    h.topk_weights = topk_weights;
    h.dst_row = layout->dst_row;
    h.node_row = layout->node_row;
    h.T = T;
    h.H = H;
    h.K = K;
    h.E = E;
    h.R = R;
    h.experts_per_rank = E / R;
    h.ranks_per_node = rpn;
    h.num_nodes = nodes;
    h.node_capacity = node_capacity;
    h.capacity = recv_capacity;
    h.recv_x = static_cast<uint8_t*>(recv_x);
    h.recv_sf = recv_sf;
    h.sf_col_major = sf_col_major ? 1 : 0;
    h.sf_stride = (recv_capacity + 3) / 4 * 4;
    h.recv_topk_idx = recv_topk_idx;
    h.recv_topk_weights = recv_topk_weights;
    h.recv_src_idx = recv_src_idx;
    h.status = d_status;
    return epg::launch_forward_scaleup(h, fp8, st) == cudaSuccess ? EP_OK : EP_RET(EP_ERR_CUDA);
}

ep_status_t ep_combine_hierarchical(const void* y, int64_t num_y_rows, const int64_t* topk_idx,
                                    const float* topk_weights, int T, int H, int K, int E, int R, int rpn,
                                    const ep_layout_t* layout, int64_t node_capacity, void* node_y, void* out,
                                    int32_t* d_status, void* cuda_stream) {
    EP_DEBUG("ep_combine_hierarchical: T=%d H=%d K=%d E=%d R=%d ranks_per_node=%d rows=%lld node_capacity=%lld %s",
             T, H, K, E, R, rpn, static_cast<long long>(num_y_rows), static_cast<long long>(node_capacity),
             topk_weights ? "weighted" : "unweighted");
    if (!layout || !d_status) return EP_RET(EP_ERR_INVALID_ARG);
    ep_status_t s = check_shape(T, K, E, R);
    if (s != EP_OK) return s;
    if (rpn < 1 || R % rpn != 0) return EP_RET(EP_ERR_INVALID_ARG);
    if (H < 1 || H % 8 != 0) return EP_RET(EP_ERR_INVALID_ARG);
    if (num_y_rows < 0 || num_y_rows > INT32_MAX) return EP_RET(EP_ERR_INVALID_ARG);
    if (node_capacity < 0 || node_capacity > INT32_MAX) return EP_RET(EP_ERR_INVALID_ARG);
    if (num_y_rows > 0 && !ok_ptr(y)) return EP_RET(EP_ERR_INVALID_ARG);
    if (node_capacity > 0 && !ok_ptr(node_y)) return EP_RET(EP_ERR_INVALID_ARG);
    if (T > 0 && (!ok_ptr(out) || !ok_ptr(layout->dst_row) || !ok_ptr(layout->node_row)))
        return EP_RET(EP_ERR_INVALID_ARG);
    if (topk_weights && T > 0 && (!ok_ptr(topk_weights) || !ok_ptr(topk_idx))) return EP_RET(EP_ERR_INVALID_ARG);
    if (T == 0) return EP_OK;
    const int nodes = R / rpn;
    cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);

    // stage 1: per (token, node) partial sums of the node's ranks
    epg::HierParams h{};
    h.topk_idx = topk_idx;
    h.topk_weights = topk_weights;
    h.dst_row = layout->dst_row;
    h.node_row = layout->node_row;
    h.T = T;
    h.H = H;
    h.K = K;
    h.E = E;
    h.R = R;
    h.experts_per_rank = E / R;
    h.ranks_per_node = rpn;
    h.num_nodes = nodes;
    h.node_capacity = node_capacity;
    h.y = static_cast<const uint8_t*>(y);
    h.num_y_rows = num_y_rows;
    h.node_y = static_cast<uint8_t*>(node_y);
    h.status = d_status;
    if (epg::launch_reduce_scaleup(h, topk_weights != nullptr, st) != cudaSuccess) return EP_RET(EP_ERR_CUDA);

    // stage 2: the ordinary unweighted combine over the node rows
    epg::CombineParams p{};
    p.y = static_cast<const uint8_t*>(node_y);
    p.num_y_rows = node_capacity;
    p.topk_idx = topk_idx;
    p.dst_row = layout->node_row;
    p.T = T;
    p.H = H;
    p.K = K;
    p.E = E;
    p.R = nodes;
    p.experts_per_rank = E / R;
    p.out = static_cast<uint8_t*>(out);
    p.status = d_status;
    return epg::launch_combine(p, false, st) == cudaSuccess ? EP_OK : EP_RET(EP_ERR_CUDA);
}

ep_status_t ep_combine(const void* y, int64_t num_y_rows, const int64_t* topk_idx,
                       const float* topk_weights, int T, int H, int K, int E, int R,
                       const ep_layout_t* layout, void* out, int num_sms, int32_t* d_status,
                       void* cuda_stream) {
    EP_DEBUG("ep_combine: T=%d H=%d K=%d E=%d R=%d rows=%lld %s num_sms=%d",
             T, H, K, E, R, static_cast<long long>(num_y_rows), topk_weights ? "weighted" : "unweighted", num_sms);
    if (!layout || !d_status || num_sms < 0) return EP_RET(EP_ERR_INVALID_ARG);
    ep_status_t s = check_shape(T, K, E, R);
    if (s != EP_OK) return s;
    if (H < 1 || H % 8 != 0) return EP_RET(EP_ERR_INVALID_ARG);
    if (num_y_rows < 0 || num_y_rows > INT32_MAX) return EP_RET(EP_ERR_INVALID_ARG);
    if (num_y_rows > 0 && !ok_ptr(y)) return EP_RET(EP_ERR_INVALID_ARG);
    if (T > 0 && (!ok_ptr(out) || !ok_ptr(layout->dst_row))) return EP_RET(EP_ERR_INVALID_ARG);
    if (topk_weights && T > 0 && (!ok_ptr(topk_weights) || !ok_ptr(topk_idx))) return EP_RET(EP_ERR_INVALID_ARG);
    if (T == 0) return EP_OK;

    epg::CombineParams p{};
    p.y = static_cast<const uint8_t*>(y);
    p.num_y_rows = num_y_rows;
    p.topk_idx = topk_idx;
    p.topk_weights = topk_weights;
    p.dst_row = layout->dst_row;
    p.T = T;
    p.H = H;
    p.K = K;
    p.E = E;
    p.R = R;
    p.experts_per_rank = E / R;
    p.out = static_cast<uint8_t*>(out);
    p.num_sms = num_sms;
    p.status = d_status;
    const cudaError_t e =
        epg::launch_combine(p, topk_weights != nullptr, static_cast<cudaStream_t>(cuda_stream));
    return e == cudaSuccess ? EP_OK : EP_RET(EP_ERR_CUDA);
}

int64_t ep_expanded_capacity_bound(int num_tokens, int num_topk, int num_experts, int expert_alignment) {
    if (num_tokens < 0 || num_topk < 0 || num_experts < 0 || expert_alignment < 1) return 0;
    return static_cast<int64_t>(num_tokens) * num_topk + static_cast<int64_t>(num_experts) * (expert_alignment - 1);
}

ep_status_t ep_dispatch_expanded(const void* x, const int64_t* topk_idx, const float* topk_weights, int T,
                                 int H, int K, int E, int R, const ep_layout_t* layout, int out_dtype,
                                 int64_t recv_capacity, void* recv_x, float* recv_sf, int sf_col_major,
                                 int32_t* recv_src_idx, float* recv_weight, int num_sms, int32_t* d_status,
                                 void* cuda_stream) {
    EP_DEBUG("ep_dispatch_expanded: T=%d H=%d K=%d E=%d R=%d %s capacity=%lld sf_col_major=%d num_sms=%d",
             T, H, K, E, R, out_dtype == EP_FP8_E4M3 ? "fp8" : "bf16", static_cast<long long>(recv_capacity),
             sf_col_major, num_sms);
    if (!layout || !d_status || num_sms < 0) return EP_RET(EP_ERR_INVALID_ARG);
    ep_status_t s = check_shape(T, K, E, R);
    if (s != EP_OK) return s;
    if (H < 1) return EP_RET(EP_ERR_INVALID_ARG);
    if (out_dtype == EP_BF16) {
        if (H % 8 != 0) return EP_RET(EP_ERR_INVALID_ARG);
    } else if (out_dtype == EP_FP8_E4M3) {
        if (H % 128 != 0) return EP_RET(EP_ERR_INVALID_ARG);
        if (H > 65536) return EP_RET(EP_ERR_UNSUPPORTED);
    } else {
        return EP_RET(EP_ERR_INVALID_ARG);
    }
    if (recv_capacity < 0 || recv_capacity > INT32_MAX) return EP_RET(EP_ERR_INVALID_ARG);
    if (static_cast<int64_t>(H) * 2 > UINT32_MAX / 2) return EP_RET(EP_ERR_UNSUPPORTED);
    if (T > 0 && (!ok_ptr(x) || !ok_ptr(layout->expanded_row))) return EP_RET(EP_ERR_INVALID_ARG);
    if (recv_capacity > 0 && !ok_ptr(recv_x)) return EP_RET(EP_ERR_INVALID_ARG);
    if (out_dtype == EP_FP8_E4M3 && recv_capacity > 0 && !ok_ptr(recv_sf)) return EP_RET(EP_ERR_INVALID_ARG);
    if (recv_weight && T > 0 && !ok_ptr(topk_weights)) return EP_RET(EP_ERR_INVALID_ARG);
    if ((recv_src_idx && !aligned16(recv_src_idx)) || (recv_weight && !aligned16(recv_weight)))
        return EP_RET(EP_ERR_INVALID_ARG);
    if (T == 0) return EP_OK;

    epg::DispatchParams p{};
    p.x = static_cast<const uint8_t*>(x);
    p.topk_idx = topk_idx;
    p.topk_weights = topk_weights;
    p.expanded_row = layout->expanded_row;
    p.T = T;
    p.H = H;
    p.K = K;
    p.E = E;
    p.R = R;
    p.experts_per_rank = E / R;
    p.capacity = recv_capacity;
    p.recv_x = static_cast<uint8_t*>(recv_x);
    p.recv_sf = recv_sf;
    p.sf_col_major = sf_col_major ? 1 : 0;
    p.sf_stride = (recv_capacity + 3) / 4 * 4;
    p.recv_src_idx = recv_src_idx;
    p.recv_weight = recv_weight;
    p.num_sms = num_sms;
    p.status = d_status;
    cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
    const cudaError_t e = out_dtype == EP_BF16 ? epg::launch_dispatch_bf16(p, st)
                                               : epg::launch_dispatch_fp8(p, st);
    return e == cudaSuccess ? EP_OK : EP_RET(EP_ERR_CUDA);
}

ep_status_t ep_combine_expanded(const void* y, int64_t num_y_rows, const float* topk_weights, int T, int H,
                                int K, int E, int R, const ep_layout_t* layout, void* out, int num_sms,
                                int32_t* d_status, void* cuda_stream) {
    EP_DEBUG("ep_combine_expanded: T=%d H=%d K=%d E=%d R=%d rows=%lld %s num_sms=%d",
             T, H, K, E, R, static_cast<long long>(num_y_rows), topk_weights ? "weighted" : "unweighted", num_sms);
    if (!layout || !d_status || num_sms < 0) return EP_RET(EP_ERR_INVALID_ARG);
    ep_status_t s = check_shape(T, K, E, R);
    if (s != EP_OK) return s;
    if (H < 1 || H % 8 != 0) return EP_RET(EP_ERR_INVALID_ARG);
    if (num_y_rows < 0 || num_y_rows > INT32_MAX) return EP_RET(EP_ERR_INVALID_ARG);
    if (num_y_rows > 0 && !ok_ptr(y)) return EP_RET(EP_ERR_INVALID_ARG);
    if (T > 0 && (!ok_ptr(out) || !ok_ptr(layout->expanded_row))) return EP_RET(EP_ERR_INVALID_ARG);
    if (topk_weights && T > 0 && !ok_ptr(topk_weights)) return EP_RET(EP_ERR_INVALID_ARG);
    if (T == 0) return EP_OK;

    epg::CombineParams p{};
    p.y = static_cast<const uint8_t*>(y);
    p.num_y_rows = num_y_rows;
    p.topk_weights = topk_weights;
    p.expanded_row = layout->expanded_row;
    p.T = T;
    p.H = H;
    p.K = K;
    p.E = E;
    p.R = R;
    p.experts_per_rank = E / R;
    p.out = static_cast<uint8_t*>(out);
    p.num_sms = num_sms;
    p.status = d_status;
    const cudaError_t e =
        epg::launch_combine(p, topk_weights != nullptr, static_cast<cudaStream_t>(cuda_stream));
    return e == cudaSuccess ? EP_OK : EP_RET(EP_ERR_CUDA);
}

ep_status_t ep_combine_topk_weights(const float* recv_topk_weights, int64_t num_rows, int T, int K, int E,
                                   int R, const ep_layout_t* layout, float* combined_topk_weights,
                                   int32_t* d_status, void* cuda_stream) {
    EP_DEBUG("ep_combine_topk_weights: T=%d K=%d E=%d R=%d rows=%lld", T, K, E, R, static_cast<long long>(num_rows));
    if (!layout || !d_status) return EP_RET(EP_ERR_INVALID_ARG);
    ep_status_t s = check_shape(T, K, E, R);
    if (s != EP_OK) return s;
    if (num_rows < 0 || num_rows > INT32_MAX) return EP_RET(EP_ERR_INVALID_ARG);
    if (num_rows > 0 && !ok_ptr(recv_topk_weights)) return EP_RET(EP_ERR_INVALID_ARG);
    if (T > 0 && (!ok_ptr(combined_topk_weights) || !ok_ptr(layout->dst_row))) return EP_RET(EP_ERR_INVALID_ARG);
    if (T == 0) return EP_OK;
    epg::CombineWeightsParams p{};
    p.recv_topk_weights = recv_topk_weights;
    p.num_rows = num_rows;
    p.dst_row = layout->dst_row;
    p.T = T;
    p.K = K;
    p.R = R;
    p.combined = combined_topk_weights;
    p.status = d_status;
    return epg::launch_combine_topk_weights(p, static_cast<cudaStream_t>(cuda_stream)) == cudaSuccess
               ? EP_OK
               : EP_ERR_CUDA;
}

ep_status_t ep_accumulate_expert_stats(const ep_layout_t* layout, int E, int64_t* stats, void* cuda_stream) {
    EP_DEBUG("ep_accumulate_expert_stats: E=%d", E);
    if (!layout || E < 1) return EP_RET(EP_ERR_INVALID_ARG);
    if (E > EP_MAX_EXPERTS) return EP_RET(EP_ERR_UNSUPPORTED);
    if (!ok_ptr(layout->num_tokens_per_expert) || !ok_ptr(stats)) return EP_RET(EP_ERR_INVALID_ARG);
    return epg::launch_accumulate_expert_stats(layout->num_tokens_per_expert, E, stats,
                                               static_cast<cudaStream_t>(cuda_stream)) == cudaSuccess
               ? EP_OK
               : EP_ERR_CUDA;
}

}  // extern "C"

namespace {

// Checks shared by ep_expert_gemm and its backward call.
ep_status_t check_experts(int64_t num_rows, int K, int N, int E, int act, const int32_t* offset,
                          const int32_t* counts, const int32_t* d_status) {
    if (!d_status || num_rows < 0 || K < 1 || N < 1 || E < 1) return EP_RET(EP_ERR_INVALID_ARG);
    if (act < EP_ACT_NONE || act > EP_ACT_SWIGLU) return EP_RET(EP_ERR_INVALID_ARG);
    if (E > EP_MAX_EXPERTS || num_rows > EP_MAX_EXPERT_ROWS || K > epg::kMaxExpertDim || N > epg::kMaxExpertDim)
        return EP_RET(EP_ERR_UNSUPPORTED);
    if (K % 8 != 0 || N % 8 != 0 || !ok_ptr(offset) || !ok_ptr(counts)) return EP_RET(EP_ERR_INVALID_ARG);
    return EP_OK;
}

}  // namespace

extern "C" {

ep_status_t ep_expert_gemm(const void* x, const float* x_sf, int sf_col_major, const void* w, const float* w_sf,
                           int in_dtype, const float* bias, int activation, const float* row_weight,
                           const void* residual, int64_t num_rows, int K, int N, int E,
                           const int32_t* expert_offset, const int32_t* num_tokens_per_expert, void* y, void* z,
                           int32_t* d_status, void* cuda_stream) {
    EP_DEBUG("ep_expert_gemm: rows=%lld K=%d N=%d E=%d %s act=%d%s%s%s%s", static_cast<long long>(num_rows), K, N, E,
             in_dtype == EP_FP8_E4M3 ? "fp8" : "bf16", activation, bias ? " bias" : "",
             row_weight ? " row_weight" : "", residual ? " residual" : "", z ? " z" : "");
    ep_status_t s = check_experts(num_rows, K, N, E, activation, expert_offset, num_tokens_per_expert, d_status);
    if (s != EP_OK) return s;
    const bool fp8 = in_dtype == EP_FP8_E4M3;
    if (in_dtype != EP_BF16 && !fp8) return EP_RET(EP_ERR_INVALID_ARG);
    if (fp8 && (K % 128 != 0 || N % 128 != 0)) return EP_RET(EP_ERR_INVALID_ARG);
    if (!aligned16(bias) || !aligned16(row_weight) || !aligned16(residual) || !aligned16(z))
        return EP_RET(EP_ERR_INVALID_ARG);
    if (!ok_ptr(w) || (fp8 && !ok_ptr(w_sf))) return EP_RET(EP_ERR_INVALID_ARG);
    if (num_rows > 0 && (!ok_ptr(x) || !ok_ptr(y) || (fp8 && !ok_ptr(x_sf)))) return EP_RET(EP_ERR_INVALID_ARG);
    if (num_rows == 0) return EP_OK;

    epg::ExpertGemmParams p{};
    p.x = static_cast<const uint8_t*>(x);
    p.x_sf = x_sf;
    p.sf_row = sf_col_major ? 1 : K / 128;
    p.sf_block = sf_col_major ? (num_rows + 3) / 4 * 4 : 1;
    p.w = static_cast<const uint8_t*>(w);
    p.w_sf = w_sf;
    p.bias = bias;
    p.row_weight = row_weight;
    p.residual = static_cast<const __nv_bfloat16*>(residual);
    p.rows = num_rows;
    p.K = K;
    p.N = N;
    p.Nw = activation == EP_ACT_SWIGLU ? 2 * N : N;
    p.E = E;
    p.act = activation;
    p.expert_offset = expert_offset;
    p.counts = num_tokens_per_expert;
    p.y = static_cast<__nv_bfloat16*>(y);
    p.z = static_cast<__nv_bfloat16*>(z);
    p.status = d_status;
    const cudaStream_t stream = static_cast<cudaStream_t>(cuda_stream);
    const cudaError_t e = fp8 ? epg::launch_expert_gemm_fp8(p, stream) : epg::launch_expert_gemm_bf16(p, stream);
    return e == cudaSuccess ? EP_OK : EP_RET(EP_ERR_CUDA);
}

size_t ep_expert_gemm_backward_workspace_bytes(int64_t num_rows, int n_dim, int num_experts, int activation) {
    if (num_rows < 0 || n_dim < 1 || num_experts < 1) return 16;
    return epg::backward_workspace(num_rows, n_dim, activation == EP_ACT_SWIGLU ? 2 * n_dim : n_dim, num_experts).total;
}

ep_status_t ep_expert_gemm_backward(const void* dy, const void* x, const void* w, const void* z, int activation,
                                    const float* row_weight, int64_t num_rows, int K, int N, int E,
                                    const int32_t* expert_offset, const int32_t* num_tokens_per_expert, void* dx,
                                    void* dw, float* dbias, float* d_row_weight, void* workspace, size_t ws_bytes,
                                    int32_t* d_status, void* cuda_stream) {
    EP_DEBUG("ep_expert_gemm_backward: rows=%lld K=%d N=%d E=%d act=%d%s%s%s%s%s", static_cast<long long>(num_rows),
             K, N, E, activation, row_weight ? " row_weight" : "", dx ? " dx" : "", dw ? " dw" : "",
             dbias ? " dbias" : "", d_row_weight ? " d_row_weight" : "");
    ep_status_t s = check_experts(num_rows, K, N, E, activation, expert_offset, num_tokens_per_expert, d_status);
    if (s != EP_OK) return s;
    if (!aligned16(row_weight) || !aligned16(dx) || !aligned16(dw) || !aligned16(dbias) || !aligned16(d_row_weight) ||
        !aligned16(x) || !aligned16(w) || !aligned16(z) || !aligned16(dy))
        return EP_RET(EP_ERR_INVALID_ARG);
    const int Nw = activation == EP_ACT_SWIGLU ? 2 * N : N;
    if (num_rows > 0 && (!dy || (dx && !w) || (dw && !x))) return EP_RET(EP_ERR_INVALID_ARG);
    if (num_rows > 0 && !z && (activation != EP_ACT_NONE || d_row_weight)) return EP_RET(EP_ERR_INVALID_ARG);
    const epg::BackwardWorkspace b = epg::backward_workspace(num_rows, N, Nw, E);
    if (!ok_ptr(workspace) || ws_bytes < b.total) return EP_RET(EP_ERR_INVALID_ARG);

    epg::ExpertBackwardParams p{};
    p.dy = static_cast<const __nv_bfloat16*>(dy);
    p.x = static_cast<const __nv_bfloat16*>(x);
    p.w = static_cast<const __nv_bfloat16*>(w);
    p.z = static_cast<const __nv_bfloat16*>(z);
    p.row_weight = row_weight;
    p.rows = num_rows;
    p.K = K;
    p.N = N;
    p.Nw = Nw;
    p.E = E;
    p.act = activation;
    p.expert_offset = expert_offset;
    p.counts = num_tokens_per_expert;
    p.dx = num_rows > 0 ? static_cast<__nv_bfloat16*>(dx) : nullptr;
    p.dw = static_cast<__nv_bfloat16*>(dw);
    p.dbias = dbias;
    p.d_row_weight = num_rows > 0 ? d_row_weight : nullptr;
    char* ws = static_cast<char*>(workspace);
    p.dz = reinterpret_cast<__nv_bfloat16*>(ws + b.off_dz);
    p.bias_part = reinterpret_cast<float*>(ws + b.off_part);
    p.weight_part = reinterpret_cast<float*>(ws + b.off_weight);
    p.blocks_fit = reinterpret_cast<int*>(ws + b.off_fit);
    p.status = d_status;
    return epg::launch_expert_backward(p, static_cast<cudaStream_t>(cuda_stream)) == cudaSuccess
               ? EP_OK
               : EP_RET(EP_ERR_CUDA);
}

size_t ep_moe_few_tokens_workspace_bytes(int num_tokens, int num_topk, int hidden, int inner, int num_experts) {
    (void)num_experts;
    if (num_tokens < 0 || num_topk < 1 || hidden < 1 || inner < 1) return 16;
    return epg::few_workspace(num_tokens, num_topk, hidden, inner).total;
}

ep_status_t ep_moe_few_tokens(const void* x, const int64_t* topk_idx, const float* topk_weights, const void* w_up,
                              const float* bias_up, int activation, const void* w_down, const float* bias_down,
                              const void* residual, int T, int H, int I, int K, int E, void* workspace,
                              size_t ws_bytes, void* out, int32_t* d_status, void* cuda_stream) {
    EP_DEBUG("ep_moe_few_tokens: T=%d H=%d I=%d K=%d E=%d act=%d%s%s%s", T, H, I, K, E, activation,
             bias_up ? " bias_up" : "", bias_down ? " bias_down" : "", residual ? " residual" : "");
    if (!d_status || T < 0 || H < 1 || I < 1 || K < 1 || E < 1) return EP_RET(EP_ERR_INVALID_ARG);
    if (activation < EP_ACT_NONE || activation > EP_ACT_SWIGLU) return EP_RET(EP_ERR_INVALID_ARG);
    if (T > EP_FEW_MAX_TOKENS || K > EP_FEW_MAX_TOPK || E > EP_MAX_EXPERTS || H > epg::kMaxExpertDim ||
        I > epg::kMaxExpertDim)
        return EP_RET(EP_ERR_UNSUPPORTED);
    if (H % 8 != 0 || I % 8 != 0) return EP_RET(EP_ERR_INVALID_ARG);
    if (!ok_ptr(w_up) || !ok_ptr(w_down) || !aligned16(bias_up) || !aligned16(bias_down) || !aligned16(residual))
        return EP_RET(EP_ERR_INVALID_ARG);
    if (T > 0 && (!ok_ptr(x) || !ok_ptr(topk_idx) || !ok_ptr(topk_weights) || !ok_ptr(out)))
        return EP_RET(EP_ERR_INVALID_ARG);
    const epg::FewWorkspace f = epg::few_workspace(T, K, H, I);
    if (!ok_ptr(workspace) || ws_bytes < f.total) return EP_RET(EP_ERR_INVALID_ARG);
    if (T == 0) return EP_OK;

    epg::FewTokensParams p{};
    p.x = static_cast<const __nv_bfloat16*>(x);
    p.topk_idx = topk_idx;
    p.topk_weights = topk_weights;
    p.w_up = static_cast<const __nv_bfloat16*>(w_up);
    p.bias_up = bias_up;
    p.w_down = static_cast<const __nv_bfloat16*>(w_down);
    p.bias_down = bias_down;
    p.residual = static_cast<const __nv_bfloat16*>(residual);
    p.T = T;
    p.H = H;
    p.I = I;
    p.Nw = activation == EP_ACT_SWIGLU ? 2 * I : I;
    p.K = K;
    p.E = E;
    p.act = activation;
    char* ws = static_cast<char*>(workspace);
    p.h = reinterpret_cast<__nv_bfloat16*>(ws + f.off_h);
    p.part = reinterpret_cast<float*>(ws + f.off_part);
    p.done = reinterpret_cast<uint32_t*>(ws + f.off_done);
    p.out = static_cast<__nv_bfloat16*>(out);
    p.status = d_status;
    return epg::launch_few_tokens(p, static_cast<cudaStream_t>(cuda_stream)) == cudaSuccess ? EP_OK
                                                                                           : EP_RET(EP_ERR_CUDA);
}

}  // extern "C"

namespace {

// Checks shared by the router's calls.
ep_status_t check_router(const void* logits, int dtype, int64_t row_stride, const int64_t* topk_idx, int T, int E, int K,
                         int score, const int32_t* d_status) {
    if (!d_status || T < 0 || E < 1 || K < 1 || K > E) return EP_RET(EP_ERR_INVALID_ARG);
    if (dtype != EP_BF16 && dtype != EP_FP16 && dtype != EP_FP32) return EP_RET(EP_ERR_INVALID_ARG);
    if (score != EP_SCORE_SOFTMAX && score != EP_SCORE_SIGMOID) return EP_RET(EP_ERR_INVALID_ARG);
    if (T > (1 << 30) || E > EP_MAX_EXPERTS || K > EP_MAX_TOPK || static_cast<int64_t>(T) * E > INT32_MAX ||
        static_cast<int64_t>(T) * K > INT32_MAX)
        return EP_RET(EP_ERR_UNSUPPORTED);
    const uintptr_t item = dtype == EP_FP32 ? 4 : 2;
    if (row_stride < E || (T > 0 && (!logits || reinterpret_cast<uintptr_t>(logits) % item != 0)))
        return EP_RET(EP_ERR_INVALID_ARG);
    if (row_stride > (INT64_MAX / 8) / (T > 0 ? T : 1)) return EP_RET(EP_ERR_UNSUPPORTED);
    if (T > 0 && !ok_ptr(topk_idx)) return EP_RET(EP_ERR_INVALID_ARG);
    return EP_OK;
}

// Sequences of the loss: how many, and where they are.
ep_status_t check_sequences(const int32_t* seq_offset, int S, int E) {
    if (S < 1 || (!seq_offset && S != 1) || !aligned16(seq_offset)) return EP_RET(EP_ERR_INVALID_ARG);
    if (static_cast<int64_t>(S) * E > INT32_MAX) return EP_RET(EP_ERR_UNSUPPORTED);
    return EP_OK;
}

// 4-bit weights of n_w features: pointers, types and groups.
ep_status_t check_w4(const void* w, const void* sf, const void* zero, int sf_dtype, int format, int group, int depth) {
    if (sf_dtype != EP_BF16 && sf_dtype != EP_FP32) return EP_RET(EP_ERR_INVALID_ARG);
    if (format != EP_W4_INT && (format != EP_W4_FP || zero)) return EP_RET(EP_ERR_INVALID_ARG);
    if ((group != 32 && group != 64 && group != 128) || depth % group != 0) return EP_RET(EP_ERR_INVALID_ARG);
    return ok_ptr(w) && ok_ptr(sf) && aligned16(zero) ? EP_OK : EP_RET(EP_ERR_INVALID_ARG);
}

epg::Weights4 weights4(const void* w, const void* sf, const void* zero, int sf_dtype, int format, int group) {
    return {static_cast<const uint8_t*>(w), sf, zero, sf_dtype == EP_FP32 ? 1 : 0, format, group};
}

}  // namespace

extern "C" {

ep_status_t ep_route(const void* logits, int logits_dtype, int64_t row_stride, const float* bias,
                     const uint8_t* token_mask, int T, int E, int K, int score, int num_groups, int topk_groups,
                     int normalize, float scale, int64_t* topk_idx, float* topk_weights, int32_t* d_status,
                     void* cuda_stream) {
    EP_DEBUG("ep_route: T=%d E=%d K=%d dtype=%d stride=%lld score=%d groups=%d/%d%s%s%s", T, E, K, logits_dtype,
             static_cast<long long>(row_stride), score, topk_groups, num_groups, bias ? " bias" : "",
             token_mask ? " mask" : "", normalize ? " normalize" : "");
    const ep_status_t s = check_router(logits, logits_dtype, row_stride, topk_idx, T, E, K, score, d_status);
    if (s != EP_OK) return s;
    if (num_groups < 1 || E % num_groups != 0 || topk_groups < 1 || topk_groups > num_groups)
        return EP_RET(EP_ERR_INVALID_ARG);
    if (num_groups > EP_MAX_GROUPS) return EP_RET(EP_ERR_UNSUPPORTED);
    if (static_cast<int64_t>(topk_groups) * (E / num_groups) < K) return EP_RET(EP_ERR_INVALID_ARG);
    if (!aligned16(bias) || (T > 0 && !ok_ptr(topk_weights))) return EP_RET(EP_ERR_INVALID_ARG);
    if (T == 0) return EP_OK;
    epg::RouteParams p{};
    p.logits = logits;
    p.dtype = logits_dtype;
    p.row_stride = row_stride;
    p.bias = bias;
    p.token_mask = token_mask;
    p.T = T;
    p.E = E;
    p.K = K;
    p.score = score;
    p.num_groups = num_groups;
    p.topk_groups = topk_groups;
    p.normalize = normalize ? 1 : 0;
    p.scale = scale;
    p.topk_idx = topk_idx;
    p.topk_weights = topk_weights;
    p.status = d_status;
    return epg::launch_route(p, static_cast<cudaStream_t>(cuda_stream)) == cudaSuccess ? EP_OK : EP_RET(EP_ERR_CUDA);
}

size_t ep_balance_loss_workspace_bytes(int num_tokens, int num_experts, int num_sequences) {
    if (num_tokens < 0 || num_experts < 1 || num_sequences < 1) return 16;
    return epg::balance_workspace(num_tokens, num_experts, num_sequences).total;
}

ep_status_t ep_balance_loss(const void* logits, int logits_dtype, int64_t row_stride, const int64_t* topk_idx,
                            const uint8_t* token_mask, const int32_t* seq_offset, int T, int E, int K, int S, int score,
                            float coeff, float* loss, float* load, int32_t* num_tokens_per_expert, void* workspace,
                            size_t ws_bytes, int32_t* d_status, void* cuda_stream) {
    EP_DEBUG("ep_balance_loss: T=%d E=%d K=%d S=%d dtype=%d stride=%lld score=%d%s%s", T, E, K, S, logits_dtype,
             static_cast<long long>(row_stride), score, token_mask ? " mask" : "", seq_offset ? " sequences" : "");
    ep_status_t s = check_router(logits, logits_dtype, row_stride, topk_idx, T, E, K, score, d_status);
    if (s != EP_OK) return s;
    s = check_sequences(seq_offset, S, E);
    if (s != EP_OK) return s;
    if (!ok_ptr(loss) || !ok_ptr(load) || !aligned16(num_tokens_per_expert)) return EP_RET(EP_ERR_INVALID_ARG);
    const epg::BalanceWorkspace b = epg::balance_workspace(T, E, S);
    if (!ok_ptr(workspace) || ws_bytes < b.total) return EP_RET(EP_ERR_INVALID_ARG);
    epg::BalanceParams p{};
    p.logits = logits;
    p.dtype = logits_dtype;
    p.row_stride = row_stride;
    p.topk_idx = topk_idx;
    p.token_mask = token_mask;
    p.seq_offset = seq_offset;
    p.T = T;
    p.E = E;
    p.K = K;
    p.S = S;
    p.score = score;
    p.coeff = coeff;
    p.loss = loss;
    p.load = load;
    p.counts = num_tokens_per_expert;
    char* ws = static_cast<char*>(workspace);
    p.part = reinterpret_cast<int2*>(ws + b.off_part);
    p.part_tokens = reinterpret_cast<int32_t*>(ws + b.off_tokens);
    p.part_loss = reinterpret_cast<float*>(ws + b.off_loss);
    p.arrived = reinterpret_cast<uint32_t*>(ws + b.off_arrived);
    p.tile_tokens = b.tile_tokens;
    p.tiles = b.tiles;
    p.status = d_status;
    return epg::launch_balance_loss(p, static_cast<cudaStream_t>(cuda_stream)) == cudaSuccess ? EP_OK
                                                                                             : EP_RET(EP_ERR_CUDA);
}

ep_status_t ep_route_backward(const void* logits, int logits_dtype, int64_t row_stride, const int64_t* topk_idx,
                              const uint8_t* token_mask, const float* d_topk_weights, const float* load,
                              const float* d_loss, const int32_t* seq_offset, int T, int E, int K, int S, int score,
                              int normalize, float scale, void* d_logits, int64_t d_row_stride, int32_t* d_status,
                              void* cuda_stream) {
    EP_DEBUG("ep_route_backward: T=%d E=%d K=%d S=%d dtype=%d stride=%lld score=%d%s%s%s", T, E, K, S, logits_dtype,
             static_cast<long long>(row_stride), score, d_topk_weights ? " weights" : "", load ? " loss" : "",
             token_mask ? " mask" : "");
    ep_status_t s = check_router(logits, logits_dtype, row_stride, topk_idx, T, E, K, score, d_status);
    if (s != EP_OK) return s;
    if (load) {
        s = check_sequences(seq_offset, S, E);
        if (s != EP_OK) return s;
    }
    const uintptr_t item = logits_dtype == EP_FP32 ? 4 : 2;
    if (d_row_stride < E || reinterpret_cast<uintptr_t>(d_logits) % item != 0 || (T > 0 && !d_logits))
        return EP_RET(EP_ERR_INVALID_ARG);
    if (d_row_stride > (INT64_MAX / 8) / (T > 0 ? T : 1)) return EP_RET(EP_ERR_UNSUPPORTED);
    if (!aligned16(d_topk_weights) || !aligned16(load) || !aligned16(d_loss) || !load != !d_loss)
        return EP_RET(EP_ERR_INVALID_ARG);
    if (T == 0) return EP_OK;
    epg::RouteBackwardParams p{};
    p.logits = logits;
    p.dtype = logits_dtype;
    p.row_stride = row_stride;
    p.topk_idx = topk_idx;
    p.token_mask = token_mask;
    p.d_topk_weights = d_topk_weights;
    p.load = load;
    p.d_loss = d_loss;
    p.seq_offset = load ? seq_offset : nullptr;
    p.T = T;
    p.E = E;
    p.K = K;
    p.S = load ? S : 1;
    p.score = score;
    p.normalize = normalize ? 1 : 0;
    p.scale = scale;
    p.d_logits = d_logits;
    p.d_row_stride = d_row_stride;
    p.status = d_status;
    return epg::launch_route_backward(p, static_cast<cudaStream_t>(cuda_stream)) == cudaSuccess ? EP_OK
                                                                                               : EP_RET(EP_ERR_CUDA);
}

ep_status_t ep_expert_gemm_w4(const void* x, const void* w, const void* w_sf, const void* w_zero, int sf_dtype,
                              int w_format, int group, const float* bias, int activation, const float* row_weight,
                              const void* residual, int64_t num_rows, int K, int N, int E,
                              const int32_t* expert_offset, const int32_t* num_tokens_per_expert, void* y,
                              int32_t* d_status, void* cuda_stream) {
    EP_DEBUG("ep_expert_gemm_w4: rows=%lld K=%d N=%d E=%d format=%d group=%d sf=%d act=%d%s%s%s%s",
             static_cast<long long>(num_rows), K, N, E, w_format, group, sf_dtype, activation, w_zero ? " zero" : "",
             bias ? " bias" : "", row_weight ? " row_weight" : "", residual ? " residual" : "");
    ep_status_t s = check_experts(num_rows, K, N, E, activation, expert_offset, num_tokens_per_expert, d_status);
    if (s != EP_OK) return s;
    s = check_w4(w, w_sf, w_zero, sf_dtype, w_format, group, K);
    if (s != EP_OK) return s;
    if (!aligned16(bias) || !aligned16(row_weight) || !aligned16(residual)) return EP_RET(EP_ERR_INVALID_ARG);
    if (num_rows > 0 && (!ok_ptr(x) || !ok_ptr(y))) return EP_RET(EP_ERR_INVALID_ARG);
    if (num_rows == 0) return EP_OK;
    epg::ExpertGemmW4Params p{};
    p.x = static_cast<const __nv_bfloat16*>(x);
    p.w = weights4(w, w_sf, w_zero, sf_dtype, w_format, group);
    p.bias = bias;
    p.row_weight = row_weight;
    p.residual = static_cast<const __nv_bfloat16*>(residual);
    p.rows = num_rows;
    p.K = K;
    p.N = N;
    p.Nw = activation == EP_ACT_SWIGLU ? 2 * N : N;
    p.E = E;
    p.act = activation;
    p.expert_offset = expert_offset;
    p.counts = num_tokens_per_expert;
    p.y = static_cast<__nv_bfloat16*>(y);
    p.status = d_status;
    return epg::launch_expert_gemm_w4(p, static_cast<cudaStream_t>(cuda_stream)) == cudaSuccess ? EP_OK
                                                                                               : EP_RET(EP_ERR_CUDA);
}

size_t ep_moe_few_tokens_w4_workspace_bytes(int num_tokens, int num_topk, int hidden, int inner, int num_experts) {
    (void)num_experts;
    if (num_tokens < 0 || num_topk < 1 || hidden < 1 || inner < 1) return 16;
    return epg::few_w4_workspace(num_tokens, num_topk, hidden, inner).total;
}

ep_status_t ep_moe_few_tokens_w4(const void* x, const int64_t* topk_idx, const float* topk_weights, const void* w_up,
                                 const void* up_sf, const void* up_zero, int up_group, const float* bias_up,
                                 int activation, const void* w_down, const void* down_sf, const void* down_zero,
                                 int down_group, const float* bias_down, int sf_dtype, int w_format,
                                 const void* residual, int T, int H, int I, int K, int E, void* workspace,
                                 size_t ws_bytes, void* out, int32_t* d_status, void* cuda_stream) {
    EP_DEBUG("ep_moe_few_tokens_w4: T=%d H=%d I=%d K=%d E=%d format=%d groups=%d,%d sf=%d act=%d%s%s%s%s", T, H, I, K, E,
             w_format, up_group, down_group, sf_dtype, activation, up_zero ? " zero" : "", bias_up ? " bias_up" : "",
             bias_down ? " bias_down" : "", residual ? " residual" : "");
    if (!d_status || T < 0 || H < 1 || I < 1 || K < 1 || E < 1) return EP_RET(EP_ERR_INVALID_ARG);
    if (activation < EP_ACT_NONE || activation > EP_ACT_SWIGLU) return EP_RET(EP_ERR_INVALID_ARG);
    if (T > EP_FEW_MAX_TOKENS || K > EP_FEW_MAX_TOPK || E > EP_MAX_EXPERTS || H > epg::kMaxExpertDim ||
        I > epg::kMaxExpertDim)
        return EP_RET(EP_ERR_UNSUPPORTED);
    if (!up_zero != !down_zero) return EP_RET(EP_ERR_INVALID_ARG);
    ep_status_t s = check_w4(w_up, up_sf, up_zero, sf_dtype, w_format, up_group, H);
    if (s != EP_OK) return s;
    s = check_w4(w_down, down_sf, down_zero, sf_dtype, w_format, down_group, I);
    if (s != EP_OK) return s;
    if (!aligned16(bias_up) || !aligned16(bias_down) || !aligned16(residual)) return EP_RET(EP_ERR_INVALID_ARG);
    if (T > 0 && (!ok_ptr(x) || !ok_ptr(topk_idx) || !ok_ptr(topk_weights) || !ok_ptr(out)))
        return EP_RET(EP_ERR_INVALID_ARG);
    const epg::FewW4Workspace f = epg::few_w4_workspace(T, K, H, I);
    if (!ok_ptr(workspace) || ws_bytes < f.total) return EP_RET(EP_ERR_INVALID_ARG);
    if (T == 0) return EP_OK;
    epg::FewTokensW4Params p{};
    p.x = static_cast<const __nv_bfloat16*>(x);
    p.topk_idx = topk_idx;
    p.topk_weights = topk_weights;
    p.up = weights4(w_up, up_sf, up_zero, sf_dtype, w_format, up_group);
    p.bias_up = bias_up;
    p.down = weights4(w_down, down_sf, down_zero, sf_dtype, w_format, down_group);
    p.bias_down = bias_down;
    p.residual = static_cast<const __nv_bfloat16*>(residual);
    p.T = T;
    p.H = H;
    p.I = I;
    p.Nw = activation == EP_ACT_SWIGLU ? 2 * I : I;
    p.K = K;
    p.E = E;
    p.act = activation;
    char* ws = static_cast<char*>(workspace);
    p.h = reinterpret_cast<__nv_bfloat16*>(ws + f.off_h);
    p.part = reinterpret_cast<float*>(ws + f.off_part);
    p.out = static_cast<__nv_bfloat16*>(out);
    p.status = d_status;
    return epg::launch_few_tokens_w4(p, static_cast<cudaStream_t>(cuda_stream)) == cudaSuccess ? EP_OK
                                                                                              : EP_RET(EP_ERR_CUDA);
}

const char* ep_status_string(int32_t status) {
    static const char* const kNames[7] = {"invalid_arg", "unsupported", "invalid_index", "capacity",
                                          "timeout",     "cuda",        "out_of_bounds"};
    static std::string table[128];
    static std::once_flag once;
    std::call_once(once, [] {
        table[0] = "ok";
        for (int v = 1; v < 128; ++v) {
            std::string sname;
            for (int b = 0; b < 7; ++b)
                if (v & (1 << b)) {
                    if (!sname.empty()) sname += "|";
                    sname += kNames[b];
                }
            table[v] = sname;
        }
    });
    if (status < 0 || status >= 128) return "unknown";
    return table[status].c_str();
}

}  // extern "C"
