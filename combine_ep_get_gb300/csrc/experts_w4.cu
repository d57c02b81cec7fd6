// The experts' products with 4-bit weights and group scales: launches, and the sum over a token's experts.
#include <algorithm>
#include <cmath>

#include "experts_w4_kernel.cuh"

namespace epg {

namespace {

using namespace w4;

// out[t] = residual[t] + sum over k ascending of weight * part[t, k], four features a thread.  (The finishing warps'
// last tile of a token doing it, by counters, took as long for one token, 53 us, and for 128 of them left their sums
// late: 1.04 -> 1.21 ms.)
__global__ void __launch_bounds__(128) few_sum_kernel(const FewTokensW4Params p) {
    pdl_wait();
    pdl_launch_dependents();
    const int64_t quad = static_cast<int64_t>(blockIdx.x) * 128 + threadIdx.x;
    if (quad >= static_cast<int64_t>(p.T) * p.H / 4) return;
    const int t = static_cast<int>(quad * 4 / p.H), f = static_cast<int>(quad * 4 % p.H);
    float4 part[EP_FEW_MAX_TOPK];
    float weight[EP_FEW_MAX_TOPK];
    uint2 res = make_uint2(0u, 0u);
    if (p.residual) res = *reinterpret_cast<const uint2*>(p.residual + quad * 4);
#pragma unroll
    for (int k = 0; k < EP_FEW_MAX_TOPK; ++k) {
        const int entry = t * p.K + k;
        const int64_t e = k < p.K ? p.topk_idx[entry] : -1;
        const bool there = e >= 0 && e < p.E && EP_IN(entry, static_cast<int64_t>(p.T) * p.K);
        weight[k] = there ? p.topk_weights[entry] : 0.0f;
        part[k] = there ? *reinterpret_cast<const float4*>(p.part + static_cast<int64_t>(entry) * p.H + f)
                        : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
    float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int k = 0; k < EP_FEW_MAX_TOPK; ++k) {
        sum.x = fmaf(weight[k], part[k].x, sum.x);
        sum.y = fmaf(weight[k], part[k].y, sum.y);
        sum.z = fmaf(weight[k], part[k].z, sum.z);
        sum.w = fmaf(weight[k], part[k].w, sum.w);
    }
    sum.x += __uint_as_float(res.x << 16);
    sum.y += __uint_as_float(res.x & 0xffff0000u);
    sum.z += __uint_as_float(res.y << 16);
    sum.w += __uint_as_float(res.y & 0xffff0000u);
    const __nv_bfloat162 lo = __floats2bfloat162_rn(sum.x, sum.y), hi = __floats2bfloat162_rn(sum.z, sum.w);
    *reinterpret_cast<uint2*>(p.out + quad * 4) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
}

// Boxes of one stage's codes, [share][half][feature][64 bytes], and scales, [group][half][feature]; a row of codes
// is pieces of 64 bytes, a share each (where a part of one is left at its end, there is one share, and the box ends
// with the row).
bool weight_maps(Args* a, const Weights4& w, int half) {
    const int item = w.sf_fp32 ? 4 : 2;
    const uint64_t E = a->E, Nw = a->Nw, N = a->N, row = a->K / 2, groups = a->K / w.group;
    const uint64_t piece = a->whole ? 64 : Nw * row;    // (of one piece: any stride, as long as it passes for one)
    const uint32_t slots = a->slots, some = kSlotK / w.group * a->slots;
    a->sf_fp32 = w.sf_fp32;
    if (a->act == EP_ACT_SWIGLU) {
        const uint32_t features = half;
        const uint64_t dims[5] = {a->whole ? 64 : row, N, 2, a->whole ? row / 64 : 1, E};
        const uint64_t strides[4] = {row, N * row, piece, Nw * row};
        const uint32_t box[5] = {64, features, 2, slots, 1};
        const uint64_t sf_dims[4] = {N, 2, groups, E}, sf_strides[3] = {N * item, Nw * item, Nw * item * groups};
        const uint32_t sf_box[4] = {features, 2, some, 1};
        return encode_bytes_map(&a->codes, 5, w.w, dims, strides, box) &&
               encode_plain_map(&a->scales, w.sf_fp32 != 0, 4, w.sf, sf_dims, sf_strides, sf_box) &&
               (!w.zero || encode_plain_map(&a->zeros, w.sf_fp32 != 0, 4, w.zero, sf_dims, sf_strides, sf_box));
    }
    const uint32_t features = 2 * half;
    const uint64_t dims[4] = {a->whole ? 64 : row, Nw, a->whole ? row / 64 : 1, E}, strides[3] = {row, piece, Nw * row};
    const uint32_t box[4] = {64, features, slots, 1};
    const uint64_t sf_dims[3] = {Nw, groups, E}, sf_strides[2] = {Nw * item, Nw * item * groups};
    const uint32_t sf_box[3] = {features, some, 1};
    return encode_bytes_map(&a->codes, 4, w.w, dims, strides, box) &&
           encode_plain_map(&a->scales, w.sf_fp32 != 0, 3, w.sf, sf_dims, sf_strides, sf_box) &&
           (!w.zero || encode_plain_map(&a->zeros, w.sf_fp32 != 0, 3, w.zero, sf_dims, sf_strides, sf_box));
}

template <class V, typename Tiles>
cudaError_t launch_variant(Which which, Args a, const Weights4& w, Tiles row_tiles, cudaStream_t stream) {
    const DeviceInfo& info = device_info();
    const auto up = [](int v, int to) { return (v + to - 1) / to * to; };
    const int pieces = kTeam / a.slots, half = pieces * 16 * V::kPieces16, item = w.sf_fp32 ? 4 : 2;
    if (!weight_maps(&a, w, half)) return cudaErrorInvalidValue;
    const int sf_bytes = 2 * (kSlotK / w.group * a.slots) * half * item;
    a.x_offset = V::kCodeBytes;
    // (FP4: behind the rows their units, and room for those of rows that a warp reads in vain)
    const int units = w.format == EP_W4_FP ? (a.slots * a.tile_rows + 32) * 4 : 0;
    a.sf_offset = up(a.x_offset + a.slots * a.tile_rows * kRowPitch + units, 128);
    a.zero_offset = a.sf_offset + sf_bytes;
    a.stage_bytes = up(a.zero_offset + (w.zero ? sf_bytes : 0), 512);
    const int fixed = 512 + kTeam * V::kTeams * V::kSums * 128 + static_cast<int>(sizeof(Shared)) +
                      a.E * 12 + a.T * a.topk * 4;
    a.stages = std::min(kMaxStages, (info.max_smem_optin - fixed) / a.stage_bytes);
    if (a.stages < 1) return cudaErrorInvalidValue;
    const size_t smem = static_cast<size_t>(fixed) + a.stages * a.stage_bytes;
    const int features = a.act == EP_ACT_SWIGLU ? half : 2 * half;
    const int64_t tiles = row_tiles(a.tile_rows) * ((a.N + features - 1) / features);
    const dim3 grid(static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>(tiles, info.num_sms))));
    if (w.format == EP_W4_FP) return launch_fp(a, w.group, which, grid, smem, stream);
    return w.zero ? launch_zero(a, w.group, which, grid, smem, stream)
                  : launch_int(a, w.group, which, grid, smem, stream);
}

// Shares for up to 8 rows of an expert: the least time of the CTAs' turns, a turn's tiles at what the memory gives
// the SMs at work (an SM's warps take no more than 47 bytes a ns), 0.8 us a tile, and the tile's rows at 60 bytes a ns.
// One row, [7168, 7168] by 2, 4, 8 shares: 31, 21, 17 us a call on its own; 8 experts of one row, 7168 -> 2 x 2048, SWIGLU, 37.5, 39.6, 43.6,
// and 2048 -> 7168 27.3, 23.2, 31; 64 experts of four rows 175, 193, 240 and 115, 124, 160.
int best_slots(const Args& a, int64_t row_tiles, int64_t likely) {
    const double sms = device_info().num_sms;
    double best = 0.0;
    int slots = 2;
    for (int s = 2; s <= 8 && s * kSlotK <= a.K; s *= 2) {
        const int half = kTeam / s * 16 * Few::kPieces16, features = a.act == EP_ACT_SWIGLU ? half : 2 * half;
        const double tiles = static_cast<double>(row_tiles) * ((a.N + features - 1) / features);
        const double bytes = half * static_cast<double>(a.K), rows = static_cast<double>((likely + 1) / 2) * a.K * 2;
        const double turns = std::floor(tiles / sms), rest = tiles - turns * sms;
        const auto turn = [&](double ctas) { return bytes / std::min(47.0, 6780.0 / ctas) + 800.0 + rows / 60.0; };
        const double time = turns * turn(sms) + (rest > 0.0 ? turn(rest) : 0.0);
        if (best == 0.0 || time < best) {
            best = time;
            slots = s;
        }
    }
    return slots;
}

// rows: of all experts; likely: of one of them; row_tiles: at least as many tiles as a tile's rows give.
template <typename Tiles>
cudaError_t launch(Args a, const Weights4& w, int64_t rows, int64_t likely, Tiles row_tiles, cudaStream_t stream) {
    a.whole = a.K % kSlotK == 0;
    // Two shares at least: one share's 512 features would be more than a box may have.  Up to 32 likely rows by tiles
    // of 16: 64 experts of 12 and 16 rows, 7168 -> 2 x 2048, 242 us, by tiles of 32 289 and 293, of 8 318 and 324 (of 8
    // rows 197, by tiles of 8 185, but 2048 -> 7168 152 and 156).
    const bool few = likely <= 8 && a.whole && a.K >= 2 * kSlotK;
    a.tile_rows = rows < 8 ? static_cast<int>(rows) : likely <= 8 ? 8 : likely <= 32 ? 16 : 32;
    const bool mid = !few && likely <= 32 && a.whole && a.K >= 2 * kSlotK;
    a.slots = few ? best_slots(a, row_tiles(a.tile_rows), likely) : mid ? 2 : 1;
    if (few) return launch_variant<Few>(kFew, a, w, row_tiles, stream);
    return mid ? launch_variant<Mid>(kMid, a, w, row_tiles, stream) : launch_variant<Wide>(kWide, a, w, row_tiles, stream);
}

}  // namespace

cudaError_t launch_expert_gemm_w4(const ExpertGemmW4Params& p, cudaStream_t stream) {
    Args a{};
    a.mode = kProduct;
    a.x = p.x;
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
    // popular experts have a few times the mean
    const int64_t likely = p.E == 1 ? p.rows : std::min(p.rows, 2 * ((p.rows + p.E - 1) / p.E));
    const int64_t active = std::min<int64_t>(p.E, p.rows);
    return launch(a, p.w, p.rows, likely, [&](int rows) { return active + (p.rows - active) / rows; }, stream);
}

cudaError_t launch_few_tokens_w4(const FewTokensW4Params& p, cudaStream_t stream) {
    Args a{};
    a.mode = kFewUp;
    a.x = p.x;
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
    const int entries = p.T * p.K, active = std::min(p.E, entries);
    const auto tiles = [&](int rows) { return static_cast<int64_t>(active) + (entries - active) / rows; };
    const int likely = std::min(p.T, 2 * ((entries + p.E - 1) / p.E));
    cudaError_t e = launch(a, p.up, entries, likely, tiles, stream);
    if (e != cudaSuccess) return e;
    a.mode = kFewDown;
    a.x = p.h;
    a.bias = p.bias_down;
    a.K = p.I;
    a.N = a.Nw = p.H;
    a.act = EP_ACT_NONE;
    a.y = nullptr;
    a.part = p.part;
    e = launch(a, p.down, entries, likely, tiles, stream);
    if (e != cudaSuccess) return e;
    const int64_t quads = static_cast<int64_t>(p.T) * p.H / 4;
    return launch_pdl(few_sum_kernel, dim3(static_cast<unsigned>((quads + 127) / 128)), dim3(128), 0, stream, p);
}

}  // namespace epg
