// What the experts' tensor-core kernels share: tiles, tables, tensor maps and
// the epilogue of a tile.
#pragma once

#include <algorithm>

#include "experts.cuh"
#include "tcgen05.cuh"

namespace epg {
namespace {

constexpr int kReadWarps = 8;   // that read accumulators: two for each 32 lanes, taking turns at the columns
constexpr int kThreads = 128 + kReadWarps * 32;
constexpr int kM = 128;          // features of a tile
constexpr int kDepth = 64;       // terms of the sum in a stage (128 bytes of bf16)
constexpr int kABytes = kM * kDepth * 2;
constexpr int kFewBoxRows = 8;   // few tokens, down: rows of a box (143 tokens over 10 experts, 896 and 5208
                                 // features: boxes of 4 rows 82 us, of 8 rows 74; one token alike)
constexpr int kGroupTiles = 8;   // row tiles whose features are walked together, for the L2 (dense 8192 x
                                 // 7168 x 7168 under the power limit: 4 538, 8 526, 16 536, 32 569 us)

// Test-only builds (EP_TEST_DROP_FIRST_LOAD): the first CTA, or pair, announces
// its first rows on a barrier and never loads them, so that the wait for them
// runs out.
#ifdef EP_TEST_DROP_FIRST_LOAD
constexpr bool kTestDropFirstLoad = true;
#else
constexpr bool kTestDropFirstLoad = false;
#endif

constexpr int kGatherWarps = 2;  // few tokens, up: warps 2 and 3
enum Mode { kProduct, kInputGrad, kFewUp, kFewDown };

struct MmaArgs {
    CUtensorMap a, b;
    int depth;                    // terms of the sum
    int F;                        // output features of an expert
    int gate_half;                // SWIGLU: rows of W from a gate row to its up row (0: not gated)
    int E, act;
    int64_t rows;
    const int32_t* expert_offset;
    const int32_t* counts;
    const float* bias;            // [E][F or 2 F]
    const float* row_weight;
    const __nv_bfloat16* residual;
    __nv_bfloat16* y;             // rows of F
    __nv_bfloat16* z;             // rows of F or 2 F
    // few tokens
    const __nv_bfloat16* x;       // up: [T][depth]
    const int64_t* topk_idx;
    const float* topk_weights;
    int T, K;
    float* part;                  // [T * K][F]
    uint32_t* done;               // [feature tiles][T]: experts of a token that are done
    int done_words;
    __nv_bfloat16* out;           // [T][F]
    int32_t* status;
    int split;                    // CTAs of a cluster that share a tile's sum, each a piece of k (1: none)
    int wait_late;                // the inputs are complete: wait only at the end ("Reads before the wait")
};

template <int NT, int kCtas>
struct Shape {
    static constexpr int kRows = NT / kCtas;   // of the row operand in one CTA
    static constexpr int kStageBytes = kABytes + kRows * kDepth * 2;
    // few tokens (64 rows) keep room for 4096 entries beside 2048 experts' tables
    static constexpr int kStages = (NT == 64 ? 172 : 192) * 1024 / kStageBytes;
    static constexpr int kBoxRows = 64;
    static constexpr int kColumns = 2 * NT;    // of tensor memory
};

struct Barriers {
    uint64_t full[12], empty[12], acc_full[2], acc_empty[2], drain;
    uint64_t tail_full[6], cleared[6];   // weight gradient: an expert's last stage
    uint32_t tmem;
    int64_t warp_rows[kThreads / 32];
    int warp_sum[kThreads / 32];
    int gave_up;                  // a wait of the epilogue ran out
    int completed;                // few tokens, down: tokens whose last expert this tile was
};

// Experts' row tiles: tile_end[e] = row tiles of experts 0 .. e.
struct Table {
    int* tile_end;    // [E]
    int* first;       // [E] first row, or first entry of the list
    int* count;       // [E]
    int16_t* list;    // few tokens: entries t * K + k (up: their tokens t), expert by expert
    int16_t* expert;  // few tokens: expert of each entry, -1 for none; behind them, tokens just completed
    uint8_t* named;   // few tokens: experts of each token
};

// A tile: expert, its rows [row0, row0 + rows) within the expert, features from f0.
struct Tile {
    int e, row0, rows, width, f0;
};

template <int NT, int kStep = 16>
__device__ __forceinline__ Tile tile_at(int g, const Table& t, int E, int feature_tiles, int tile_features) {
    int lo = 0, hi = E - 1;
    while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (static_cast<int64_t>(t.tile_end[mid]) * feature_tiles > g)
            hi = mid;
        else
            lo = mid + 1;
    }
    Tile r;
    r.e = lo;
    const int before = lo > 0 ? t.tile_end[lo - 1] : 0;
    const int n = t.tile_end[lo] - before, cnt = t.count[lo];
    int local = g - before * feature_tiles;
    const int group = local / (kGroupTiles * feature_tiles);
    local -= group * kGroupTiles * feature_tiles;
    const int in_group = min(kGroupTiles, n - group * kGroupTiles);
    const int f = local / in_group, row_tile = group * kGroupTiles + local % in_group;
    // an expert's tiles share its rows evenly, unless the rounding to an MMA's
    // step would leave the last one without any
    const int even = ((cnt - 1) / n + kStep) / kStep * kStep;   // ceil(cnt / n), without cnt + n: it may pass 2^31
    const int per = (n - 1) * even < cnt ? even : NT;
    r.row0 = row_tile * per;
    r.rows = min(per, cnt - r.row0);
    r.width = (r.rows + kStep - 1) / kStep * kStep;
    r.f0 = f * tile_features;
    return r;
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float2 unpack2(uint32_t v) {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}

// Two neighbouring lanes hold two neighbouring features, each of two tokens as
// a pair of bf16: trading halves gives each lane both features of one token
// (the even lane the first's, the odd one the second's), and back.
__device__ __forceinline__ uint32_t trade_halves(uint32_t w, int lane) {
    const uint32_t got = __shfl_xor_sync(0xffffffffu, w, 1);
    return __byte_perm(w, got, lane & 1 ? 0x3276 : 0x5410);
}

// A lane's feature of y and its row of W within the expert.
struct Lane {
    int f, wrow;
    bool up;
};
__device__ __forceinline__ Lane lane_of(const MmaArgs& p, const Tile& r, int q, int lane) {
    Lane l;
    const bool gated = p.gate_half != 0;
    l.up = gated && (lane & 8);
    l.f = gated ? r.f0 + q * 16 + (lane / 16) * 8 + (lane & 7) : r.f0 + q * 32 + lane;
    l.wrow = l.up ? p.gate_half + l.f : l.f;
    return l;
}
__device__ __forceinline__ float bias_of(const MmaArgs& p, const Tile& r, int q, int lane) {
    const Lane l = lane_of(p, r, q, lane);
    const int Fw = p.gate_half ? 2 * p.F : p.F;
    return p.bias && l.f < p.F ? p.bias[static_cast<int64_t>(r.e) * Fw + l.wrow] : 0.0f;
}

// The 32 columns c0 .. of a tile (its rows) as one lane sees them.  Stores and
// loads of bf16 are four bytes, two neighbouring features of one token: a
// lane's i-th is column `column0 + i * step`, 64 bytes of a row from 16 lanes
// (gated: 32 from 8).
template <int kMode>
struct Columns {
    static constexpr bool kByEntry = kMode == kFewDown;   // rows of [T * K] by (token, slot), not by the list
    const MmaArgs& p;
    const Table& t;
    int first, left, column0;   // first: of the 32; left: columns there are

    __device__ __forceinline__ Columns(const MmaArgs& args, const Table& table, const Tile& r, int first_row, int lane,
                                       int c0)
        : p(args), t(table), first(first_row + c0), left(r.rows - c0) {
        column0 = p.gate_half ? ((lane & 8) ? 1 : 0) + 2 * (lane & 1) : (lane & 1);
    }
    __device__ __forceinline__ int64_t row_of(int c) const {   // of column c of the 32
        return kByEntry ? static_cast<int64_t>(t.list[first + c]) : static_cast<int64_t>(first) + c;
    }
    __device__ __forceinline__ bool has(int c) const { return c < left && EP_IN(row_of(c), p.rows); }
    // A lane's words of rows of `pitch` elements, from feature f; none if !ok.
    template <int kStep, class F>
    __device__ __forceinline__ void words(__nv_bfloat16* base, int pitch, int f, bool ok, F use) const {
        __nv_bfloat16* at = base + row_of(column0) * pitch + f;
        const int64_t next = static_cast<int64_t>(kStep) * pitch;
        const int here = ok ? left - column0 : 0;
#pragma unroll
        for (int i = 0; i < 32 / kStep; ++i, at += next)
            if (i * kStep < here && EP_IN(row_of(column0 + i * kStep), p.rows)) use(i, reinterpret_cast<uint32_t*>(at));
    }
};

// What the epilogue of 32 columns reads: asked for before it is needed.  (The
// residual may be y itself: its loads would have to wait for the stores
// before them.)
struct Ahead {
    uint32_t residual[16];
    float row_weight;   // of column `lane`
};
template <int kMode>
__device__ __forceinline__ void ask_ahead(const MmaArgs& p, const Table& t, const Tile& r, int first, int q, int lane,
                                          int c0, Ahead* a) {
    if (kMode != kProduct || (!p.row_weight && !p.residual)) return;
    const Columns<kMode> m(p, t, r, first, lane, c0);
    const Lane l = lane_of(p, r, q, lane);
    if (p.row_weight) a->row_weight = m.has(lane) ? p.row_weight[m.row_of(lane)] : 0.0f;
    if (p.residual) {
        __nv_bfloat16* const from = const_cast<__nv_bfloat16*>(p.residual);
        const auto take = [&](int i, const uint32_t* at) { a->residual[i] = *at; };
        if (p.gate_half)
            m.template words<4>(from, p.F, l.f & ~1, l.f < p.F, take);
        else
            m.template words<2>(from, p.F, l.f & ~1, l.f < p.F, take);
    }
}

// Row weight, residual and store of a lane's feature in N tokens, two for each
// word: i-th word, o[2 i] and o[2 i + 1].  column(i): of o[i].
template <int kMode, int kStep, class F>
__device__ __forceinline__ void store_rows(const MmaArgs& p, const Columns<kMode>& m, const Lane& l, int lane,
                                           const Ahead& ahead, float (&o)[64 / kStep], F column) {
    if (kMode == kProduct && p.row_weight)
#pragma unroll
        for (int i = 0; i < 64 / kStep; ++i) o[i] *= __shfl_sync(0xffffffffu, ahead.row_weight, column(i));
    if (kMode == kProduct && p.residual)
#pragma unroll
        for (int i = 0; i < 32 / kStep; ++i) {
            const float2 s = unpack2(trade_halves(ahead.residual[i], lane));
            o[2 * i] += s.x;
            o[2 * i + 1] += s.y;
        }
    uint32_t w[32 / kStep];
#pragma unroll
    for (int i = 0; i < 32 / kStep; ++i) w[i] = trade_halves(pack2(o[2 * i], o[2 * i + 1]), lane);
    m.template words<kStep>(p.y, p.F, l.f & ~1, l.f < p.F, [&](int i, uint32_t* at) { *at = w[i]; });
}

// The epilogue of 32 of a tile's columns, lane = feature, q = the warp's 32
// lanes of the accumulator.
template <int kMode>
__device__ __forceinline__ void finish_columns(const MmaArgs& p, const Table& t, const Tile& r, int first, int q,
                                               int lane, float bias, int c0, float (&v)[32], const Ahead& ahead) {
    const Columns<kMode> m(p, t, r, first, lane, c0);
    const Lane l = lane_of(p, r, q, lane);
    const bool gated = p.gate_half != 0;
    if (kMode != kInputGrad)
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] += bias;
    if (kMode == kFewDown) {
#pragma unroll 8
        for (int j = 0; j < 32; ++j)
            if (l.f < p.F && m.has(j)) p.part[m.row_of(j) * p.F + l.f] = v[j];
        return;
    }
    if (kMode == kProduct && p.z) {
        // tokens 2 i and 2 i + 1, whatever the activation
        Columns<kMode> mz = m;
        mz.column0 = lane & 1;
        uint32_t w[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] = trade_halves(pack2(v[2 * i], v[2 * i + 1]), lane);
        mz.template words<2>(p.z, gated ? 2 * p.F : p.F, l.wrow & ~1, l.f < p.F,
                             [&](int i, uint32_t* at) { *at = w[i]; });
    }
    if (kMode != kInputGrad && gated) {
        const bool up = l.up;
        float o[16];
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
            // gate lanes take tokens j and j + 2, up lanes tokens j + 1 and j + 3
            const float g0 = __shfl_xor_sync(0xffffffffu, up ? v[j] : v[j + 1], 8);
            const float g1 = __shfl_xor_sync(0xffffffffu, up ? v[j + 2] : v[j + 3], 8);
            o[j / 2] = up ? silu(g0) * v[j + 1] : silu(v[j]) * g0;
            o[j / 2 + 1] = up ? silu(g1) * v[j + 3] : silu(v[j + 2]) * g1;
        }
        store_rows<kMode, 4>(p, m, l, lane, ahead, o, [&](int i) { return 2 * i + (up ? 1 : 0); });
    } else {
        if (kMode != kInputGrad) activate_all(v, p.act);
        store_rows<kMode, 2>(p, m, l, lane, ahead, v, [](int i) { return i; });
    }
}

// Weights [E][rows][cols] as a map of boxes of 128 bytes of columns x `box` rows.
inline bool weight_map(CUtensorMap* m, const void* w, int E, int rows, int cols, int box, bool fp8 = false) {
    const uint64_t dims[3] = {static_cast<uint64_t>(cols), static_cast<uint64_t>(rows), static_cast<uint64_t>(E)};
    const uint64_t pitch = static_cast<uint64_t>(cols) * (fp8 ? 1 : 2);
    const uint64_t strides[2] = {pitch, pitch * rows};
    const uint32_t boxes[3] = {fp8 ? 128u : 64u, static_cast<uint32_t>(box), 1};
    return encode_map(m, fp8, 3, w, dims, strides, boxes);
}
// Gate and up rows in turns of 8, for tiles of 64 + 64 rows (see above).
inline bool gated_map(CUtensorMap* m, const void* w, int E, int n, int cols, bool fp8 = false) {
    const uint64_t pitch = static_cast<uint64_t>(cols) * (fp8 ? 1 : 2), half = pitch * n;
    const uint64_t dims[5] = {static_cast<uint64_t>(cols), 8, 2, static_cast<uint64_t>(n / 8),
                              static_cast<uint64_t>(E)};
    const uint64_t strides[4] = {pitch, half, 8 * pitch, 2 * half};
    const uint32_t boxes[5] = {fp8 ? 128u : 64u, 8, 2, kM / 16, 1};
    return encode_map(m, fp8, 5, w, dims, strides, boxes);
}
inline bool row_map(CUtensorMap* m, const void* x, int64_t rows, int cols, int box, bool fp8 = false) {
    const uint64_t dims[2] = {static_cast<uint64_t>(cols), static_cast<uint64_t>(rows)};
    const uint64_t strides[1] = {static_cast<uint64_t>(cols) * (fp8 ? 1 : 2)};
    const uint32_t boxes[2] = {fp8 ? 128u : 64u, static_cast<uint32_t>(box)};
    return encode_map(m, fp8, 2, x, dims, strides, boxes);
}

// The product's arguments; the maps are the caller's.
inline MmaArgs product_args(const ExpertGemmParams& p) {
    MmaArgs a{};
    a.depth = p.K;
    a.F = p.N;
    a.gate_half = p.act == EP_ACT_SWIGLU ? p.N : 0;
    a.E = p.E;
    a.act = p.act;
    a.rows = p.rows;
    a.expert_offset = p.expert_offset;
    a.counts = p.counts;
    a.bias = p.bias;
    a.row_weight = p.row_weight;
    a.residual = p.residual;
    a.y = p.y;
    a.z = p.z;
    a.status = p.status;
    return a;
}

inline int bound_tiles(int64_t row_tiles, int feature_tiles) {
    const int64_t v = row_tiles * feature_tiles;
    return v > (1 << 20) ? 1 << 20 : static_cast<int>(v);
}

}  // namespace
}  // namespace epg
