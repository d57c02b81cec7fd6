// The experts' products with 4-bit weights and group scales.
//
// z[row, f] = sum over groups of scale[group, f] * sum over the group's k of (u[f, k] - zero[group, f]) x[row, k]
//
// A call reads half a byte a weight and has few rows to multiply it by, so the
// weights' bytes bound it if what is done to each weight is little: about 11
// of them a cycle go through each quarter of an SM at the memory's rate.
// Codes become bf16 values in registers, exactly, and meet the rows in the
// warp's own MMA (m16n8k16), whose operands are registers: tcgen05 would want
// the values written to shared or tensor memory first, twice the bytes that
// its wider tiles save on the few rows there are.
//   int  16 + u is 0x4180 | u << 3: a shift and one three-input operation for
//        two weights.  The 16 and the zero point come off once a group, by the sum of
//        the group's x, which one more MMA gives (a row operand of ones).
//   FP4  sign, exponent and fraction move to bf16's places, 2^-126 of the
//        value; one multiplication of two by 2^126.
// Sums of a group stay in the MMA's fp32; the scale is applied in fp32.
//
// A word of eight codes of one feature gives the pairs (k, k + 4), k = 0 .. 3: the
// operand's order of k is any that both sides share, so x is paired that way
// too (four byte permutations a 16-byte read).  32 k's are 16 bytes of a
// feature, a word for each of four lanes; the 128-byte swizzle lets 8
// features' reads meet all banks.
//
// One CTA per SM walks the tiles (expert, rows, features).  Warp 0 loads codes,
// scales and zero points by tensor maps, warps 1-4 copy the rows, 16 bytes a
// lane, both into a ring of stages of 32 KB of codes; warps 5-12 multiply.  The
// eight warps are `slots` shares of k times 8 / slots pieces of 32 features (two
// halves of 16: gate and up for SWIGLU, so a pair meets in one lane).  Many
// shares: tiles of few features, which fill the SMs evenly, but rows are
// read for each tile again; one share: tiles of 256 features.
#include "experts_w4.cuh"
#include "tcgen05.cuh"

namespace epg {

namespace {

constexpr int kCopyWarps = 4, kMmaWarps = 8;
constexpr int kThreads = (1 + kCopyWarps + kMmaWarps) * 32;
constexpr int kMaxStages = 8;
constexpr int kSlotK = 256;                  // k's of a share in one stage: 128 bytes of codes
constexpr int kCodeBytes = kMmaWarps * 32 * kSlotK / 2;
constexpr int kRowPitch = kSlotK * 2 + 64;   // a row's share: eight lanes' reads of two rows meet all banks
constexpr int kMaxTiles8 = 4;                // row tiles of 8 in a tile

#ifdef EP_TEST_DROP_FIRST_LOAD
constexpr bool kTestDropFirstLoad = true;
#else
constexpr bool kTestDropFirstLoad = false;
#endif

enum Mode { kProduct, kFewUp, kFewDown };

struct Args {
    CUtensorMap codes;           // [E][Nw][K / 2], boxes of 128 bytes x 16 features a piece
    CUtensorMap scales, zeros;   // [E][K / group][Nw]
    const __nv_bfloat16* x;
    const float* bias;           // [E][Nw] or null
    int mode, K, N, Nw, E, act;  // depth, features out, features of the weights
    int has_zero, sf_fp32;
    int slots, tile_rows;        // shares of k; rows of a tile
    int stages, stage_bytes, x_offset, sf_offset, zero_offset;
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

struct Shared {
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t sums_full[2][kMmaWarps], sums_empty[2][kMmaWarps];
    int64_t warp_rows[kThreads / 32];
    int warp_sum[kThreads / 32];
};
// Where the shares' sums meet: [buffer][share - 1][piece][value][lane], at most 4096 floats a buffer.
constexpr int kSumsBytes = 2 * 4096 * 4;

struct Tile {
    int e, first, rows, f0;      // expert, its first row or entry here, how many, first feature
};

struct Table {
    int* tile_end;
    int* first;
    int* count;
    int16_t* list;
    int16_t* expert;
};

__device__ __forceinline__ Tile tile_at(const Args& p, const Table& t, int64_t g, int feature_tiles, int tile_features) {
    const int row_tile = static_cast<int>(g / feature_tiles);
    int lo = 0, hi = p.E - 1;      // the expert: the first with tile_end > row_tile
    while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (t.tile_end[mid] > row_tile)
            hi = mid;
        else
            lo = mid + 1;
    }
    Tile r;
    r.e = lo;
    const int before = lo > 0 ? t.tile_end[lo - 1] : 0, n = t.tile_end[lo] - before, at = row_tile - before;
    // an expert's tiles share its rows evenly, in steps of 8
    const int each = n > 1 ? min(p.tile_rows, ((t.count[lo] + n - 1) / n + 7) / 8 * 8) : t.count[lo];
    r.first = t.first[lo] + at * each;
    r.rows = max(0, min(each, t.count[lo] - at * each));
    r.f0 = static_cast<int>(g % feature_tiles) * tile_features;
    return r;
}

__device__ __forceinline__ uint32_t load_shared(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}
__device__ __forceinline__ uint4 load_shared4(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}
__device__ __forceinline__ float load_scale(uint32_t addr, int i, int fp32) {
    if (fp32) return __uint_as_float(load_shared(addr + i * 4));
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr + i * 2));
    return __uint_as_float(static_cast<uint32_t>(v) << 16);
}

// Codes i and i + 4 of a word as two bf16 values: 16 + u, or the FP4 value.
template <int kForm, int i>
__device__ __forceinline__ uint32_t two_values(uint32_t w) {
    if (kForm == EP_W4_INT) {
        const uint32_t s = i == 0 ? w << 3 : w >> (i == 0 ? 0 : 4 * i - 3);
        return (s & 0x00780078u) | 0x41804180u;
    }
    const uint32_t sign = i == 3 ? w : w << (12 - 4 * i);
    const uint32_t rest = i < 2 ? w << (i < 2 ? 6 - 4 * i : 0) : w >> (i < 2 ? 0 : 4 * i - 6);
    const uint32_t small = (sign & 0x80008000u) | (rest & 0x01c001c0u);
    uint32_t v;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(v) : "r"(small), "r"(0x7e807e80u));   // 2^126
    return v;
}

// d = a b + c for 16 features, 8 rows and 16 k's.
__device__ __forceinline__ void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// One stage of one warp's share: kBlocks blocks of 32 k's a group.
template <int kForm, int kBlocks>
__device__ __forceinline__ void multiply_stage(const Args& p, uint32_t stage, int tiles8, int piece, int slot, int lane,
                                               float (&total)[2][kMaxTiles8][4]) {
    const int g = lane >> 2, t = lane & 3, pieces = kMmaWarps / p.slots;
    const uint32_t half_bytes = kCodeBytes / 2;
    const uint32_t codes = stage + (slot * pieces + piece) * 16 * 128 + g * 128 + t * 4;
    const uint32_t x = stage + p.x_offset + slot * p.tile_rows * kRowPitch + t * 16;
    uint32_t x_row[kMaxTiles8];    // (rows that are not there may be any: their columns are not kept)
#pragma unroll
    for (int j = 0; j < kMaxTiles8; ++j) x_row[j] = x + min(j * 8 + g, p.tile_rows - 1) * kRowPitch;
    constexpr int kGroups = 8 / kBlocks;
    const int width = pieces * 16, item = p.sf_fp32 ? 4 : 2, all_groups = kGroups * p.slots;
    const uint32_t sf_at = ((slot * kGroups) * width + piece * 16 + g) * item, sf_half = all_groups * width * item;
#pragma unroll
    for (int group = 0; group < kGroups; ++group) {
        float acc[2][kMaxTiles8][4], ones[kMaxTiles8][4];
#pragma unroll
        for (int j = 0; j < kMaxTiles8; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[0][j][i] = acc[1][j][i] = ones[j][i] = 0.0f;
#pragma unroll
        for (int b = group * kBlocks; b < (group + 1) * kBlocks; ++b) {
            uint32_t v[2][8];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t at = codes + h * half_bytes + ((b ^ g) << 4);
                const uint32_t lo = load_shared(at), hi = load_shared(at + 8 * 128);
                v[h][0] = two_values<kForm, 0>(lo);
                v[h][1] = two_values<kForm, 0>(hi);
                v[h][2] = two_values<kForm, 1>(lo);
                v[h][3] = two_values<kForm, 1>(hi);
                v[h][4] = two_values<kForm, 2>(lo);
                v[h][5] = two_values<kForm, 2>(hi);
                v[h][6] = two_values<kForm, 3>(lo);
                v[h][7] = two_values<kForm, 3>(hi);
            }
#pragma unroll
            for (int j = 0; j < kMaxTiles8; ++j) {
                if (j >= tiles8) break;
                const uint4 r = load_shared4(x_row[j] + b * 64);
                const uint32_t b0 = __byte_perm(r.x, r.z, 0x5410), b1 = __byte_perm(r.x, r.z, 0x7632);
                const uint32_t b2 = __byte_perm(r.y, r.w, 0x5410), b3 = __byte_perm(r.y, r.w, 0x7632);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    mma16(acc[h][j], v[h][0], v[h][1], v[h][2], v[h][3], b0, b1);
                    mma16(acc[h][j], v[h][4], v[h][5], v[h][6], v[h][7], b2, b3);
                }
                if (kForm == EP_W4_INT) {
                    mma16(ones[j], 0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u, b0, b1);
                    mma16(ones[j], 0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u, b2, b3);
                }
            }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t at = sf_at + h * sf_half + group * width * item;
            const float s0 = load_scale(stage + p.sf_offset + at, 0, p.sf_fp32);
            const float s1 = load_scale(stage + p.sf_offset + at, 8, p.sf_fp32);
            float z0 = -24.0f, z1 = -24.0f;
            if (kForm == EP_W4_INT && p.has_zero) {
                z0 = -16.0f - load_scale(stage + p.zero_offset + at, 0, p.sf_fp32);
                z1 = -16.0f - load_scale(stage + p.zero_offset + at, 8, p.sf_fp32);
            }
#pragma unroll
            for (int j = 0; j < kMaxTiles8; ++j) {
                if (j >= tiles8) break;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float sum = kForm == EP_W4_INT ? fmaf(i < 2 ? z0 : z1, ones[j][i & 1], acc[h][j][i]) : acc[h][j][i];
                    total[h][j][i] = fmaf(i < 2 ? s0 : s1, sum, total[h][j][i]);
                }
            }
        }
    }
}

template <int kForm, int kBlocks>
__global__ void __launch_bounds__(kThreads, 1) experts_w4_kernel(const __grid_constant__ Args p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* const stages = smem_raw + (1024 - (smem_addr(smem_raw) & 1023)) % 1024;
    float* const sums = reinterpret_cast<float*>(stages + p.stages * p.stage_bytes);
    Shared* const s = reinterpret_cast<Shared*>(reinterpret_cast<uint8_t*>(sums) + (p.slots > 1 ? kSumsBytes : 0));
    Table t;
    t.tile_end = reinterpret_cast<int*>(s + 1);
    t.first = t.tile_end + p.E;
    t.count = t.first + p.E;
    t.list = reinterpret_cast<int16_t*>(t.count + p.E);
    t.expert = t.list + p.T * p.topk;
    const int warp = uniform_warp(), lane = threadIdx.x & 31;
    const bool few = p.mode != kProduct, gated = p.act == EP_ACT_SWIGLU;
    const int pieces = kMmaWarps / p.slots;
    const int half = pieces * 16, tile_features = gated ? half : 2 * half;
    const int feature_tiles = (p.N + tile_features - 1) / tile_features;
    const int steps = (p.K + kSlotK * p.slots - 1) / (kSlotK * p.slots);

    if (threadIdx.x == 0) {
        for (int i = 0; i < p.stages; ++i) {
            mbar_init(&s->full[i], 1 + kCopyWarps * 32);
            mbar_init(&s->empty[i], kMmaWarps);
        }
        for (int i = 0; i < 2; ++i)
            for (int m = 0; m < pieces; ++m) {
                mbar_init(&s->sums_full[i][m], p.slots > 1 ? p.slots - 1 : 1);
                mbar_init(&s->sums_empty[i][m], 1);
            }
        fence_mbar_init();
        prefetch_map(&p.codes);
        prefetch_map(&p.scales);
    }
    // The down product's kernel may start, and route, once every CTA of the
    // up product's has seen its own inputs complete ("Reads before the wait").
    if (p.mode != kFewDown) {
        pdl_wait();
        pdl_launch_dependents();
    }
    if (few) {
        const int entries = p.T * p.topk;
        for (int i = threadIdx.x; i < entries; i += kThreads) {
            const int64_t e = __ldcg(reinterpret_cast<const long long*>(p.topk_idx) + i);   // (may come before the wait)
            const bool ok = e >= 0 && e < p.E;
            if (!ok && e != -1 && p.mode == kFewUp && blockIdx.x == 0) atomicOr(p.status, EP_ERR_INVALID_INDEX);
            t.expert[i] = ok ? static_cast<int16_t>(e) : static_cast<int16_t>(-1);
        }
        for (int e = threadIdx.x; e < p.E; e += kThreads) t.count[e] = 0;
        __syncthreads();
        for (int i = threadIdx.x; i < entries; i += kThreads)
            if (t.expert[i] >= 0) atomicAdd(&t.count[t.expert[i]], 1);
        __syncthreads();
        scan_experts<kThreads>(p.E, t.first, s->warp_sum, [&](int e) { return t.count[e]; });
        // first[e] is where e's entries end; filled from the last one down, in
        // the order of (token, slot), it becomes where they begin: every CTA
        // has to give a tile the same rows
        if (warp == 0)
            for (int i0 = (entries - 1) / 32 * 32; i0 >= 0; i0 -= 32) {
                const int i = i0 + lane, e = i < entries ? t.expert[i] : -1;
                const unsigned same = __match_any_sync(0xffffffffu, e);
                if (e >= 0) t.list[t.first[e] - __popc(same >> lane)] = static_cast<int16_t>(i);
                __syncwarp();
                if (e >= 0 && (same >> lane) == 1u) t.first[e] -= __popc(same);
                __syncwarp();
            }
        __syncthreads();
    } else {
        expert_blocks<kThreads>(p.expert_offset, p.counts, p.E, p.rows, t.first, t.count, s->warp_rows, p.status);
    }
    scan_experts<kThreads>(p.E, t.tile_end, s->warp_sum, [&](int e) { return (t.count[e] + p.tile_rows - 1) / p.tile_rows; });
    const int64_t tiles = static_cast<int64_t>(t.tile_end[p.E - 1]) * feature_tiles;
    if (p.mode == kFewDown) {
        if (warp != 0) pdl_wait();
        pdl_launch_dependents();
    }

    int stage = 0;
    uint32_t parity = 0;
    const auto next = [&] {
        if (++stage == p.stages) {
            stage = 0;
            parity ^= 1;
        }
    };
    if (warp == 0) {
        int issued = 0;
        bool ok = true;
        const int groups = 8 / kBlocks * p.slots;
        const int sf_bytes = 2 * groups * half * (p.sf_fp32 ? 4 : 2);
        const uint32_t bytes = kCodeBytes + sf_bytes * (p.has_zero ? 2 : 1);
        for (int64_t g = blockIdx.x; g < tiles && ok; g += gridDim.x) {
            const Tile r = tile_at(p, t, g, feature_tiles, tile_features);
            const int second = gated ? p.N + r.f0 : r.f0 + half;
            for (int step = 0; step < steps; ++step, ++issued, next()) {
                ok = warp_wait(&s->empty[stage], parity ^ 1);
                if (!ok) break;
                uint8_t* const at = stages + stage * p.stage_bytes;
                const uint32_t bar = smem_addr(&s->full[stage]);
                if (elect_one()) {
                    mbar_arrive_expect_tx(&s->full[stage], bytes);
                    for (int h = 0; h < 2; ++h) {
                        const int f = h == 0 ? r.f0 : second;
                        for (int i = 0; i < p.slots; ++i)
                            tma_load_3d<1>(at + h * (kCodeBytes / 2) + i * half * 128, &p.codes, bar,
                                           (step * p.slots + i) * (kSlotK / 2), f, r.e);
                        tma_load_3d<1>(at + p.sf_offset + h * (sf_bytes / 2), &p.scales, bar, f, step * groups, r.e);
                        if (p.has_zero)
                            tma_load_3d<1>(at + p.zero_offset + h * (sf_bytes / 2), &p.zeros, bar, f, step * groups, r.e);
                    }
                }
                __syncwarp();
            }
        }
        if (!ok) atomicOr(p.status, EP_ERR_TIMEOUT);
        if (p.mode == kFewDown) pdl_wait();
        // no copy may still be in flight when the CTA ends
        for (int i = max(0, issued - p.stages); i < issued; ++i)
            if (!warp_wait(&s->full[i % p.stages], (i / p.stages) & 1)) break;
    } else if (warp <= kCopyWarps) {
        const int tid = threadIdx.x - 32, chunks = 32 * p.slots;      // 16-byte pieces of a row in a stage
        const int chunk = tid & (chunks - 1), row0 = tid / chunks, row_step = kCopyWarps * 32 / chunks;
        constexpr int kMost = 8;      // rows of one thread: tile_rows <= 32 / slots
        bool ok = true;
        bool drop = kTestDropFirstLoad && blockIdx.x == 0;
        for (int64_t g = blockIdx.x; g < tiles && ok; g += gridDim.x) {
            const Tile r = tile_at(p, t, g, feature_tiles, tile_features);
            int64_t from[kMost];
#pragma unroll
            for (int i = 0; i < kMost; ++i) {
                const int row = row0 + i * row_step;
                from[i] = -1;
                if (row < r.rows) {
                    const int at = r.first + row, entry = few ? t.list[at] : 0;
                    const int64_t source = !few ? at : p.mode == kFewUp ? entry / p.topk : entry;
                    if (EP_IN(source, p.mode == kFewUp ? p.T : few ? p.T * p.topk : p.rows)) from[i] = source * p.K;
                }
            }
            for (int step = 0; step < steps; ++step, next()) {
                ok = warp_wait(&s->empty[stage], parity ^ 1);
                if (!ok) break;
                if (drop) {
                    drop = false;
                    continue;
                }
                const int k = step * kSlotK * p.slots + chunk * 8;
                const bool inside = k < p.K;
                const uint32_t to = smem_addr(stages + stage * p.stage_bytes) + p.x_offset +
                                    (chunk >> 5) * p.tile_rows * kRowPitch + row0 * kRowPitch + (chunk & 31) * 16;
#pragma unroll
                for (int i = 0; i < kMost; ++i)
                    if (from[i] >= 0)
                        copy16_async(to + i * row_step * kRowPitch, p.x + from[i] + (inside ? k : 0), inside);
                copies_arrive(&s->full[stage]);
            }
        }
        if (!ok) atomicOr(p.status, EP_ERR_TIMEOUT);
        copies_commit();
        copies_wait<0>();
    } else {
        const int w = warp - 1 - kCopyWarps, piece = w % pieces, slot = w / pieces;
        const int g8 = lane >> 2, t2 = (lane & 3) * 2;
        int turn = 0;
        bool ok = true;
        for (int64_t g = blockIdx.x; g < tiles; g += gridDim.x, ++turn) {
            const Tile r = tile_at(p, t, g, feature_tiles, tile_features);
            const int tiles8 = (r.rows + 7) / 8;
            float total[2][kMaxTiles8][4];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int j = 0; j < kMaxTiles8; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) total[h][j][i] = 0.0f;
            for (int step = 0; step < steps; ++step, next()) {
                ok = warp_wait(&s->full[stage], parity);
                if (!ok) break;
                if ((step * p.slots + slot) * kSlotK < p.K)
                    multiply_stage<kForm, kBlocks>(p, smem_addr(stages + stage * p.stage_bytes), tiles8, piece, slot, lane,
                                                   total);
                __syncwarp();
                if (lane == 0) mbar_arrive(&s->empty[stage]);
            }
            if (!ok) break;
            if (p.slots > 1) {
                // the shares' sums meet in the first share's warp, in their order
                const int buffer = turn & 1;
                const uint32_t use = (turn >> 1) & 1;
                float* const mine = sums + buffer * 4096 + piece * (2 * kMaxTiles8 * 4 * 32 / p.slots) + lane;
                const int per_slot = kMmaWarps * 2 * kMaxTiles8 * 4 * 32 / (p.slots * p.slots);
                if (slot > 0) {
                    ok = warp_wait(&s->sums_empty[buffer][piece], use ^ 1);
                    if (!ok) break;
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int j = 0; j < kMaxTiles8; ++j) {
                            if (j >= tiles8) break;
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                mine[(slot - 1) * per_slot + ((j * 2 + h) * 4 + i) * 32] = total[h][j][i];
                        }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&s->sums_full[buffer][piece]);
                    continue;
                }
                ok = warp_wait(&s->sums_full[buffer][piece], use);
                if (!ok) break;
                for (int other = 0; other < p.slots - 1; ++other)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int j = 0; j < kMaxTiles8; ++j) {
                            if (j >= tiles8) break;
#pragma unroll
                            for (int i = 0; i < 4; ++i) total[h][j][i] += mine[other * per_slot + ((j * 2 + h) * 4 + i) * 32];
                        }
                __syncwarp();
                if (lane == 0) mbar_arrive(&s->sums_empty[buffer][piece]);
            }
            // features f and f + 8 of each half, rows 8 j + t2 and the next one
#pragma unroll
            for (int up = 0; up < 2; ++up) {
                const int f = r.f0 + piece * 16 + g8 + up * 8;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (h == 1 && gated) break;
                    const int feature = f + h * half;
                    if (feature >= p.N) continue;
                    const float* const bias = p.bias ? p.bias + static_cast<int64_t>(r.e) * p.Nw + feature : nullptr;
                    const float b0 = bias ? bias[0] : 0.0f, b1 = bias && gated ? bias[p.N] : 0.0f;
#pragma unroll
                    for (int j = 0; j < kMaxTiles8; ++j) {
                        if (j >= tiles8) break;
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int row = j * 8 + t2 + i;
                            if (row >= r.rows) continue;
                            const float z = total[h][j][up * 2 + i] + b0;
                            float a = gated ? silu(z) * (total[1][j][up * 2 + i] + b1) : activate(z, p.act);
                            const int64_t at = few ? t.list[r.first + row] : r.first + row;
                            if (!EP_IN(at, few ? static_cast<int64_t>(p.T) * p.topk : p.rows)) continue;
                            if (p.mode == kProduct) {
                                if (p.row_weight) a *= p.row_weight[at];
                                if (p.residual) a += __bfloat162float(p.residual[at * p.N + feature]);
                            }
                            if (p.mode == kFewDown)
                                p.part[at * p.N + feature] = a;
                            else
                                p.y[at * p.N + feature] = __float2bfloat16_rn(a);
                        }
                    }
                }
            }
        }
        if (!ok) atomicOr(p.status, EP_ERR_TIMEOUT);
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

bool weight_maps(Args* a, const Weights4& w) {
    const int rows = kMmaWarps / a->slots * 16, item = w.sf_fp32 ? 4 : 2;
    const uint64_t E = a->E, Nw = a->Nw, half = a->K / 2, groups = a->K / w.group;
    const uint64_t dims[3] = {half, Nw, E}, strides[2] = {half, half * Nw};
    const uint32_t box[3] = {128, static_cast<uint32_t>(rows), 1};
    if (!encode_map(&a->codes, true, 3, w.w, dims, strides, box)) return false;
    const uint64_t sf_dims[3] = {Nw, groups, E}, sf_strides[2] = {Nw * item, Nw * item * groups};
    const uint32_t sf_box[3] = {static_cast<uint32_t>(rows), static_cast<uint32_t>(kSlotK / w.group * a->slots), 1};
    if (!encode_plain_map(&a->scales, w.sf_fp32 != 0, 3, w.sf, sf_dims, sf_strides, sf_box)) return false;
    a->has_zero = w.zero != nullptr;
    a->sf_fp32 = w.sf_fp32;
    return !w.zero || encode_plain_map(&a->zeros, w.sf_fp32 != 0, 3, w.zero, sf_dims, sf_strides, sf_box);
}

// rows: of all experts; likely: of one of them; row_tiles: at least as many tiles as a tile's rows give.
template <typename Tiles>
cudaError_t launch(Args a, const Weights4& w, int64_t rows, int64_t likely, Tiles row_tiles, cudaStream_t stream) {
    const DeviceInfo& info = device_info();
    const auto up = [](int v, int to) { return (v + to - 1) / to * to; };
    a.slots = likely <= 8 ? 4 : likely <= 16 ? 2 : 1;
    while (a.slots > 1 && a.slots * kSlotK > a.K) a.slots /= 2;
    a.tile_rows = rows < 8 ? static_cast<int>(rows) : std::min(32 / a.slots, up(static_cast<int>(std::min<int64_t>(likely, 32)), 8));
    if (!weight_maps(&a, w)) return cudaErrorInvalidValue;
    const int half = kMmaWarps / a.slots * 16, item = w.sf_fp32 ? 4 : 2;
    const int sf_bytes = 2 * (kSlotK / w.group * a.slots) * half * item;
    a.x_offset = kCodeBytes;
    a.sf_offset = up(a.x_offset + a.slots * a.tile_rows * kRowPitch, 128);
    a.zero_offset = a.sf_offset + sf_bytes;
    a.stage_bytes = up(a.zero_offset + (w.zero ? sf_bytes : 0), 1024);
    const int fixed = 1024 + (a.slots > 1 ? kSumsBytes : 0) + static_cast<int>(sizeof(Shared)) + a.E * 12 +
                      a.T * a.topk * 4;
    a.stages = std::min(kMaxStages, (info.max_smem_optin - fixed) / a.stage_bytes);
    if (a.stages < 1) return cudaErrorInvalidValue;
    const size_t smem = static_cast<size_t>(fixed) + a.stages * a.stage_bytes;
    const int features = a.act == EP_ACT_SWIGLU ? half : 2 * half;
    const int64_t tiles = row_tiles(a.tile_rows) * ((a.N + features - 1) / features);
    const dim3 grid(static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>(tiles, info.num_sms))));
    const auto go = [&](auto kernel, std::atomic<bool>* ready) {
        const cudaError_t e = allow_all_smem(reinterpret_cast<const void*>(kernel), ready);
        return e != cudaSuccess ? e : launch_experts(kernel, grid, dim3(kThreads), smem, stream, 1, a);
    };
    static std::atomic<bool> ready[6][kMaxDevices];
    if (w.format == EP_W4_INT) {
        if (w.group == 128) return go(experts_w4_kernel<EP_W4_INT, 4>, ready[0]);
        if (w.group == 64) return go(experts_w4_kernel<EP_W4_INT, 2>, ready[1]);
        return go(experts_w4_kernel<EP_W4_INT, 1>, ready[2]);
    }
    if (w.group == 128) return go(experts_w4_kernel<EP_W4_FP, 4>, ready[3]);
    if (w.group == 64) return go(experts_w4_kernel<EP_W4_FP, 2>, ready[4]);
    return go(experts_w4_kernel<EP_W4_FP, 1>, ready[5]);
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
    return launch(a, p.w, p.rows, likely, [&](int rows) { return p.rows / rows + p.E; }, stream);
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
    const auto tiles = [&](int rows) { return static_cast<int64_t>(entries) / rows + active; };
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
    const int64_t outs = static_cast<int64_t>(p.T) * p.H;
    return launch_pdl(few_sum_kernel, dim3(static_cast<unsigned>((outs + 255) / 256)), dim3(256), 0, stream, p);
}

}  // namespace epg
