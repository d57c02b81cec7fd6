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
//   int  u or 16 u as the low bits of a bf16 is that many 2^-133; one
//        multiply-add of two gives (u - 8) 2^-6.  Zero points come off once a
//        group, by the sum of the group's x, which one more MMA gives (a row
//        operand of ones).
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
// A CTA walks tiles (expert, rows, features).  Warp 0 asks for codes, scales and
// zero points by tensor maps, warps 0 and 1 copy the rows, 16 bytes a lane
// (bulk copies of a row's 256 bytes: 64 experts of 8 rows 271 -> 480 us),
// into a ring of stages.  Teams of eight warps multiply, a stage a team in
// turn: a stage is `slots` shares of 128 k's, a share 8 / slots pieces of
// features (two halves: gate and up for SWIGLU).  Many shares: tiles of few
// features, which fill the SMs evenly, but rows are read for each tile
// again.  The warps leave their sums in shared memory for warps 2 and 3, which
// add the shares in their order and finish the outputs under the next
// tile's products.
#include <cmath>
#include <type_traits>

#include "experts_w4.cuh"
#include "tcgen05.cuh"

namespace epg {

namespace {

constexpr int kFirstFinishWarp = 2, kFinishWarps = 2, kFirstTeamWarp = kFirstFinishWarp + kFinishWarps;
constexpr int kIntZero = 2;                   // EP_W4_INT with zero points, as a kernel's form
constexpr int kTeam = 8;                     // multiplying warps that share a stage
constexpr int kMaxStages = 12;
constexpr int kSlotK = 128;                  // k's of a share in one stage: 64 bytes of codes
constexpr int kRowPitch = kSlotK * 2 + 64;   // a row's share: eight lanes' reads of two rows meet all banks

// A variant of the kernel.  kPieces16: pieces of 16 features in a half of a warp's features; kTiles8: row tiles of
// 8 in a tile; kTeams: teams of warps that take stages in turn.
template <int kPieces16_, int kTiles8_, int kTeams_>
struct Variant {
    static_assert(kTeams_ == 1 || kTeams_ == 2, "which team a step is follows from its parity");
    static constexpr int kPieces16 = kPieces16_, kTiles8 = kTiles8_, kTeams = kTeams_;
    static constexpr int kThreads = (kFirstTeamWarp + kTeam * kTeams) * 32;
    static constexpr int kCodeBytes = kTeam * 32 * kPieces16 * (kSlotK / 2);   // of a stage
    static constexpr int kSums = 2 * kPieces16 * kTiles8 * 4;                  // of a lane
};
using Few = Variant<2, 1, 2>;      // up to 8 rows of an expert
using Wide = Variant<1, 4, 1>;     // up to 32

#ifdef EP_TEST_DROP_FIRST_LOAD
constexpr bool kTestDropFirstLoad = true;
#else
constexpr bool kTestDropFirstLoad = false;
#endif

enum Mode { kProduct, kFewUp, kFewDown };

struct Args {
    CUtensorMap codes;           // [E][Nw][K / 2], boxes of 64 bytes x the features of a half
    CUtensorMap scales, zeros;   // [E][K / group][Nw]
    const __nv_bfloat16* x;
    const float* bias;           // [E][Nw] or null
    int mode, K, N, Nw, E, act;  // depth, features out, features of the weights
    int sf_fp32;
    int whole;                   // a row of codes is whole pieces of 64 bytes
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
    // A stage's uses go to the teams in turn, so one that does not look at every use needs two barriers: with one, a
    // use's end would pass for the end of the next but one, whose parity is the same.
    uint64_t full[kMaxStages][2], empty[kMaxStages];
    uint64_t sums_full, sums_empty;
    int64_t warp_rows[32];
    int warp_sum[32];
};

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

// warp_wait that leaves the issue slots to the warps that multiply: the barrier
// may hold a waiting warp for as long as the hint says.
__device__ __forceinline__ bool wait_quietly(uint64_t* bar, uint32_t parity) {
    const auto done = [&] {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(smem_addr(bar)), "r"(parity), "r"(100000u)
            : "memory");
        return ok != 0;
    };
    bool ok = done();
    if (!ok) {
        const uint64_t t0 = global_timer_ns();
        for (uint32_t i = 0; i < (1u << 30) && !ok; ++i) {
            ok = done();
            if (!ok && global_timer_ns() - t0 > kWaitTimeoutNs) break;
        }
    }
    return __all_sync(0xffffffffu, ok ? 1 : 0) != 0;
}

// Codes i and i + 4 of a word as two bf16 values: (u - 8) 2^-6, or the FP4 value.
template <int kForm, int i>
__device__ __forceinline__ uint32_t two_values(uint32_t w) {
    uint32_t v;
    if (kForm != EP_W4_FP) {
        // bf16's numbers below 2^-125 are their bits times 2^-133: a code in the
        // low 8 bits is u or 16 u of those, times 2^127 or 2^123
        const uint32_t bits = (i < 2 ? w : w >> 8) & (i % 2 == 0 ? 0x000f000fu : 0x00f000f0u);
        asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(v) : "r"(bits), "r"(i % 2 == 0 ? 0x7f007f00u : 0x7d007d00u), "r"(0xbe00be00u));
        return v;
    }
    const uint32_t sign = i == 3 ? w : w << (12 - 4 * i);
    const uint32_t rest = i < 2 ? w << (i < 2 ? 6 - 4 * i : 0) : w >> (i < 2 ? 0 : 4 * i - 6);
    const uint32_t small = (sign & 0x80008000u) | (rest & 0x01c001c0u);
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

// d = a b, the first of a sum.
__device__ __forceinline__ void mma16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                            uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

// Where a lane of a team's warp reads in a stage.
template <class V>
struct Place {
    uint32_t codes;              // feature g of the piece, word t of block (g / 2) % 4: block b is at this ^ b * 16
    uint32_t x[V::kTiles8];      // (rows that are not there may be any: their columns are not kept)
    uint32_t half;               // to the second half's codes
    uint32_t sf, sf_half;        // scales, and to the second half's; a group's are both halves'
};

// One stage of one warp's share: kBlocks blocks of 32 k's a group, kTiles row tiles of 8; `left` k's are there.
template <int kForm, int kBlocks, int kTiles, class V>
__device__ __forceinline__ void multiply_stage(const Args& p, uint32_t stage, const Place<V>& at, int left,
                                               float (&total)[2][V::kPieces16][V::kTiles8][4]) {
    constexpr int kM = V::kPieces16, kGroups = kSlotK / 32 / kBlocks;
    const uint32_t codes = stage + at.codes;
    const int item = p.sf_fp32 ? 4 : 2;
#pragma unroll
    for (int group = 0; group < kGroups; ++group) {
        if (kGroups > 1 && group * kBlocks * 32 >= left) break;      // (what is not there is not loaded either)
        float acc[2][kM][kTiles][4], ones[kTiles][4];
#pragma unroll
        for (int b = group * kBlocks; b < (group + 1) * kBlocks; ++b) {
            const bool first = b == group * kBlocks;
            uint32_t x0[kTiles], x1[kTiles], x2[kTiles], x3[kTiles];
#pragma unroll
            for (int j = 0; j < kTiles; ++j) {
                const uint4 r = load_shared4(stage + at.x[j] + b * 64);
                x0[j] = __byte_perm(r.x, r.z, 0x5410);
                x1[j] = __byte_perm(r.x, r.z, 0x7632);
                x2[j] = __byte_perm(r.y, r.w, 0x5410);
                x3[j] = __byte_perm(r.y, r.w, 0x7632);
                constexpr uint32_t kOnes = 0x3f803f80u;
                if (kForm == kIntZero) {
                    if (first)
                        mma16_first(ones[j], kOnes, kOnes, kOnes, kOnes, x0[j], x1[j]);
                    else
                        mma16(ones[j], kOnes, kOnes, kOnes, kOnes, x0[j], x1[j]);
                    mma16(ones[j], kOnes, kOnes, kOnes, kOnes, x2[j], x3[j]);
                }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int m = 0; m < kM; ++m) {
                    const uint32_t from = (codes ^ (b << 4)) + h * at.half + m * 16 * (kSlotK / 2);
                    const uint32_t lo = load_shared(from), hi = load_shared(from + 8 * (kSlotK / 2));
                    const uint32_t v0 = two_values<kForm, 0>(lo), v1 = two_values<kForm, 0>(hi);
                    const uint32_t v2 = two_values<kForm, 1>(lo), v3 = two_values<kForm, 1>(hi);
                    const uint32_t v4 = two_values<kForm, 2>(lo), v5 = two_values<kForm, 2>(hi);
                    const uint32_t v6 = two_values<kForm, 3>(lo), v7 = two_values<kForm, 3>(hi);
#pragma unroll
                    for (int j = 0; j < kTiles; ++j) {
                        if (first)
                            mma16_first(acc[h][m][j], v0, v1, v2, v3, x0[j], x1[j]);
                        else
                            mma16(acc[h][m][j], v0, v1, v2, v3, x0[j], x1[j]);
                        mma16(acc[h][m][j], v4, v5, v6, v7, x2[j], x3[j]);
                    }
                }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int m = 0; m < kM; ++m) {
                const uint32_t from = stage + p.sf_offset + at.sf + (group * 2 + h) * at.sf_half + m * 16 * item;
                const float s0 = load_scale(from, 0, p.sf_fp32), s1 = load_scale(from, 8, p.sf_fp32);
                float z0 = 0.0f, z1 = 0.0f;
                if (kForm == kIntZero) {    // (8 - zero) 2^-6
                    const uint32_t zero = from + (p.zero_offset - p.sf_offset);
                    z0 = fmaf(load_scale(zero, 0, p.sf_fp32), -0.015625f, 0.125f);
                    z1 = fmaf(load_scale(zero, 8, p.sf_fp32), -0.015625f, 0.125f);
                }
#pragma unroll
                for (int j = 0; j < kTiles; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float sum =
                            kForm == kIntZero ? fmaf(i < 2 ? z0 : z1, ones[j][i & 1], acc[h][m][j][i]) : acc[h][m][j][i];
                        total[h][m][j][i] = fmaf(i < 2 ? s0 : s1, sum, total[h][m][j][i]);
                    }
            }
    }
}

template <int kForm, int kBlocks, class V>
__global__ void __launch_bounds__(V::kThreads, 1) experts_w4_kernel(const __grid_constant__ Args p) {
    constexpr int kM = V::kPieces16, kThreads = V::kThreads, kCodeBytes = V::kCodeBytes;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* const stages = smem_raw + (512 - (smem_addr(smem_raw) & 511)) % 512;
    float* const sums = reinterpret_cast<float*>(stages + p.stages * p.stage_bytes);
    const int pieces = kTeam / p.slots, shares = p.slots * V::kTeams;
    Shared* const s = reinterpret_cast<Shared*>(sums + shares * pieces * V::kSums * 32);
    Table t;
    t.tile_end = reinterpret_cast<int*>(s + 1);
    t.first = t.tile_end + p.E;
    t.count = t.first + p.E;
    t.list = reinterpret_cast<int16_t*>(t.count + p.E);
    t.expert = t.list + p.T * p.topk;
    const int warp = uniform_warp(), lane = threadIdx.x & 31;
    const bool few = p.mode != kProduct, gated = p.act == EP_ACT_SWIGLU;
    const int half = pieces * 16 * kM, tile_features = gated ? half : 2 * half;
    const int feature_tiles = (p.N + tile_features - 1) / tile_features;
    const int steps = (p.K + kSlotK * p.slots - 1) / (kSlotK * p.slots);

    if (threadIdx.x == 0) {
        for (int i = 0; i < p.stages; ++i) {
            for (int k = 0; k < 2; ++k)
                mbar_init(&s->full[i][k], 1 + 32);   // the tensor maps' bytes, and the rows' copies
            mbar_init(&s->empty[i], kTeam);
        }
        mbar_init(&s->sums_full, kTeam * V::kTeams);
        mbar_init(&s->sums_empty, kFinishWarps);
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
        if (warp != 0) pdl_wait();     // (warp 0 does when it has asked for its first weights)
        pdl_launch_dependents();
    }

    if (warp == 0) {
        const int groups = kSlotK / 32 / kBlocks * p.slots;
        const uint32_t bytes = kCodeBytes + 2 * groups * half * (p.sf_fp32 ? 4 : 2) * (kForm == kIntZero ? 2 : 1);
        const auto load_weights = [&](const Tile& r, int stage, uint32_t use, int step) {
            uint8_t* const at = stages + stage * p.stage_bytes;
            uint64_t* const full = &s->full[stage][use & 1];
            const uint32_t bar = smem_addr(full);
            const int byte = p.whole ? 0 : step * (kSlotK / 2), part = p.whole ? step * p.slots : 0;
            if (elect_one()) {
                mbar_arrive_expect_tx(full, bytes);
                if (gated) {
                    tma_load_5d<1>(at, &p.codes, bar, byte, r.f0, 0, part, r.e);
                    tma_load_4d(at + p.sf_offset, &p.scales, bar, r.f0, 0, step * groups, r.e);
                    if (kForm == kIntZero) tma_load_4d(at + p.zero_offset, &p.zeros, bar, r.f0, 0, step * groups, r.e);
                } else {
                    tma_load_4d(at, &p.codes, bar, byte, r.f0, part, r.e);
                    tma_load_3d<1>(at + p.sf_offset, &p.scales, bar, r.f0, step * groups, r.e);
                    if (kForm == kIntZero) tma_load_3d<1>(at + p.zero_offset, &p.zeros, bar, r.f0, step * groups, r.e);
                }
            }
            __syncwarp();
        };
        int stage = 0, issued = 0, early = 0;
        uint32_t use = 0;
        bool ok = true;
        if (p.mode == kFewDown) {
            // the down product's first weights come while the up product ends
            if (blockIdx.x < tiles) {
                const Tile r = tile_at(p, t, blockIdx.x, feature_tiles, tile_features);
                early = min(p.stages, steps);
                for (int i = 0; i < early; ++i) load_weights(r, i, 0, i);
            }
            pdl_wait();
        }
        for (int64_t g = blockIdx.x; g < tiles && ok; g += gridDim.x) {
            const Tile r = tile_at(p, t, g, feature_tiles, tile_features);
            for (int step = 0; step < steps; ++step, ++issued) {
                // (a stage that was asked for early may be empty again before this warp comes here: its wait, for the
                // use before, would be for the one after)
                if (issued >= early) {
                    ok = wait_quietly(&s->empty[stage], (use & 1) ^ 1);
                    if (!ok) break;
                    load_weights(r, stage, use, step);
                }
                if (++stage == p.stages) {
                    stage = 0;
                    ++use;
                }
            }
        }
        if (!ok) atomicOr(p.status, EP_ERR_TIMEOUT);
        // no copy may still be in flight when the CTA ends
        issued = max(issued, early);
        for (int i = max(0, issued - p.stages); i < issued; ++i)
            if (!wait_quietly(&s->full[i % p.stages][i / p.stages & 1], (i / p.stages >> 1) & 1)) break;
    } else if (warp == 1) {
        // 16-byte pieces of a row in a stage; rows of a lane
        const int chunks = kSlotK / 8 * p.slots, passes = (chunks + 31) / 32, lane_rows = chunks < 32 ? 32 / chunks : 1;
        const int row0 = chunks < 32 ? lane / chunks : 0, chunk0 = lane & (chunks - 1);
        int stage = 0;
        uint32_t use = 0;
        bool ok = true;
        bool drop = kTestDropFirstLoad && blockIdx.x == 0;
        for (int64_t g = blockIdx.x; g < tiles && ok; g += gridDim.x) {
            const Tile r = tile_at(p, t, g, feature_tiles, tile_features);
            constexpr int kMost = 16;       // rows of a lane: two rows at a time where a share is all there is
            const __nv_bfloat16* from[kMost];
#pragma unroll
            for (int i = 0; i < kMost; ++i) {
                const int row = row0 + i * lane_rows;
                from[i] = nullptr;
                if (row < r.rows) {
                    const int at = r.first + row, entry = few ? t.list[at] : at;
                    const int64_t source = p.mode == kFewUp ? entry / p.topk : entry;
                    if (EP_IN(source, p.mode == kFewUp ? p.T : few ? p.T * p.topk : p.rows)) from[i] = p.x + source * p.K;
                }
            }
            for (int step = 0; step < steps; ++step) {
                ok = wait_quietly(&s->empty[stage], (use & 1) ^ 1);
                if (!ok) break;
                if (!drop) {
                    for (int pass = 0; pass < passes; ++pass) {
                        const int chunk = chunk0 + pass * 32, k = step * kSlotK * p.slots + chunk * 8;
                        const bool inside = k < p.K;
                        const uint32_t to = smem_addr(stages) + stage * p.stage_bytes + p.x_offset +
                                            (chunk / (kSlotK / 8) * p.tile_rows + row0) * kRowPitch +
                                            chunk % (kSlotK / 8) * 16;
#pragma unroll
                        for (int i = 0; i < kMost; ++i) {
                            if (i * lane_rows >= r.rows) break;
                            if (from[i]) copy16_async(to + i * lane_rows * kRowPitch, from[i] + (inside ? k : 0), inside);
                        }
                    }
                    copies_arrive(&s->full[stage][use & 1]);
                }
                drop = false;
                if (++stage == p.stages) {
                    stage = 0;
                    ++use;
                }
            }
        }
        if (!ok) atomicOr(p.status, EP_ERR_TIMEOUT);
        copies_commit();
        copies_wait<0>();       // none may still be in flight when the CTA ends
    } else if (warp >= kFirstTeamWarp) {
        const int w = (warp - kFirstTeamWarp) % kTeam, team = (warp - kFirstTeamWarp) / kTeam;
        const int piece = w % pieces, slot = w / pieces, g8 = lane >> 2, t4 = lane & 3;
        Place<V> at;
        at.codes = (slot * 2 * half + piece * 16 * kM + g8) * (kSlotK / 2) + ((g8 >> 1) & 3) * 16 + t4 * 4;
        at.half = half * (kSlotK / 2);
#pragma unroll
        for (int j = 0; j < V::kTiles8; ++j)
            at.x[j] = p.x_offset + (slot * p.tile_rows + min(j * 8 + g8, p.tile_rows - 1)) * kRowPitch + t4 * 16;
        const int item = p.sf_fp32 ? 4 : 2, groups = kSlotK / 32 / kBlocks;
        at.sf = (slot * groups * 2 * half + piece * 16 * kM + g8) * item;
        at.sf_half = half * item;
        float* const mine = sums + ((team * p.slots + slot) * pieces + piece) * V::kSums * 32;
        int stage = team % p.stages, before = 0;      // steps of the tiles before, modulo the teams
        uint32_t use = team / p.stages, turn = 0;
        bool ok = true;
        for (int64_t g = blockIdx.x; g < tiles; g += gridDim.x, turn ^= 1) {
            const int tiles8 = (tile_at(p, t, g, feature_tiles, tile_features).rows + 7) / 8;
            float total[2][kM][V::kTiles8][4];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int m = 0; m < kM; ++m)
#pragma unroll
                    for (int j = 0; j < V::kTiles8; ++j)
#pragma unroll
                        for (int i = 0; i < 4; ++i) total[h][m][j][i] = 0.0f;
            for (int step = V::kTeams == 2 ? team ^ before : 0; step < steps; step += V::kTeams) {
                ok = wait_quietly(&s->full[stage][use & 1], (use >> 1) & 1);
                if (!ok) break;
                const int left = p.K - (step * p.slots + slot) * kSlotK;
                if (left > 0) {
                    const uint32_t from = smem_addr(stages) + stage * p.stage_bytes;
                    if (V::kTiles8 == 1 || tiles8 <= 1)
                        multiply_stage<kForm, kBlocks, 1, V>(p, from, at, left, total);
                    else if (tiles8 == 2)
                        multiply_stage<kForm, kBlocks, V::kTiles8 < 2 ? 1 : 2, V>(p, from, at, left, total);
                    else
                        multiply_stage<kForm, kBlocks, V::kTiles8, V>(p, from, at, left, total);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&s->empty[stage]);
                stage += V::kTeams;
                while (stage >= p.stages) {
                    stage -= p.stages;
                    ++use;
                }
            }
            if (!ok) break;
            if (V::kTeams > 1) before = (before + steps) & 1;
            ok = wait_quietly(&s->sums_empty, turn ^ 1);
            if (!ok) break;
#pragma unroll
            for (int j = 0; j < V::kTiles8; ++j) {
                if (j >= tiles8) break;
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int m = 0; m < kM; ++m)
#pragma unroll
                        for (int i = 0; i < 4; ++i)     // (see the reader's banks)
                            mine[(((j * 2 + h) * kM + m) * 4 + i) * 32 + (lane ^ (((piece * kM + m) * 2 + i / 2) & 3))] =
                                total[h][m][j][i];
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&s->sums_full);
        }
        if (!ok) atomicOr(p.status, EP_ERR_TIMEOUT);
    } else {
        // What the teams' sums become: the shares in their order, bias, activation, row weight and residual.  A
        // lane is a feature, so that 32 of them are stored together; a feature's place in the sums is piece, m, up
        // (eight features on) and g (lane g * 4 + t of the MMA's result, t by row), and 32 features' reads meet all
        // banks by what the writers added to t.  Two warps have a tile's time for it, so the loops are
        // short of branches and instructions (one output a lane and turn, its place by divisions: 64
        // experts of 4 rows, 2048 -> 7168, 158 us).
        const auto finish = [&](auto gate, const Tile& r) {
            constexpr bool kGate = decltype(gate)::value;
            const int chunks = half / 32 * (kGate ? 1 : 2), share_step = pieces * V::kSums * 32;
            for (int chunk = warp - kFirstFinishWarp; chunk < chunks; chunk += kFinishWarps) {
                const int h = kGate ? 0 : chunk & 1, f = (kGate ? chunk : chunk >> 1) * 32 + lane;     // in the half
                const int feature = r.f0 + h * half + f;
                if (feature >= p.N) continue;
                const float* const bias = p.bias ? p.bias + static_cast<int64_t>(r.e) * p.Nw + feature : nullptr;
                const float b0 = bias ? bias[0] : 0.0f, b1 = kGate && bias ? bias[p.N] : 0.0f;
                const float* const base = sums + (f / (16 * kM) * V::kSums + (h * kM + f / 16 % kM) * 4 + (f >> 3 & 1) * 2) * 32 +
                                          (f & 7) * 4;
                const int turn = f >> 3 & 3;
#pragma unroll 2
                for (int row = 0; row < r.rows; ++row) {
                    const float* from = base + (row >> 3) * (2 * kM * 4 * 32) + (row & 1) * 32 + ((row >> 1 & 3) ^ turn);
                    float z = 0.0f, other = 0.0f;
                    for (int share = 0; share < shares; share += 2, from += 2 * share_step) {
                        z += from[0];
                        if (kGate) other += from[kM * 4 * 32];
                        if (share + 1 < shares) {
                            z += from[share_step];
                            if (kGate) other += from[share_step + kM * 4 * 32];
                        }
                    }
                    constexpr float kScale = kForm != EP_W4_FP ? 64.0f : 1.0f;
                    z = fmaf(z, kScale, b0);
                    float a = kGate ? silu(z) * fmaf(other, kScale, b1) : activate(z, p.act);
                    const int64_t to = few ? t.list[r.first + row] : r.first + row;
                    if (!EP_IN(to, few ? static_cast<int64_t>(p.T) * p.topk : p.rows)) continue;
                    const int64_t out = to * p.N + feature;
                    if (p.mode == kFewDown) {
                        p.part[out] = a;
                        continue;
                    }
                    if (p.row_weight) a *= p.row_weight[to];
                    if (p.residual) a += __bfloat162float(p.residual[out]);
                    p.y[out] = __float2bfloat16_rn(a);
                }
            }
        };
        uint32_t turn = 0;
        bool ok = true;
        for (int64_t g = blockIdx.x; g < tiles; g += gridDim.x, turn ^= 1) {
            const Tile r = tile_at(p, t, g, feature_tiles, tile_features);
            ok = wait_quietly(&s->sums_full, turn);
            if (!ok) break;
            if (gated)
                finish(std::true_type(), r);
            else
                finish(std::false_type(), r);
            __syncwarp();
            if (lane == 0) mbar_arrive(&s->sums_empty);
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
cudaError_t launch_variant(Args a, const Weights4& w, Tiles row_tiles, cudaStream_t stream) {
    const DeviceInfo& info = device_info();
    const auto up = [](int v, int to) { return (v + to - 1) / to * to; };
    const int pieces = kTeam / a.slots, half = pieces * 16 * V::kPieces16, item = w.sf_fp32 ? 4 : 2;
    if (!weight_maps(&a, w, half)) return cudaErrorInvalidValue;
    const int sf_bytes = 2 * (kSlotK / w.group * a.slots) * half * item;
    a.x_offset = V::kCodeBytes;
    a.sf_offset = up(a.x_offset + a.slots * a.tile_rows * kRowPitch, 128);
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
    const auto go = [&](auto form, auto blocks) {
        const auto kernel = experts_w4_kernel<decltype(form)::value, decltype(blocks)::value, V>;
        static std::atomic<bool> ready[kMaxDevices];
        const cudaError_t e = allow_all_smem(reinterpret_cast<const void*>(kernel), ready);
        return e != cudaSuccess ? e : launch_experts(kernel, grid, dim3(V::kThreads), smem, stream, 1, a);
    };
    const auto grouped = [&](auto form) {
        if (w.group == 128) return go(form, std::integral_constant<int, 4>());
        if (w.group == 64) return go(form, std::integral_constant<int, 2>());
        return go(form, std::integral_constant<int, 1>());
    };
    if (w.format == EP_W4_FP) return grouped(std::integral_constant<int, EP_W4_FP>());
    return w.zero ? grouped(std::integral_constant<int, kIntZero>()) : grouped(std::integral_constant<int, EP_W4_INT>());
}

// Shares for up to 8 rows of an expert: the least time of the CTAs' turns, a turn's tiles at what the memory gives
// the SMs at work (an SM takes no more than 100 bytes a ns), 0.8 us a tile, and the tile's rows at 60.  One row, [7168, 7168]
// by 2, 4, 8 shares: 31, 21, 17 us a call on its own; 8 experts of one row, 7168 -> 2 x 2048, SWIGLU, 37.5, 39.6, 43.6,
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
        const auto turn = [&](double ctas) { return bytes / std::min(100.0, 6780.0 / ctas) + 800.0 + rows / 60.0; };
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
    // two shares at least: one share's 512 features would be more than a box may have
    const bool few = likely <= 8 && a.whole && a.K >= 2 * kSlotK;
    a.tile_rows = rows < 8 ? static_cast<int>(rows) : likely <= 8 ? 8 : likely <= 16 ? 16 : 32;
    a.slots = few ? best_slots(a, row_tiles(a.tile_rows), likely) : !a.whole || likely > 16 || a.K < 2 * kSlotK ? 1 : 2;
    return few ? launch_variant<Few>(a, w, row_tiles, stream) : launch_variant<Wide>(a, w, row_tiles, stream);
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
