// The experts' products with 4-bit weights and group scales: the kernel.
//
// z[row, f] = sum over groups of scale[group, f] * sum over the group's k of (u[f, k] - zero[group, f]) x[row, k]
//
// A call reads half a byte a weight and has few rows to multiply it by, so the
// weights' bytes bound it if what is done to each weight is little: about 11
// of them a cycle go through each quarter of an SM at the memory's rate.  256
// experts of 4 rows, 7168 -> 2 x 2048, int with groups of 128: 600 us for 3.83
// GB, 6.4 TB/s.  Groups of 32 have four times the scales to apply to the sums,
// and FP4 rows to convert as well: 2048 -> 7168, 565 us for 2.1 GB, bound by
// the instructions' issue.
// Codes become bf16 values in registers, exactly, and meet the rows in the
// warp's own MMA (m16n8k16), whose operands are registers: tcgen05 would want
// the values written to shared or tensor memory first, twice the bytes that
// its wider tiles save on the few rows there are.
//   int  u or 16 u as the low bits of a bf16 is that many 2^-133; one
//        multiply-add of two gives (u - 8) 2^-6.  Zero points come off once a
//        group, by the sum of the group's x, which one more MMA gives (a row
//        operand of ones).
//   FP4  the hardware's conversion to fp16, a byte an instruction (moving the
//        bits by hand took twice as long); rows become fp16 too, in units of
//        a power of two for each row's 128 k's.
// Sums of a group stay in the MMA's fp32; the scale is applied in fp32.
//
// A word of eight int codes of one feature gives the pairs (k, k + 4), k = 0 .. 3:
// the operand's order of k is any that both sides share, so x is paired that
// way too (four byte permutations a 16-byte read).  32 k's are 16 bytes of a
// feature, a word for each of four lanes; the 64-byte swizzle lets 8
// features' reads meet all banks.
//
// A CTA walks tiles (expert, rows, features).  Warp 0 asks for codes, scales and
// zero points by tensor maps, warps 0 and 1 copy the rows, 16 bytes a lane (bulk
// copies of a row's 256 bytes: 64 experts of 8 rows 271 -> 480 us), for FP4
// through registers, where they become fp16, into a ring of stages.  Teams of eight warps multiply, a stage a team in
// turn: a stage is `slots` shares of 128 k's, a share 8 / slots pieces of
// features (two halves: gate and up for SWIGLU).  Many shares: tiles of few
// features, which fill the SMs evenly, but rows are read for each tile
// again.  The warps leave their sums in shared memory for warps 2 and 3, which
// add the shares in their order and finish the outputs under the next
// tile's products.
#pragma once

#include <type_traits>

#include "experts_w4.cuh"
#include "tcgen05.cuh"

namespace epg {

namespace w4 {

constexpr int kCopyWarps = 2, kFirstFinishWarp = kCopyWarps, kFinishWarps = 2, kFirstTeamWarp = kFirstFinishWarp + kFinishWarps;
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
using Mid = Variant<2, 2, 1>;      // up to 16
using Wide = Variant<1, 4, 1>;     // up to 32, and where a row of codes is not whole pieces of 64 bytes

#ifdef EP_TEST_DROP_FIRST_LOAD
constexpr bool kTestDropFirstLoad = true;
#else
constexpr bool kTestDropFirstLoad = false;
#endif

enum Mode { kProduct, kFewUp, kFewDown };
enum Which { kFew, kMid, kWide };      // the variant

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

// The launches of a form, each compiled in a file of its own.
cudaError_t launch_int(const Args& a, int group, Which which, dim3 grid, size_t smem, cudaStream_t stream);
cudaError_t launch_zero(const Args& a, int group, Which which, dim3 grid, size_t smem, cudaStream_t stream);
cudaError_t launch_fp(const Args& a, int group, Which which, dim3 grid, size_t smem, cudaStream_t stream);

struct Shared {
    // A stage's uses go to the teams in turn, so one that does not look at every use needs two barriers: with one, a
    // use's end would pass for the end of the next but one, whose parity is the same.
    uint64_t full[kMaxStages][2], empty[kMaxStages];
    uint64_t sums_full, sums_empty;
    int64_t warp_rows[32];
    int warp_sum[32];
    int listed;                  // experts in the table
    int16_t id[32];              // which they are, where they are at most 32; else expert i is the i-th
};

namespace {      // (a copy of the library for a test has kernels of its own)

struct Tile {
    int e, first, rows, f0;      // expert, its first row or entry here, how many, first feature
};

// The experts' row tiles: tile_end[i] = row tiles of the table's experts 0 .. i.
struct Table {
    int* tile_end;
    int* first;                  // first row, or first entry of the list
    int* count;
    int16_t* list;               // few: entries (token, slot), expert by expert
    int16_t* expert;             // few: expert of each entry, -1 for none
    const Shared* s;
};

// Tile g, by a whole warp.
__device__ __forceinline__ Tile tile_at(const Args& p, const Table& t, int64_t g, int feature_tiles, int tile_features,
                                        int lane) {
    const bool small = g <= INT32_MAX;
    const int row_tile = small ? static_cast<int>(g) / feature_tiles : static_cast<int>(g / feature_tiles);
    // the expert: the first with tile_end > row_tile, 32 at a time
    int lo = 0, n = t.s->listed;
    while (n > 1) {
        const int step = (n + 31) / 32, at = min(lo + (lane + 1) * step, lo + n) - 1;
        const int before = __popc(__ballot_sync(0xffffffffu, t.tile_end[at] <= row_tile));
        const int skip = min(before * step, n - 1);
        lo += skip;
        n = min(step, n - skip);
    }
    Tile r;
    r.e = t.s->listed <= 32 ? t.s->id[lo] : lo;
    const int start = lo > 0 ? t.tile_end[lo - 1] : 0, of = t.tile_end[lo] - start, at = row_tile - start;
    // an expert's tiles share its rows evenly, in steps of 8
    const int each = of > 1 ? min(p.tile_rows, ((t.count[lo] + of - 1) / of + 7) / 8 * 8) : t.count[lo];
    r.first = t.first[lo] + at * each;
    r.rows = max(0, min(each, t.count[lo] - at * each));
    r.f0 = static_cast<int>(g - static_cast<int64_t>(row_tile) * feature_tiles) * tile_features;
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

__device__ __forceinline__ void store_shared(uint32_t addr, uint32_t v) {
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void store_shared4(uint32_t addr, uint4 v) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
// Eight bf16 values of a lane as fp16 in units of a power of two, by all lanes of a warp: the largest of 16 lanes' (a
// row's 128 k's) comes to lie in [2^14, 2^15).  fp16 holds bf16's 8 bits down to 2^-31 of that one; what is smaller is
// off by 2^-39 of it at most, far below the last place of the fp32 sum that both go into.
__device__ __forceinline__ uint4 to_fp16(uint4 x, float* unit) {
    uint32_t largest = __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu), __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu));
    largest = max(largest >> 16, largest & 0xffffu);
#pragma unroll
    for (int o = 1; o < 16; o *= 2) largest = max(largest, __shfl_xor_sync(0xffffffffu, largest, o));
    const uint32_t e = min(max(largest >> 7, 15u), 254u);      // (infinities and NaN stay what they are)
    *unit = __uint_as_float((e - 14) << 23);
    const float by = __uint_as_float((268 - e) << 23);
    const auto two = [&](uint32_t v) {
        uint32_t r;
        asm("cvt.rn.f16x2.f32 %0, %1, %2;"
            : "=r"(r)
            : "f"(__uint_as_float(v & 0xffff0000u) * by), "f"(__uint_as_float(v << 16) * by));
        return r;
    };
    return make_uint4(two(x.x), two(x.y), two(x.z), two(x.w));
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

// Codes of a word as four pairs of 16-bit values.  int: codes i and i + 4 as bf16, (u - 8) 2^-6: bf16's numbers below
// 2^-125 are their bits times 2^-133, a code in the low 8 bits is u or 16 u of those, times 2^127 or 2^123.  FP4: codes
// 2 i and 2 i + 1 as fp16, by the hardware's conversion.
template <int kForm>
__device__ __forceinline__ void values_of(uint32_t w, uint32_t (&v)[4]) {
    if (kForm == EP_W4_FP) {
        asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
            "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
            "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
            : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
            : "r"(w));
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t bits = (i < 2 ? w : w >> 8) & (i % 2 == 0 ? 0x000f000fu : 0x00f000f0u);
        asm("fma.rn.bf16x2 %0, %1, %2, %3;"
            : "=r"(v[i])
            : "r"(bits), "r"(i % 2 == 0 ? 0x7f007f00u : 0x7d007d00u), "r"(0xbe00be00u));
    }
}

// d = a b + c for 16 features, 8 rows and 16 k's; without c for the first of a sum.
template <int kForm>
__device__ __forceinline__ void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1, bool first) {
#define EP_MMA16(type)                                                                                             \
    if (first)                                                                                                     \
        asm("mma.sync.aligned.m16n8k16.row.col.f32." type "." type ".f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "     \
            "{%8, %9}, {%10, %10, %10, %10};"                                                                      \
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])                                                       \
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));                                    \
    else                                                                                                           \
        asm("mma.sync.aligned.m16n8k16.row.col.f32." type "." type ".f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "     \
            "{%8, %9}, {%0, %1, %2, %3};"                                                                          \
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])                                                       \
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1))
    if (kForm == EP_W4_FP) {
        EP_MMA16("f16");
    } else {
        EP_MMA16("bf16");
    }
#undef EP_MMA16
}

// Where a lane of a team's warp reads in a stage.
template <class V>
struct Place {
    uint32_t codes;              // feature g of the piece, word t of block (g / 2) % 4: block b is at this ^ b * 16
    uint32_t x[V::kTiles8];      // (rows that are not there may be any: their columns are not kept)
    uint32_t half;               // to the second half's codes
    uint32_t unit[V::kTiles8];   // FP4: what the rows were multiplied by, of this lane's two rows
    uint32_t sf, sf_half;        // scales, and to the second half's; a group's are both halves'
};

// One stage of one warp's share: kBlocks blocks of 32 k's a group, kTiles row tiles of 8; `left` k's are there.
template <int kForm, int kBlocks, int kTiles, class V>
__device__ __forceinline__ void multiply_stage(const Args& p, uint32_t stage, const Place<V>& at, int left,
                                               float (&total)[2][V::kPieces16][V::kTiles8][4]) {
    constexpr int kM = V::kPieces16, kGroups = kSlotK / 32 / kBlocks;
    const uint32_t codes = stage + at.codes;
    const int item = p.sf_fp32 ? 4 : 2;
    float unit[kTiles][2];
    if (kForm == EP_W4_FP)
#pragma unroll
        for (int j = 0; j < kTiles; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i) unit[j][i] = __uint_as_float(load_shared(stage + at.unit[j] + i * 4));
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
                if (kForm == EP_W4_FP) {
                    x0[j] = r.x;
                    x1[j] = r.y;
                    x2[j] = r.z;
                    x3[j] = r.w;
                } else {
                    x0[j] = __byte_perm(r.x, r.z, 0x5410);
                    x1[j] = __byte_perm(r.x, r.z, 0x7632);
                    x2[j] = __byte_perm(r.y, r.w, 0x5410);
                    x3[j] = __byte_perm(r.y, r.w, 0x7632);
                }
                if (kForm == kIntZero) {
                    constexpr uint32_t kOnes = 0x3f803f80u;
                    mma16<kForm>(ones[j], kOnes, kOnes, kOnes, kOnes, x0[j], x1[j], first);
                    mma16<kForm>(ones[j], kOnes, kOnes, kOnes, kOnes, x2[j], x3[j], false);
                }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int m = 0; m < kM; ++m) {
                    const uint32_t from = (codes ^ (b << 4)) + h * at.half + m * 16 * (kSlotK / 2);
                    uint32_t lo[4], hi[4];
                    values_of<kForm>(load_shared(from), lo);
                    values_of<kForm>(load_shared(from + 8 * (kSlotK / 2)), hi);
#pragma unroll
                    for (int j = 0; j < kTiles; ++j) {
                        mma16<kForm>(acc[h][m][j], lo[0], hi[0], lo[1], hi[1], x0[j], x1[j], first);
                        mma16<kForm>(acc[h][m][j], lo[2], hi[2], lo[3], hi[3], x2[j], x3[j], false);
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
                        const float sum = kForm == kIntZero   ? fmaf(i < 2 ? z0 : z1, ones[j][i & 1], acc[h][m][j][i])
                                          : kForm == EP_W4_FP ? acc[h][m][j][i] * unit[j][i & 1]
                                                              : acc[h][m][j][i];
                        total[h][m][j][i] = fmaf(i < 2 ? s0 : s1, sum, total[h][m][j][i]);
                    }
            }
    }
}

// The table, by all threads of a CTA.  Up to 32 entries (or experts) are put in order by one warp, without a
// barrier: one token's layer 54 -> 50 us.
template <int kThreads>
__device__ __forceinline__ void make_table(const Args& p, const Table& t, Shared* s, uint8_t* stages, int warp, int lane) {
    const int entries = p.T * p.topk;
    const auto tiles_of = [&](int rows) { return (rows + p.tile_rows - 1) / p.tile_rows; };
    const auto named = [&](int i) {      // (may come before the wait)
        const int64_t e = __ldcg(reinterpret_cast<const long long*>(p.topk_idx) + i);
        const bool ok = e >= 0 && e < p.E;
        if (!ok && e != -1 && p.mode == kFewUp && blockIdx.x == 0) atomicOr(p.status, EP_ERR_INVALID_INDEX);
        return ok ? static_cast<int>(e) : -1;
    };
    if (p.mode != kProduct ? entries <= 32 : p.E <= 32) {
        if (warp == 0) {
            int count, first, id, place;      // of the lane's expert, in the table if place >= 0
            if (p.mode != kProduct) {
                id = lane < entries ? named(lane) : -1;
                if (lane < entries) t.expert[lane] = static_cast<int16_t>(id);
                const unsigned same = __match_any_sync(0xffffffffu, id), before = (1u << lane) - 1;
                const bool leads = id >= 0 && (same & before) == 0;
                const unsigned leaders = __ballot_sync(0xffffffffu, leads);
                place = leads ? __popc(leaders & before) : -1;
                count = __popc(same);
                first = warp_inclusive_scan(leads ? count : 0) - (leads ? count : 0);
                const int group = __shfl_sync(0xffffffffu, first, __ffs(same) - 1);
                if (id >= 0) t.list[group + __popc(same & before)] = static_cast<int16_t>(lane);
                if (lane == 0) s->listed = __popc(leaders);
            } else {
                id = place = lane < p.E ? lane : -1;
                int64_t at = 0;
                count = lane < p.E ? expert_rows<true>(p.expert_offset, p.counts, lane, p.rows, &at, p.status) : 0;
                first = static_cast<int>(at);
                if (warp_sum64(count) > p.rows) {      // they overlap
                    if (lane == 0) atomicOr(p.status, EP_ERR_CAPACITY);
                    count = 0;
                }
                if (lane == 0) s->listed = p.E;
            }
            const int ends = warp_inclusive_scan(place >= 0 ? tiles_of(count) : 0);
            if (place >= 0) {
                t.first[place] = first;
                t.count[place] = count;
                t.tile_end[place] = ends;
                s->id[place] = static_cast<int16_t>(id);
            }
        }
        __syncthreads();
        return;
    }
    if (threadIdx.x == 0) s->listed = p.E;
    if (p.E <= 32 && threadIdx.x < 32) s->id[threadIdx.x] = static_cast<int16_t>(threadIdx.x);
    if (p.mode == kProduct) {
        expert_blocks<kThreads>(p.expert_offset, p.counts, p.E, p.rows, t.first, t.count, s->warp_rows, p.status);
    } else {
        for (int i = threadIdx.x; i < entries; i += kThreads) t.expert[i] = static_cast<int16_t>(named(i));
        for (int e = threadIdx.x; e < p.E; e += kThreads) t.count[e] = 0;
        // Few entries: one warp puts them in place, 32 at a time.  More: every warp its share, after counting how many
        // of each expert's lie in the shares before it (counted where the stages will be).
        const bool shared = entries > 256;
        const int share = (entries + kThreads - 1) / kThreads * 32;
        const int begin = shared ? min(entries, warp * share) : 0;
        const int end = shared ? min(entries, begin + share) : warp == 0 ? entries : 0;
        uint16_t* const at = reinterpret_cast<uint16_t*>(stages);      // [warps][E]
        if (shared)
            for (int i = threadIdx.x; i < kThreads / 32 * p.E; i += kThreads) at[i] = 0;
        __syncthreads();
        for (int i = threadIdx.x; i < entries; i += kThreads)
            if (t.expert[i] >= 0) atomicAdd(&t.count[t.expert[i]], 1);
        for (int i0 = begin; shared && i0 < end; i0 += 32) {
            const int e = i0 + lane < end ? t.expert[i0 + lane] : -1;
            const unsigned same = __match_any_sync(0xffffffffu, e);
            if (e >= 0 && (same >> lane) == 1u) at[warp * p.E + e] += static_cast<uint16_t>(__popc(same));
            __syncwarp();
        }
        __syncthreads();
        scan_experts<kThreads>(p.E, t.first, s->warp_sum, [&](int e) { return t.count[e]; });
        // first[e] is where e's entries end; filled from the last one down, in
        // the order of (token, slot), it becomes where they begin: every CTA
        // has to give a tile the same rows
        if (shared) {
            for (int e = threadIdx.x; e < p.E; e += kThreads) {
                int end_at = t.first[e];
                for (int w = kThreads / 32 - 1; w >= 0; --w) {
                    const int n = at[w * p.E + e];
                    at[w * p.E + e] = static_cast<uint16_t>(end_at);
                    end_at -= n;
                }
                t.first[e] = end_at;
            }
            __syncthreads();
        }
        for (int i0 = begin + (end - begin - 1) / 32 * 32; i0 >= begin && begin < end; i0 -= 32) {
            const int i = i0 + lane, e = i < end ? t.expert[i] : -1;
            const unsigned same = __match_any_sync(0xffffffffu, e);
            const int end_at = e < 0 ? 0 : shared ? at[warp * p.E + e] : t.first[e];
            if (e >= 0) t.list[end_at - __popc(same >> lane)] = static_cast<int16_t>(i);
            __syncwarp();
            if (e >= 0 && (same >> lane) == 1u) {
                if (shared)
                    at[warp * p.E + e] = static_cast<uint16_t>(end_at - __popc(same));
                else
                    t.first[e] = end_at - __popc(same);
            }
            __syncwarp();
        }
        if (shared) fence_proxy_async_smem();      // before the stages are loaded
        __syncthreads();
    }
    scan_experts<kThreads>(p.E, t.tile_end, s->warp_sum, [&](int e) { return tiles_of(t.count[e]); });
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
    t.s = s;
    const int warp = uniform_warp(), lane = threadIdx.x & 31;
    const bool few = p.mode != kProduct, gated = p.act == EP_ACT_SWIGLU;
    const int half = pieces * 16 * kM, tile_features = gated ? half : 2 * half;
    const int feature_tiles = (p.N + tile_features - 1) / tile_features;
    const int steps = (p.K + kSlotK * p.slots - 1) / (kSlotK * p.slots);

    if (threadIdx.x == 0) {
        for (int i = 0; i < p.stages; ++i) {
            for (int k = 0; k < 2; ++k)
                mbar_init(&s->full[i][k], 1 + kCopyWarps * 32);   // the tensor maps' bytes, and the rows' copies
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
    make_table<kThreads>(p, t, s, stages, warp, lane);
    const int64_t tiles = s->listed > 0 ? static_cast<int64_t>(t.tile_end[s->listed - 1]) * feature_tiles : 0;
    if (p.mode == kFewDown) {
        if (warp >= kCopyWarps) pdl_wait();     // (the others do when the first weights have been asked for)
        pdl_launch_dependents();
    }

    if (warp < kCopyWarps) {
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
        // 16-byte pieces of a row in a stage; rows of a thread
        const int tid = threadIdx.x, chunks = kSlotK / 8 * p.slots, passes = max(1, chunks / (kCopyWarps * 32));
        const int row_step = max(1, kCopyWarps * 32 / chunks), row0 = passes > 1 ? 0 : tid / chunks, chunk0 = tid & (chunks - 1);
        int stage = 0, issued = 0, early = 0;
        uint32_t use = 0;
        bool ok = true;
        bool drop = kTestDropFirstLoad && blockIdx.x == 0;
        if (p.mode == kFewDown) {
            // the down product's first weights come while the up product ends
            if (warp == 0 && blockIdx.x < tiles) {
                const Tile r = tile_at(p, t, blockIdx.x, feature_tiles, tile_features, lane);
                early = min(p.stages, steps);
                for (int i = 0; i < early; ++i)
                    if (!drop || i > 0) load_weights(r, i, 0, i);
            }
            pdl_wait();
        }
        for (int64_t g = blockIdx.x; g < tiles && ok; g += gridDim.x) {
            const Tile r = tile_at(p, t, g, feature_tiles, tile_features, lane);
            constexpr int kMost = 8;       // rows of a thread: one share's 32 rows, four at a time
            const __nv_bfloat16* from[kMost];
#pragma unroll
            for (int i = 0; i < kMost; ++i) {
                const int row = row0 + i * row_step;
                from[i] = nullptr;
                if (row < r.rows) {
                    const int at = r.first + row, entry = few ? t.list[at] : at;
                    const int64_t source = p.mode == kFewUp ? entry / p.topk : entry;
                    if (EP_IN(source, p.mode == kFewUp ? p.T : few ? p.T * p.topk : p.rows)) from[i] = p.x + source * p.K;
                }
            }
            // FP4: rows come through registers, those of the next stage asked for as the last leave them (64 experts of 8
            // rows, 7168 -> 2 x 2048: 288 us, two stages ahead 289; asked for just before the stage's wait 298, turned
            // where asynchronous copies had left them 312).
            uint4 asked[kForm == EP_W4_FP ? kMost : 1];
            const auto ask = [&](int i, int step, int pass) {
                const int k = step * kSlotK * p.slots + (chunk0 + pass * (kCopyWarps * 32)) * 8;
                asked[i] = from[i] && k < p.K ? __ldcg(reinterpret_cast<const uint4*>(from[i] + k)) : make_uint4(0u, 0u, 0u, 0u);
            };
            const auto to_stage = [&](int step, int stage, uint32_t use) {
                const uint32_t x_at = smem_addr(stages) + stage * p.stage_bytes + p.x_offset;
                for (int pass = 0; pass < passes; ++pass) {
                    const int chunk = chunk0 + pass * (kCopyWarps * 32), slot = chunk / (kSlotK / 8);
                    const int next_pass = pass + 1 < passes ? pass + 1 : 0, next = next_pass > 0 ? step : step + 1;
#pragma unroll
                    for (int i = 0; i < kMost; ++i) {
                        if (i * row_step >= r.rows) break;
                        const int place = slot * p.tile_rows + row0 + i * row_step;
                        float unit;
                        const uint4 v = to_fp16(asked[i], &unit);
                        if (from[i]) {
                            store_shared4(x_at + place * kRowPitch + chunk % (kSlotK / 8) * 16, v);
                            if (chunk % (kSlotK / 8) == 0)
                                store_shared(x_at + p.slots * p.tile_rows * kRowPitch + place * 4, __float_as_uint(unit));
                        }
                        if (next < steps) ask(i, next, next_pass);
                    }
                }
                mbar_arrive(&s->full[stage][use & 1]);
            };
            if (kForm == EP_W4_FP)
#pragma unroll
                for (int i = 0; i < kMost; ++i) ask(i, 0, 0);
            for (int step = 0; step < steps; ++step, ++issued) {
                // (A stage whose weights were asked for early is there to be filled.  Its wait, for the use before,
                // would be for the one after once it had been consumed.)
                if (issued >= early) {
                    ok = wait_quietly(&s->empty[stage], (use & 1) ^ 1);
                    if (!ok) break;
                    if (warp == 0 && !drop) load_weights(r, stage, use, step);
                }
                if (kForm == EP_W4_FP) {
                    if (!drop) to_stage(step, stage, use);
                } else if (!drop) {
                    for (int pass = 0; pass < passes; ++pass) {
                        const int chunk = chunk0 + pass * (kCopyWarps * 32), k = step * kSlotK * p.slots + chunk * 8;
                        const bool inside = k < p.K;
                        const uint32_t to = smem_addr(stages) + stage * p.stage_bytes + p.x_offset +
                                            (chunk / (kSlotK / 8) * p.tile_rows + row0) * kRowPitch +
                                            chunk % (kSlotK / 8) * 16;
#pragma unroll
                        for (int i = 0; i < kMost; ++i) {
                            if (i * row_step >= r.rows) break;
                            if (from[i]) copy16_async(to + i * row_step * kRowPitch, from[i] + (inside ? k : 0), inside);
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
        // no copy may still be in flight when the CTA ends (after a wait that ran out, each stage's all the same)
        copies_commit();
        copies_wait<0>();
        if (warp == 0) {
            issued = max(issued, early);
            for (int i = max(0, issued - p.stages); i < issued; ++i)
                wait_quietly(&s->full[i % p.stages][i / p.stages & 1], (i / p.stages >> 1) & 1);
        }
    } else if (warp >= kFirstTeamWarp) {
        const int w = (warp - kFirstTeamWarp) % kTeam, team = (warp - kFirstTeamWarp) / kTeam;
        const int piece = w % pieces, slot = w / pieces, g8 = lane >> 2, t4 = lane & 3;
        Place<V> at;
        at.codes = (slot * 2 * half + piece * 16 * kM + g8) * (kSlotK / 2) + ((g8 >> 1) & 3) * 16 + t4 * 4;
        at.half = half * (kSlotK / 2);
#pragma unroll
        for (int j = 0; j < V::kTiles8; ++j)
            at.x[j] = p.x_offset + (slot * p.tile_rows + min(j * 8 + g8, p.tile_rows - 1)) * kRowPitch + t4 * 16;
#pragma unroll
        for (int j = 0; j < V::kTiles8; ++j)      // (room for 32 units a share)
            at.unit[j] = p.x_offset + p.slots * p.tile_rows * kRowPitch + (slot * p.tile_rows + j * 8 + t4 * 2) * 4;
        const int item = p.sf_fp32 ? 4 : 2, groups = kSlotK / 32 / kBlocks;
        at.sf = (slot * groups * 2 * half + piece * 16 * kM + g8) * item;
        at.sf_half = half * item;
        float* const mine = sums + ((team * p.slots + slot) * pieces + piece) * V::kSums * 32;
        int stage = team % p.stages, before = 0;      // steps of the tiles before, modulo the teams
        uint32_t use = team / p.stages, turn = 0;
        bool ok = true;
        for (int64_t g = blockIdx.x; g < tiles; g += gridDim.x, turn ^= 1) {
            const int tiles8 = (tile_at(p, t, g, feature_tiles, tile_features, lane).rows + 7) / 8;
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
                    else if (V::kTiles8 == 2 || tiles8 == 2)
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
        constexpr float kSumScale = kForm != EP_W4_FP ? 64.0f : 1.0f;
        // Several rows without a gate: four at a time, whose sums and residuals are asked for together, places and
        // weights known before (row by row, 64 experts of 4, 8, 16 rows, 2048 -> 7168: 115, 152, 234 us, so 107, 117,
        // 181; with a gate, where a tile has twice the products for half the outputs, row by row is as fast or faster:
        // 256 experts of a decode step, 7168 -> 2 x 2048, 598 us, four at a time 616).
        const auto finish_rows = [&](const Tile& r, int64_t mine, float weight) {
            const int chunks = half / 32 * 2, share_step = pieces * V::kSums * 32;
            for (int chunk = warp - kFirstFinishWarp; chunk < chunks; chunk += kFinishWarps) {
                const int h = chunk & 1, f = (chunk >> 1) * 32 + lane, feature = r.f0 + h * half + f;
                const bool inside = feature < p.N;
                const float bias = p.bias && inside && EP_IN(r.e, p.E) ? p.bias[static_cast<int64_t>(r.e) * p.Nw + feature] : 0.0f;
                const float* const base = sums + (f / (16 * kM) * V::kSums + (h * kM + f / 16 % kM) * 4 + (f >> 3 & 1) * 2) * 32 +
                                          (f & 7) * 4;
                const int turn = f >> 3 & 3;
                constexpr int kAtOnce = 4;
                for (int row0 = 0; row0 < r.rows; row0 += kAtOnce) {
                    float z[kAtOnce] = {}, add[kAtOnce] = {};
                    int64_t out[kAtOnce];
#pragma unroll
                    for (int i = 0; i < kAtOnce; ++i) {
                        const int64_t to = __shfl_sync(0xffffffffu, mine, row0 + i);
                        out[i] = to >= 0 && inside ? to * p.N + feature : -1;
                        if (p.residual && out[i] >= 0) add[i] = __bfloat162float(p.residual[out[i]]);
                    }
                    const float* from = base + (row0 >> 3) * (2 * kM * 4 * 32);
                    for (int share = 0; share < shares; ++share, from += share_step)
#pragma unroll
                        for (int i = 0; i < kAtOnce; ++i) z[i] += from[(i & 1) * 32 + (((row0 + i) >> 1 & 3) ^ turn)];
#pragma unroll
                    for (int i = 0; i < kAtOnce; ++i) {
                        const float a = activate(fmaf(z[i], kSumScale, bias), p.act);
                        const float by = __shfl_sync(0xffffffffu, weight, row0 + i);
                        if (out[i] < 0) continue;
                        if (p.mode == kFewDown)
                            p.part[out[i]] = a;
                        else
                            p.y[out[i]] = __float2bfloat16_rn(p.residual ? a * by + add[i] : a * by);
                    }
                }
            }
        };
        const auto finish_row_by_row = [&](auto gate, const Tile& r) {
            constexpr bool kGate = decltype(gate)::value;
            const int chunks = half / 32 * (kGate ? 1 : 2), share_step = pieces * V::kSums * 32;
            for (int chunk = warp - kFirstFinishWarp; chunk < chunks; chunk += kFinishWarps) {
                const int h = kGate ? 0 : chunk & 1, f = (kGate ? chunk : chunk >> 1) * 32 + lane;     // in the half
                const int feature = r.f0 + h * half + f;
                if (feature >= p.N) continue;
                const float* const bias = p.bias && EP_IN(r.e, p.E) ? p.bias + static_cast<int64_t>(r.e) * p.Nw + feature : nullptr;
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
                    z = fmaf(z, kSumScale, b0);
                    float a = kGate ? silu(z) * fmaf(other, kSumScale, b1) : activate(z, p.act);
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
            const Tile r = tile_at(p, t, g, feature_tiles, tile_features, lane);
            // a lane's row: where it goes, and its weight
            int64_t mine = -1;
            if (lane < r.rows) {
                mine = few ? t.list[r.first + lane] : r.first + lane;
                if (!EP_IN(mine, few ? static_cast<int64_t>(p.T) * p.topk : p.rows)) mine = -1;
            }
            const float weight = p.row_weight && mine >= 0 ? p.row_weight[mine] : 1.0f;
            ok = wait_quietly(&s->sums_full, turn);
            if (!ok) break;
            if (gated)
                finish_row_by_row(std::true_type(), r);
            else if (r.rows == 1)
                finish_row_by_row(std::false_type(), r);
            else
                finish_rows(r, mine, weight);
            __syncwarp();
            if (lane == 0) mbar_arrive(&s->sums_empty);
        }
        if (!ok) atomicOr(p.status, EP_ERR_TIMEOUT);
    }
}

// The kernel for a group and a variant.
template <int kForm>
cudaError_t launch_form(const Args& a, int group, Which which, dim3 grid, size_t smem, cudaStream_t stream) {
    const auto go = [&](auto blocks, auto variant) {
        using V = decltype(variant);
        const auto kernel = experts_w4_kernel<kForm, decltype(blocks)::value, V>;
        static std::atomic<bool> ready[kMaxDevices];
        const cudaError_t e = allow_all_smem(reinterpret_cast<const void*>(kernel), ready);
        return e != cudaSuccess ? e : launch_experts(kernel, grid, dim3(V::kThreads), smem, stream, 1, a);
    };
    const auto of = [&](auto blocks) {
        return which == kFew ? go(blocks, Few()) : which == kMid ? go(blocks, Mid()) : go(blocks, Wide());
    };
    if (group == 128) return of(std::integral_constant<int, 4>());
    if (group == 64) return of(std::integral_constant<int, 2>());
    return of(std::integral_constant<int, 1>());
}

}  // namespace

}  // namespace w4

}  // namespace epg
