// The experts' product on FP8 rows and weights, tcgen05 (f8f6f4 kind).
//
//   z[d, n] = sum over 128-channel blocks b of
//             x_sf[d, b] * w_sf[n / 128, b] * sum over k in b of x[d, k] * W[n, k]
//
// The scales change every 128 terms of the sum, so a block's product goes to
// tensor memory by itself (four MMAs, the first overwriting) and sixteen warps
// scale it and add it to fp32 sums in their registers, 64 a thread, while the
// MMAs of the next block fill the other accumulator.
//
// Here the rows are the M side, 128 a tile, and 256 of the weights' features
// the N side: a lane is a row, so a block's scale is one register a lane (with
// lanes as features, as in the bf16 product, every warp read the scales of its
// 32 rows from shared memory, whose bandwidth, already taken by the copies in
// and the operands out, bounded the kernel: 1.15 PFLOP/s).  SWIGLU: 8 gate and 8 up features
// in turns (one box of a five-dimensional map).
//
// What bounds it: with 512 rows an expert the summing warps (a block of 128
// terms takes them ~700 of the ~1000 cycles, the MMAs 512): 64 experts x 512
// rows, [4096, 7168] weights, 0.83 ms = 2.33 PFLOP/s (0.92-0.97 ms = 2.0-2.1 PFLOP/s
// after seconds of it, under the power limit).  All 19 warps are launched with 96
// registers: 64 sums spill a little (48-80 bytes), and a warp waits for each of
// its four reads of tensor memory before it multiplies.  Not tried: registers
// moved from the three issuing warps to these, the next read asked for ahead.
// Tried and slower: pairs of CTAs on 256 rows (278
// against 240 us on 16 experts x 512 rows; shared memory is freed, the summing
// warps have as much to do and the pair waits for both), two-wide fp32
// multiply-adds (their packing costs what they save).  With 32 rows an expert the weights bound it:
// 1.95 GB in 0.289-0.291 ms = 6.7 TB/s.
#include "experts_mma.cuh"

namespace epg {
namespace {

constexpr int kFp8Warps = 19;          // loads, MMAs, scales, 16 that sum
constexpr int kFp8Threads = kFp8Warps * 32;
constexpr int kSumWarps = 16;
constexpr int kRows = 128;             // rows of a tile
constexpr int kFeatures = 256;         // features of a tile
constexpr int kSumColumns = kFeatures / (kSumWarps / 4);
constexpr int kBlock = 128;            // terms that share their scales: one stage
constexpr int kRowBytes = kRows * kBlock;
constexpr int kFp8Stage = kRowBytes + kFeatures * kBlock;
constexpr int kFp8Stages = 4;
constexpr int kAccs = 2;
constexpr int kScaleBatch = 8;         // blocks whose scales are asked for at once

struct Fp8Args {
    MmaArgs m;                   // m.a: the weights' map, m.b: the rows'
    const float* x_sf;           // element (d, b) at d * sf_row + b * sf_block
    int64_t sf_row, sf_block;
    const float* w_sf;           // [E][Nw / 128][K / 128]
};

struct Fp8Shared {
    // acc_full: the MMAs of a block and its scales; acc_empty: both may be overwritten
    uint64_t full[kFp8Stages], empty[kFp8Stages], acc_full[kAccs], acc_empty[kAccs], drain;
    // a block's row scales times the two weight scales of the tile: of its
    // first and last 128 features, or of its gate and up features
    float scales[kAccs][2][kRows];
    int64_t warp_rows[kFp8Warps];
    uint32_t tmem;
    int warp_sum[kFp8Warps];
};

// 16 neighbouring bf16 features of a row, a whole 32-byte sector: in one access
// where y, z and the residual start on 32 bytes, else in two (a lane is a row, so
// an access touches 32 lines whatever its width.  Two: 40405 rows, 256 -> 3200,
// residual 288 against 239 us, 8192 rows, 512 -> 2 x 2048, z 60 against 41,
// 32768 rows, 7168 -> 2 x 2048 861 against 826).
struct Words8 {
    uint32_t w[8];
};
__device__ __forceinline__ void store16(__nv_bfloat16* at, const Words8& v, bool wide) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(at), "r"(v.w[0]), "r"(v.w[1]),
                     "r"(v.w[2]), "r"(v.w[3]), "r"(v.w[4]), "r"(v.w[5]), "r"(v.w[6]), "r"(v.w[7]) : "memory");
    } else {
        st_v4(at, make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]));
        st_v4(at + 8, make_uint4(v.w[4], v.w[5], v.w[6], v.w[7]));
    }
}
__device__ __forceinline__ Words8 load16(const __nv_bfloat16* at, bool wide) {
    Words8 v;
    if (wide) {
        asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];" : "=r"(v.w[0]), "=r"(v.w[1]),
                     "=r"(v.w[2]), "=r"(v.w[3]), "=r"(v.w[4]), "=r"(v.w[5]), "=r"(v.w[6]), "=r"(v.w[7]) : "l"(at)
                     : "memory");
    } else {
        const uint4 a = reinterpret_cast<const uint4*>(at)[0], b = reinterpret_cast<const uint4*>(at)[1];
        v = {{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
    }
    return v;
}
__device__ __forceinline__ Words8 pack16(const float* a, const float* b) {
    return {{pack2(a[0], a[1]), pack2(a[2], a[3]), pack2(a[4], a[5]), pack2(a[6], a[7]), pack2(b[0], b[1]),
             pack2(b[2], b[3]), pack2(b[4], b[5]), pack2(b[6], b[7])}};
}

// The epilogue of a row's 64 columns in a warp: 64 features from f, or, gated,
// 32 from f (8 gate columns, then 8 up ones, four times).  F is a multiple of
// 128, so all of them exist or none.  The bias is read before the first store
// and the residual 32 features at a time before theirs: it may be y itself, so
// a load after a store would wait for it.
template <bool kGated>
__device__ __forceinline__ void finish_row(const MmaArgs& p, int e, int64_t d, int f, float (&v)[kSumColumns]) {
    const int Fw = kGated ? 2 * p.F : p.F;
    const bool wide = ((reinterpret_cast<uintptr_t>(p.y) | reinterpret_cast<uintptr_t>(p.z) |
                        reinterpret_cast<uintptr_t>(p.residual)) & 31) == 0;
    const float w = p.row_weight ? p.row_weight[d] : 1.0f;
    // columns 8 i .. 8 i + 7 are these rows of W
    const auto wrow = [&](int i) { return kGated ? (i % 2) * p.gate_half + f + i / 2 * 8 : f + i * 8; };
    if (p.bias) {
        const float* const bias = p.bias + static_cast<int64_t>(e) * Fw;
#pragma unroll
        for (int i = 0; i < kSumColumns / 8; ++i) {
            const float4* const b = reinterpret_cast<const float4*>(bias + wrow(i));
            const float4 b0 = b[0], b1 = b[1];
            float* const u = v + 8 * i;
            u[0] += b0.x;
            u[1] += b0.y;
            u[2] += b0.z;
            u[3] += b0.w;
            u[4] += b1.x;
            u[5] += b1.y;
            u[6] += b1.z;
            u[7] += b1.w;
        }
    }
    if (p.z)
#pragma unroll
        for (int i = 0; i < kSumColumns / 16; ++i) {
            // columns 8 a .. 8 a + 7 and 8 b .. 8 b + 7 are neighbours in W
            const int a = kGated ? i / 2 * 4 + i % 2 : 2 * i, b = kGated ? a + 2 : a + 1;
            store16(p.z + d * Fw + wrow(a), pack16(v + 8 * a, v + 8 * b), wide);
        }
    constexpr int kOut = kGated ? kSumColumns / 2 : kSumColumns;
    if (kGated) {
#pragma unroll
        for (int i = 0; i < kOut; ++i) v[i] = silu(v[i / 8 * 16 + i % 8]) * v[i / 8 * 16 + 8 + i % 8];
    }
    __nv_bfloat16* const out = p.y + d * p.F + f;
#pragma unroll
    for (int c0 = 0; c0 < kOut; c0 += 32) {
        Words8 r[2];
        if (p.residual)
#pragma unroll
            for (int i = 0; i < 2; ++i) r[i] = load16(p.residual + d * p.F + f + c0 + 16 * i, wide);
        if (!kGated) activate_all(*reinterpret_cast<float(*)[32]>(v + c0), p.act);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float* const a = v + c0 + 16 * i;
#pragma unroll
            for (int j = 0; j < 16; ++j) a[j] *= w;
            if (p.residual)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float2 s = unpack2(r[i].w[j]);
                    a[2 * j] += s.x;
                    a[2 * j + 1] += s.y;
                }
            store16(out + c0 + 16 * i, pack16(a, a + 8), wide);
        }
    }
}

template <bool kGated>
__global__ void __launch_bounds__(kFp8Threads, 1) experts_fp8_kernel(const __grid_constant__ Fp8Args args) {
    const MmaArgs& p = args.m;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* stages = smem_raw + (1024 - (smem_addr(smem_raw) & 1023)) % 1024;
    Fp8Shared* s = reinterpret_cast<Fp8Shared*>(stages + kFp8Stages * kFp8Stage);
    Table t{};
    t.tile_end = reinterpret_cast<int*>(s + 1);
    t.first = t.tile_end + p.E;
    t.count = t.first + p.E;
    const int warp = uniform_warp(), lane = threadIdx.x & 31;
    constexpr int kTileFeatures = kGated ? kFeatures / 2 : kFeatures;
    const int feature_tiles = (p.F + kTileFeatures - 1) / kTileFeatures;
    const int k_blocks = p.depth / kBlock;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kFp8Stages; ++i) {
            mbar_init(&s->full[i], 1);
            mbar_init(&s->empty[i], 1);
        }
        for (int i = 0; i < kAccs; ++i) {
            mbar_init(&s->acc_full[i], 2);
            mbar_init(&s->acc_empty[i], kSumWarps);
        }
        mbar_init(&s->drain, 1);
        fence_mbar_init();
        prefetch_map(&p.a);
        prefetch_map(&p.b);
    }
    if (warp == 2) tmem_alloc<1>(&s->tmem, kAccs * kFeatures);
    pdl_wait();
    pdl_launch_dependents();
    expert_blocks<kFp8Threads>(p.expert_offset, p.counts, p.E, p.rows, t.first, t.count, s->warp_rows, p.status);
    scan_experts<kFp8Threads>(p.E, t.tile_end, s->warp_sum, [&](int e) { return (t.count[e] + kRows - 1) / kRows; });
    tcgen05_before_sync();
    __syncthreads();
    tcgen05_after_sync();
    const uint32_t tmem = s->tmem;
    const int tiles = t.tile_end[p.E - 1] * feature_tiles;

    if (warp == 0) {
        Ring<kFp8Stages> ring;
        int issued = 0;
        bool ok = true;
        for (int g = blockIdx.x; g < tiles && ok; g += gridDim.x) {
            const Tile r = tile_at<kRows>(g, t, p.E, feature_tiles, kTileFeatures);
            const int first = t.first[r.e] + r.row0, boxes = (r.rows + 63) / 64;
            // the second 128 features, where there are any
            const int halves = p.F - r.f0 > kTileFeatures / 2 ? 2 : 1;
            for (int kb = 0; kb < k_blocks; ++kb, ++issued, ring.next()) {
                ok = warp_wait(&s->empty[ring.stage], ring.parity ^ 1);
                if (!ok) break;
                if (elect_one()) {
                    uint8_t* const sa = stages + ring.stage * kFp8Stage;
                    const uint32_t bar = smem_addr(&s->full[ring.stage]);
                    mbar_arrive_expect_tx(&s->full[ring.stage], (boxes * 64 + halves * 128) * kBlock);
                    for (int i = 0; i < halves; ++i) {
                        uint8_t* const sb = sa + kRowBytes + i * 128 * kBlock;
                        if (kGated)
                            tma_load_5d<1>(sb, &p.a, bar, kb * kBlock, 0, 0, r.f0 / 8 + i * 8, r.e);
                        else
                            tma_load_3d<1>(sb, &p.a, bar, kb * kBlock, r.f0 + i * 128, r.e);
                    }
                    for (int i = 0; i < boxes && !(kTestDropFirstLoad && blockIdx.x == 0 && issued == 0); ++i)
                        tma_load_2d<1>(sa + i * 64 * kBlock, &p.b, bar, kb * kBlock, first + i * 64);
                }
                __syncwarp();
            }
        }
        if (!ok) atomicOr(p.status, EP_ERR_TIMEOUT);
        // no copy may still be in flight when the CTA ends
        for (int i = max(0, issued - kFp8Stages); i < issued; ++i)
            warp_wait(&s->full[i % kFp8Stages], (i / kFp8Stages) & 1);
    } else if (warp == 1) {
        Ring<kFp8Stages> ring;
        Ring<kAccs> accs;
        const uint64_t desc = operand_desc(smem_addr(stages), 16);
        bool ok = true;
        for (int g = blockIdx.x; g < tiles && ok; g += gridDim.x) {
            const Tile r = tile_at<kRows>(g, t, p.E, feature_tiles, kTileFeatures);
            const uint32_t idesc =
                instr_desc(true, false, false, kM, p.F - r.f0 > kTileFeatures / 2 ? kFeatures : kFeatures / 2);
            for (int kb = 0; kb < k_blocks; ++kb, ring.next(), accs.next()) {
                ok = warp_wait(&s->full[ring.stage], ring.parity) &&
                     warp_wait(&s->acc_empty[accs.stage], accs.parity ^ 1);
                if (!ok) break;
                tcgen05_after_sync();
                if (elect_one()) {
                    const uint64_t da = desc_at(desc, ring.stage * kFp8Stage), db = desc_at(da, kRowBytes);
#pragma unroll
                    for (int k = 0; k < kBlock / 32; ++k)
                        mma<1, true>(tmem + accs.stage * kFeatures, desc_at(da, k * 32), desc_at(db, k * 32), idesc,
                                     k > 0);
                    mma_commit<1>(&s->acc_full[accs.stage]);
                    mma_commit<1>(&s->empty[ring.stage]);
                }
                __syncwarp();
            }
        }
        if (!ok) {
            atomicOr(p.status, EP_ERR_TIMEOUT);
            if (elect_one()) mma_commit<1>(&s->drain);
            __syncwarp();
            warp_wait(&s->drain, 0);
        }
    } else if (warp == 2) {
        // lane l: the scales of rows l, l + 32, l + 64, l + 96
        Ring<kAccs> accs;
        bool ok = true;
        for (int g = blockIdx.x; g < tiles && ok; g += gridDim.x) {
            const Tile r = tile_at<kRows>(g, t, p.E, feature_tiles, kTileFeatures);
            const int64_t first = t.first[r.e] + r.row0;
            const int Fw = kGated ? 2 * p.F : p.F;
            const float* const w0 = args.w_sf + (static_cast<int64_t>(r.e) * (Fw / 128) + r.f0 / 128) * k_blocks;
            const int next = kGated ? p.gate_half / 128 : (p.F - r.f0 > 128 ? 1 : 0);
            const float* const w1 = w0 + static_cast<int64_t>(next) * k_blocks;
            const float* const x_sf = args.x_sf + (first + lane) * args.sf_row;
            for (int kb0 = 0; kb0 < k_blocks && ok; kb0 += kScaleBatch) {
                float x[4][kScaleBatch], a[kScaleBatch], b[kScaleBatch];
#pragma unroll
                for (int i = 0; i < kScaleBatch; ++i) {
                    const int kb = kb0 + i;
                    const bool in = kb < k_blocks;
                    a[i] = in ? w0[kb] : 0.0f;
                    b[i] = in ? w1[kb] : 0.0f;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        x[j][i] = in && lane + 32 * j < r.rows && EP_IN(first + lane + 32 * j, p.rows)
                                      ? x_sf[32 * j * args.sf_row + kb * args.sf_block]
                                      : 0.0f;
                }
#pragma unroll
                for (int i = 0; i < kScaleBatch; ++i) {
                    if (kb0 + i >= k_blocks || !ok) break;
                    ok = warp_wait(&s->acc_empty[accs.stage], accs.parity ^ 1);
                    if (!ok) break;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        s->scales[accs.stage][0][lane + 32 * j] = x[j][i] * a[i];
                        s->scales[accs.stage][1][lane + 32 * j] = x[j][i] * b[i];
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&s->acc_full[accs.stage]);
                    accs.next();
                }
            }
        }
        if (!ok) atomicOr(p.status, EP_ERR_TIMEOUT);
    } else {
        const int q = warp & 3, group = (warp - 3) / 4, row = q * 32 + lane;
        const uint32_t column = tmem + group * kSumColumns + (static_cast<uint32_t>(q * 32) << 16);
        Ring<kAccs> accs;
        bool ok = true;
        for (int g = blockIdx.x; g < tiles && ok; g += gridDim.x) {
            const Tile r = tile_at<kRows>(g, t, p.E, feature_tiles, kTileFeatures);
            float sum[kSumColumns];
#pragma unroll
            for (int i = 0; i < kSumColumns; ++i) sum[i] = 0.0f;
            for (int kb = 0; kb < k_blocks; ++kb, accs.next()) {
                ok = warp_wait(&s->acc_full[accs.stage], accs.parity);
                if (!ok) break;
                tcgen05_after_sync();
                const float f0 = s->scales[accs.stage][kGated ? 0 : group / 2][row];
                const float f1 = kGated ? s->scales[accs.stage][1][row] : f0;
#pragma unroll
                for (int c = 0; c < kSumColumns / 16; ++c) {
                    float v[16];
                    tmem_load16(column + accs.stage * kFeatures + c * 16, v);
                    if (c == kSumColumns / 16 - 1) {
                        tcgen05_before_sync();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&s->acc_empty[accs.stage]);
                    }
#pragma unroll
                    for (int i = 0; i < 16; ++i) sum[c * 16 + i] = fmaf(v[i], i < 8 ? f0 : f1, sum[c * 16 + i]);
                }
            }
            if (!ok) break;
            const int64_t d = static_cast<int64_t>(t.first[r.e]) + r.row0 + row;
            const int f = r.f0 + group * kSumColumns / (kGated ? 2 : 1);
            if (row < r.rows && f < p.F && EP_IN(d, p.rows)) finish_row<kGated>(p, r.e, d, f, sum);
            __syncwarp();
        }
        if (!ok) atomicOr(p.status, EP_ERR_TIMEOUT);
    }
    __syncthreads();
    if (warp == 2) tmem_free<1>(tmem, kAccs * kFeatures);
}

}  // namespace

cudaError_t launch_expert_gemm_fp8(const ExpertGemmParams& p, cudaStream_t stream) {
    const bool gated = p.act == EP_ACT_SWIGLU;
    Fp8Args a{product_args(p), p.x_sf, p.sf_row, p.sf_block, p.w_sf};
    if (!(gated ? gated_map(&a.m.a, p.w, p.E, p.N, p.K, true) : weight_map(&a.m.a, p.w, p.E, p.Nw, p.K, 128, true)) ||
        !row_map(&a.m.b, p.x, p.rows, p.K, 64, true))
        return cudaErrorInvalidValue;
    const size_t smem = 1024 + kFp8Stages * kFp8Stage + sizeof(Fp8Shared) + static_cast<size_t>(p.E) * 12;
    const auto kernel = gated ? experts_fp8_kernel<true> : experts_fp8_kernel<false>;
    static std::atomic<bool> ready[2][kMaxDevices];
    const cudaError_t e = allow_all_smem(reinterpret_cast<const void*>(kernel), ready[gated]);
    if (e != cudaSuccess) return e;
    const int per = gated ? kFeatures / 2 : kFeatures;
    const int grid = std::max(1, std::min(device_info().num_sms, bound_tiles(p.rows / kRows + p.E, (p.N + per - 1) / per)));
    return launch_experts(kernel, dim3(grid), dim3(kFp8Threads), smem, stream, 1, a);
}

}  // namespace epg
