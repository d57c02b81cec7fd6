// The experts' product on FP8 rows and weights, tcgen05 (f8f6f4 kind).
//
//   z[d, n] = sum over 128-channel blocks b of
//             x_sf[d, b] * w_sf[n / 128, b] * sum over k in b of x[d, k] * W[n, k]
//
// The scales change every 128 terms of the sum, so a block's product goes to
// tensor memory by itself (four MMAs, the first overwriting) and sixteen warps
// scale it and add it to fp32 sums in their registers, 32 a thread, while the
// MMAs of the next blocks fill three more accumulators.  128 features x 128
// rows a tile.  Two warps multiply row scales by weight scales ahead of their
// use, so that a product's element costs one multiply-add (two elements an
// instruction).
#include "experts_mma.cuh"

namespace epg {
namespace {

constexpr int kFp8Threads = 640;
constexpr int kSumWarps = 16;
constexpr int kRows = 128;             // rows of a tile
constexpr int kBlock = 128;            // terms that share their scales: one stage
constexpr int kFp8Stage = (kM + kRows) * kBlock;
constexpr int kFp8Stages = 6;
constexpr int kAccs = 4;
constexpr int kScaleStages = 8;
constexpr int kScaleBatch = 8;         // blocks whose scales are asked for at once
// A block's scales of the tile's rows, times the gate's (or only) weight scale
// and times the up rows'; the second four words on, so that the two are read
// from different banks.
constexpr int kScaleWords = kRows + 4;

struct Fp8Args {
    MmaArgs m;
    const float* x_sf;           // element (d, b) at d * sf_row + b * sf_block
    int64_t sf_row, sf_block;
    const float* w_sf;           // [E][Nw / 128][K / 128]
};

struct Fp8Shared {
    uint64_t full[kFp8Stages], empty[kFp8Stages], acc_full[kAccs], acc_empty[kAccs];
    uint64_t sc_full[kScaleStages], sc_empty[kScaleStages], drain;
    alignas(16) float scales[kScaleStages][2][kScaleWords];
    uint32_t tmem;
    int warp_sum[kFp8Threads / 32];
};

// Two fp32 multiply-adds in one instruction, each rounded as the scalar one;
// pairs stay in 64-bit registers, or their packing would cost what it saves.
__device__ __forceinline__ void fma2(uint64_t& sum, uint64_t a, uint64_t b) {
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(sum) : "l"(a), "l"(b));
}
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
    return v;
}

// sum += v * scale, 32 columns; the scales lie in shared memory.
__device__ __forceinline__ void add_scaled(uint64_t (&sum)[16], const float (&v)[32], const float* scale) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(scale + 4 * i);
        fma2(sum[2 * i], pair(v[4 * i], v[4 * i + 1]), x.x);
        fma2(sum[2 * i + 1], pair(v[4 * i + 2], v[4 * i + 3]), x.y);
    }
}

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
    const bool gated = p.gate_half != 0;
    const int tile_features = gated ? kM / 2 : kM;
    const int feature_tiles = (p.F + tile_features - 1) / tile_features;
    const int k_blocks = p.depth / kBlock;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kFp8Stages; ++i) {
            mbar_init(&s->full[i], 1);
            mbar_init(&s->empty[i], 1);
        }
        for (int i = 0; i < kAccs; ++i) {
            mbar_init(&s->acc_full[i], 1);
            mbar_init(&s->acc_empty[i], kSumWarps);
        }
        for (int i = 0; i < kScaleStages; ++i) {
            mbar_init(&s->sc_full[i], 2);
            mbar_init(&s->sc_empty[i], kSumWarps);
        }
        mbar_init(&s->drain, 1);
        fence_mbar_init();
        prefetch_map(&p.a);
        prefetch_map(&p.b);
    }
    if (warp == 2) tmem_alloc<1>(&s->tmem, kAccs * kRows);
    pdl_wait();
    pdl_launch_dependents();
    for (int e = threadIdx.x; e < p.E; e += kFp8Threads) {
        int64_t first;
        t.count[e] = expert_rows(p.expert_offset, p.counts, e, p.rows, &first, p.status);
        t.first[e] = static_cast<int>(first);
    }
    __syncthreads();
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
            const Tile r = tile_at<kRows>(g, t, p.E, feature_tiles, tile_features);
            const int first = t.first[r.e] + r.row0, boxes = (r.rows + 63) / 64;
            for (int kb = 0; kb < k_blocks; ++kb, ++issued, ring.next()) {
                ok = warp_wait(&s->empty[ring.stage], ring.parity ^ 1);
                if (!ok) break;
                if (elect_one()) {
                    uint8_t* const sa = stages + ring.stage * kFp8Stage;
                    const uint32_t bar = smem_addr(&s->full[ring.stage]);
                    mbar_arrive_expect_tx(&s->full[ring.stage], (kM + boxes * 64) * kBlock);
                    if (gated)
                        tma_load_5d<1>(sa, &p.a, bar, kb * kBlock, 0, 0, r.f0 / 8, r.e);
                    else
                        tma_load_3d<1>(sa, &p.a, bar, kb * kBlock, r.f0, r.e);
                    for (int i = 0; i < boxes; ++i)
                        tma_load_2d<1>(sa + (kM + i * 64) * kBlock, &p.b, bar, kb * kBlock, first + i * 64);
                }
                __syncwarp();
            }
        }
        if (!ok) atomicOr(p.status, EP_ERR_TIMEOUT);
        // no copy may still be in flight when the CTA ends
        for (int i = max(0, issued - kFp8Stages); i < issued; ++i)
            if (!warp_wait(&s->full[i % kFp8Stages], (i / kFp8Stages) & 1)) break;
    } else if (warp == 1) {
        Ring<kFp8Stages> ring;
        Ring<kAccs> accs;
        const uint64_t desc = operand_desc(smem_addr(stages), 16);
        bool ok = true;
        for (int g = blockIdx.x; g < tiles && ok; g += gridDim.x) {
            const Tile r = tile_at<kRows>(g, t, p.E, feature_tiles, tile_features);
            const uint32_t idesc = instr_desc(true, false, false, kM, r.width);
            for (int kb = 0; kb < k_blocks; ++kb, ring.next(), accs.next()) {
                ok = warp_wait(&s->acc_empty[accs.stage], accs.parity ^ 1) &&
                     warp_wait(&s->full[ring.stage], ring.parity);
                if (!ok) break;
                tcgen05_after_sync();
                if (elect_one()) {
                    const uint64_t da = desc_at(desc, ring.stage * kFp8Stage), db = desc_at(da, kM * kBlock);
#pragma unroll
                    for (int k = 0; k < kBlock / 32; ++k)
                        mma<1, true>(tmem + accs.stage * kRows, desc_at(da, k * 32), desc_at(db, k * 32), idesc, k > 0);
                    mma_commit<1>(&s->empty[ring.stage]);
                    mma_commit<1>(&s->acc_full[accs.stage]);
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
    } else if (warp < 4) {
        const int tid = threadIdx.x - 64;
        int it = 0;
        bool ok = true;
        for (int g = blockIdx.x; g < tiles && ok; g += gridDim.x) {
            const Tile r = tile_at<kRows>(g, t, p.E, feature_tiles, tile_features);
            const int64_t first = t.first[r.e] + r.row0;
            const int Fw = gated ? 2 * p.F : p.F;
            const float* const w_gate = args.w_sf + (static_cast<int64_t>(r.e) * (Fw / 128) + r.f0 / 128) * k_blocks;
            const float* const w_up = w_gate + static_cast<int64_t>(p.gate_half / 128) * k_blocks;
            const bool mine[2] = {tid < r.rows && EP_IN(first + tid, p.rows),
                                  tid + 64 < r.rows && EP_IN(first + tid + 64, p.rows)};
            const float* const x_sf = args.x_sf + (first + tid) * args.sf_row;
            for (int kb0 = 0; kb0 < k_blocks && ok; kb0 += kScaleBatch) {
                float x[2][kScaleBatch], wg[kScaleBatch], wu[kScaleBatch];
#pragma unroll
                for (int i = 0; i < kScaleBatch; ++i) {
                    const int kb = kb0 + i;
                    const bool in = kb < k_blocks;
                    x[0][i] = in && mine[0] ? x_sf[kb * args.sf_block] : 0.0f;
                    x[1][i] = in && mine[1] ? x_sf[64 * args.sf_row + kb * args.sf_block] : 0.0f;
                    wg[i] = in ? w_gate[kb] : 0.0f;
                    wu[i] = in ? w_up[kb] : 0.0f;
                }
#pragma unroll
                for (int i = 0; i < kScaleBatch; ++i) {
                    if (kb0 + i >= k_blocks || !ok) break;
                    const int sc = it % kScaleStages;
                    ok = __all_sync(0xffffffffu,
                                    mbar_wait_bounded(&s->sc_empty[sc], ((it / kScaleStages) & 1) ^ 1) ? 1 : 0) != 0;
                    if (!ok) break;
                    s->scales[sc][0][tid] = x[0][i] * wg[i];
                    s->scales[sc][0][tid + 64] = x[1][i] * wg[i];
                    if (gated) {
                        s->scales[sc][1][tid] = x[0][i] * wu[i];
                        s->scales[sc][1][tid + 64] = x[1][i] * wu[i];
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&s->sc_full[sc]);
                    ++it;
                }
            }
        }
        if (!ok) atomicOr(p.status, EP_ERR_TIMEOUT);
    } else {
        const int q = warp & 3, c0 = (warp - 4) / 4 * 32;
        const uint32_t column = tmem + static_cast<uint32_t>(c0) + (static_cast<uint32_t>(q * 32) << 16);
        const int up = gated && (lane & 8) ? 1 : 0;
        Ring<kAccs> accs;
        Ring<kScaleStages> scs;
        bool ok = true;
        for (int g = blockIdx.x; g < tiles && ok; g += gridDim.x) {
            const Tile r = tile_at<kRows>(g, t, p.E, feature_tiles, tile_features);
            uint64_t sum[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) sum[i] = 0;
            for (int kb = 0; kb < k_blocks; ++kb, accs.next(), scs.next()) {
                ok = warp_wait(&s->sc_full[scs.stage], scs.parity) && warp_wait(&s->acc_full[accs.stage], accs.parity);
                if (!ok) break;
                tcgen05_after_sync();
                float v[32];
                tmem_load32(column + accs.stage * kRows, v);
                tcgen05_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s->acc_empty[accs.stage]);
                add_scaled(sum, v, s->scales[scs.stage][up] + c0);
                __syncwarp();
                if (lane == 0) mbar_arrive(&s->sc_empty[scs.stage]);
            }
            if (!ok) break;
            if (c0 < r.rows) {
                float v[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(static_cast<uint32_t>(sum[i / 2] >> (i % 2 * 32)));
                finish_columns<kProduct>(p, t, r, t.first[r.e] + r.row0, q, lane, bias_of(p, r, q, lane), c0, v);
            }
        }
        if (!ok) atomicOr(p.status, EP_ERR_TIMEOUT);
    }
    __syncthreads();
    if (warp == 2) tmem_free<1>(tmem, kAccs * kRows);
}

}  // namespace

cudaError_t launch_expert_gemm_fp8(const ExpertGemmParams& p, cudaStream_t stream) {
    const bool gated = p.act == EP_ACT_SWIGLU;
    Fp8Args a{product_args(p), p.x_sf, p.sf_row, p.sf_block, p.w_sf};
    if (!(gated ? gated_map(&a.m.a, p.w, p.E, p.N, p.K, true) : weight_map(&a.m.a, p.w, p.E, p.Nw, p.K, kM, true)) ||
        !row_map(&a.m.b, p.x, p.rows, p.K, 64, true))
        return cudaErrorInvalidValue;
    const size_t smem = 1024 + kFp8Stages * kFp8Stage + sizeof(Fp8Shared) + static_cast<size_t>(p.E) * 12;
    const cudaError_t e = cudaFuncSetAttribute(experts_fp8_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    const int per = gated ? kM / 2 : kM;
    const int grid = std::max(1, std::min(device_info().num_sms, bound_tiles(p.rows / kRows + p.E, (p.N + per - 1) / per)));
    return launch_experts(experts_fp8_kernel, dim3(grid), dim3(kFp8Threads), smem, stream, 1, a);
}

}  // namespace epg
