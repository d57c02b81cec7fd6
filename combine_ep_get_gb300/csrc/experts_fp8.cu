// The experts' product on FP8 rows and weights, tcgen05 (f8f6f4 kind).
//
//   z[d, n] = sum over 128-channel blocks b of
//             x_sf[d, b] * w_sf[n / 128, b] * sum over k in b of x[d, k] * W[n, k]
//
// The scales change every 128 terms of the sum, so a block's product goes to
// tensor memory by itself (four MMAs, the first overwriting) and eight warps
// scale it and add it to fp32 sums in their registers, while the MMAs of the
// next blocks fill three more accumulators.  128 features x 128 rows a tile:
// 64 sums a thread.  The row scales of a block come through shared memory,
// copied there asynchronously by two warps well ahead of their use.
#include "experts_mma.cuh"

namespace epg {
namespace {

constexpr int kFp8Threads = 384;
constexpr int kRows = 128;             // rows of a tile
constexpr int kBlock = 128;            // terms that share their scales: one stage
constexpr int kFp8Stage = (kM + kRows) * kBlock;
constexpr int kFp8Stages = 6;
constexpr int kAccs = 4;
constexpr int kScaleStages = 8;
static_assert((kRows + 4) % 4 == 0, "rows of scales are read 16 bytes at a time");
constexpr int kScaleWords = kRows + 4; // row scales, then the gate's and the up rows' weight scales

struct Fp8Args {
    MmaArgs m;
    const float* x_sf;           // element (d, b) at d * sf_row + b * sf_block
    int64_t sf_row, sf_block;
    const float* w_sf;           // [E][Nw / 128][K / 128]
};

struct Fp8Shared {
    uint64_t full[kFp8Stages], empty[kFp8Stages], acc_full[kAccs], acc_empty[kAccs];
    uint64_t sc_full[kScaleStages], sc_empty[kScaleStages], drain;
    alignas(16) float scales[kScaleStages][kScaleWords];
    uint32_t tmem;
    int warp_sum[kFp8Threads / 32];
};

// 4 bytes from global to shared memory, asynchronously; zeros if not wanted.
__device__ __forceinline__ void copy_word_async(float* dst, const float* src, bool wanted) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(wanted ? 4 : 0)
                 : "memory");
}
// One arrival on `bar` once this thread's copies so far have landed.
__device__ __forceinline__ void copies_arrive(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 z, x, y, z;\n\tmov.b64 {%0, %1}, z;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
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
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
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
            mbar_init(&s->acc_empty[i], 8);
        }
        for (int i = 0; i < kScaleStages; ++i) {
            mbar_init(&s->sc_full[i], 64);
            mbar_init(&s->sc_empty[i], 8);
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
        if (lane == 0) {
            int it = 0;
            bool ok = true;
            for (int g = blockIdx.x; g < tiles && ok; g += gridDim.x) {
                const Tile r = tile_at<kRows>(g, t, p.E, feature_tiles, tile_features);
                const int first = t.first[r.e] + r.row0, boxes = (r.rows + 63) / 64;
                for (int kb = 0; kb < k_blocks; ++kb, ++it) {
                    const int st = it % kFp8Stages;
                    ok = mbar_wait_bounded(&s->empty[st], ((it / kFp8Stages) & 1) ^ 1);
                    if (!ok) break;
                    uint8_t* sa = stages + st * kFp8Stage;
                    const uint32_t bar = smem_addr(&s->full[st]);
                    mbar_arrive_expect_tx(&s->full[st], (kM + boxes * 64) * kBlock);
                    if (gated)
                        tma_load_5d<1>(sa, &p.a, bar, kb * kBlock, 0, 0, r.f0 / 8, r.e);
                    else
                        tma_load_3d<1>(sa, &p.a, bar, kb * kBlock, r.f0, r.e);
                    for (int i = 0; i < boxes; ++i)
                        tma_load_2d<1>(sa + (kM + i * 64) * kBlock, &p.b, bar, kb * kBlock, first + i * 64);
                }
            }
            if (!ok) atomicOr(p.status, EP_ERR_TIMEOUT);
            // no copy may still be in flight when the CTA ends
            for (int i = max(0, it - kFp8Stages); i < it; ++i)
                if (!mbar_wait_bounded(&s->full[i % kFp8Stages], (i / kFp8Stages) & 1)) break;
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0) {
            int it = 0;
            bool ok = true;
            for (int g = blockIdx.x; g < tiles && ok; g += gridDim.x) {
                const Tile r = tile_at<kRows>(g, t, p.E, feature_tiles, tile_features);
                const uint32_t idesc = instr_desc(true, false, false, kM, r.width);
                for (int kb = 0; kb < k_blocks; ++kb, ++it) {
                    const int st = it % kFp8Stages, acc = it % kAccs;
                    ok = mbar_wait_bounded(&s->acc_empty[acc], ((it / kAccs) & 1) ^ 1) &&
                         mbar_wait_bounded(&s->full[st], (it / kFp8Stages) & 1);
                    if (!ok) break;
                    tcgen05_after_sync();
                    const uint32_t sa = smem_addr(stages + st * kFp8Stage), sb = sa + kM * kBlock;
#pragma unroll
                    for (int k = 0; k < kBlock / 32; ++k)
                        mma<1, true>(tmem + acc * kRows, operand_desc(sa + k * 32, 16), operand_desc(sb + k * 32, 16),
                                     idesc, k > 0);
                    mma_commit<1>(&s->empty[st]);
                    mma_commit<1>(&s->acc_full[acc]);
                }
            }
            if (!ok) {
                atomicOr(p.status, EP_ERR_TIMEOUT);
                mma_commit<1>(&s->drain);
                mbar_wait_bounded(&s->drain, 0);
            }
        }
        __syncwarp();
    } else if (warp < 4) {
        const int tid = threadIdx.x - 64;
        int it = 0;
        bool ok = true;
        for (int g = blockIdx.x; g < tiles && ok; g += gridDim.x) {
            const Tile r = tile_at<kRows>(g, t, p.E, feature_tiles, tile_features);
            const int64_t first = t.first[r.e] + r.row0;
            const int wf = (tid == 1 && gated ? p.gate_half : 0) + r.f0, Fw = gated ? 2 * p.F : p.F;
            const float* const w_sf = args.w_sf + (static_cast<int64_t>(r.e) * (Fw / 128) + wf / 128) * k_blocks;
            for (int kb = 0; kb < k_blocks; ++kb, ++it) {
                const int sc = it % kScaleStages;
                ok = mbar_wait_bounded(&s->sc_empty[sc], ((it / kScaleStages) & 1) ^ 1);
                if (!ok) break;
                for (int i = tid; i < kRows; i += 64) {
                    const bool wanted = i < r.rows && EP_IN(first + i, p.rows);
                    copy_word_async(&s->scales[sc][i],
                                    args.x_sf + (wanted ? (first + i) * args.sf_row + kb * args.sf_block : 0), wanted);
                }
                if (tid < 2) copy_word_async(&s->scales[sc][kRows + tid], w_sf + kb, true);
                copies_arrive(&s->sc_full[sc]);
            }
        }
        if (!ok) atomicOr(p.status, EP_ERR_TIMEOUT);
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else {
        const int q = warp & 3, half = (warp - 4) / 4;
        int it = 0;
        bool ok = true;
        for (int g = blockIdx.x; g < tiles && ok; g += gridDim.x) {
            const Tile r = tile_at<kRows>(g, t, p.E, feature_tiles, tile_features);
            const int first = t.first[r.e] + r.row0;
            const int up = gated && (lane & 8) ? 1 : 0;
            float sum[64];
#pragma unroll
            for (int i = 0; i < 64; ++i) sum[i] = 0.0f;
            for (int kb = 0; kb < k_blocks; ++kb, ++it) {
                const int sc = it % kScaleStages, acc = it % kAccs;
                ok = __all_sync(0xffffffffu, mbar_wait_bounded(&s->sc_full[sc], (it / kScaleStages) & 1) &&
                                                     mbar_wait_bounded(&s->acc_full[acc], (it / kAccs) & 1)
                                                 ? 1
                                                 : 0) != 0;
                if (!ok) break;
                tcgen05_after_sync();
                const float ws = s->scales[sc][kRows + up];
                const float2 w2 = make_float2(ws, ws), zero = make_float2(0.0f, 0.0f);
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float v[32];
                    tmem_load32(tmem + acc * kRows + half * 64 + c * 32 + (static_cast<uint32_t>(q * 32) << 16), v);
                    if (c == 1) {
                        tcgen05_before_sync();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&s->acc_empty[acc]);
                    }
#pragma unroll
                    for (int i = 0; i < 32; i += 4) {
                        const float4 x = *reinterpret_cast<const float4*>(&s->scales[sc][half * 64 + c * 32 + i]);
                        const float2 s0 = fma2(make_float2(x.x, x.y), w2, zero);
                        const float2 s1 = fma2(make_float2(x.z, x.w), w2, zero);
                        float* const o = sum + c * 32 + i;
                        const float2 a = fma2(make_float2(v[i], v[i + 1]), s0, make_float2(o[0], o[1]));
                        const float2 b = fma2(make_float2(v[i + 2], v[i + 3]), s1, make_float2(o[2], o[3]));
                        o[0] = a.x;
                        o[1] = a.y;
                        o[2] = b.x;
                        o[3] = b.y;
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&s->sc_empty[sc]);
            }
            if (!ok) break;
            const float bias = bias_of(p, r, q, lane);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float v[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = sum[c * 32 + i];
                if (half * 64 + c * 32 < r.rows)
                    finish_columns<kProduct>(p, t, r, first, q, lane, bias, half * 64 + c * 32, v);
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
    return launch_pdl(experts_fp8_kernel, dim3(grid), dim3(kFp8Threads), smem, stream, a);
}

}  // namespace epg
