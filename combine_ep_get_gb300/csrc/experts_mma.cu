// The experts' products on the tensor cores (tcgen05): rows of the expanded
// receive layout times each expert's weights, the input gradient, and the two
// products of the few-token layer.
//
// D[feature, row] = sum over k of W[feature, k] * rows[row, k].  The weights'
// features are the M side (128 a CTA, always full) and an expert's rows the N
// side, whose width an MMA may choose in steps of 16: a tile takes the rows
// an expert has instead of padding them to 128, and the weights, which are
// what a call with few rows per expert has to read, stream through the wide
// side.  Accumulators: fp32 in tensor memory, two of them, so that the
// epilogue of one tile runs under the MMAs of the next.
//
// One CTA per SM, or a pair of CTAs on a tile twice as wide in features, walks
// the tiles (expert, rows, features): warp 0 issues the tensor-map loads of
// 128-byte-swizzled operand tiles, 64 terms of the sum a stage; warp 1 issues
// the MMAs; warps 4-11 read the accumulators, lane = feature, and apply the
// epilogue.  SWIGLU: the 128 features of a CTA are, in turns, 8 gate rows and
// the 8 up rows that belong to them (one box of a five-dimensional map), so
// one exchange between lanes 8 apart brings each pair together.
//
// What bounds it.  Below about 290 rows an expert the weights' bytes do: 256
// experts x 128 rows, [4096, 7168] weights each, 15.6 GB in 2.27-2.32 ms = 6.7-6.9
// TB/s.  Above, the tensor cores: 4096 x 7168 x 7168 with bias, GELU and
// residual 225-229 us, tensor pipe 86% busy (input gradient, nothing in its
// epilogue: 92-93%); seconds of it run at the power limit, 1.63 PFLOP/s where a
// library product of the same sizes without epilogue reaches 1.73.  With one
// CTA a tile shared memory bounds it (a stage of 64 terms: 48 KB in, 48 KB
// out, 768 cycles at 128 B each; measured ~800): pairs halve each CTA's share
// of the rows (1.58 -> 1.87 PFLOP/s, 4096 x 7168 x 7168 alone).
//
// Few tokens: the same walk over the experts that some token names, with the
// tokens' rows gathered by index, by 16-byte copies of two warps (gathers of four
// rows by tensor map take up to 16 instructions a stage of 64 rows, ~90 cycles
// each: 143 tokens over 10 experts 72 us, by copies 60; 6 tokens 17.4 against
// 18.4).  Each CTA sorts topk_idx itself.  The up
// product leaves h, rounded to bf16 for the down product's tensor cores (one
// token, SWIGLU: the output is off by 2.3e-3 of its norm, 1.6e-3 of it its own
// rounding) and expert by expert, so that its loads are boxes of rows and not gathers (143
// tokens over 10 experts, 896 and 5208 features: 100 -> 72 us at that step), the down
// product fp32 rows for each (token, slot); whichever tile completes a
// token's last expert sums the token's rows, k ascending, so the order of the
// sum does not depend on timing.  Bound by the weights: one token, 8 experts
// of 88 MB, 705 MB in 114-118 us = 6.0-6.2 TB/s; 128 tokens, 22 GB in 3.11-3.2 ms =
// 6.9-7.1 TB/s.
#include "experts_mma.cuh"

namespace epg {

namespace {

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
    static const EncodeFn fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) !=
                cudaSuccess ||
            found != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            f = nullptr;
        }
        return reinterpret_cast<EncodeFn>(f);
    }();
    return fn;
}

}  // namespace

bool encode_map(CUtensorMap* map, bool fp8, int rank, const void* base, const uint64_t* dims, const uint64_t* strides,
                const uint32_t* box) {
    const EncodeFn fn = encode_fn();
    if (!fn) return false;
    cuuint64_t d[5], s[5];
    cuuint32_t b[5], one[5] = {1, 1, 1, 1, 1};
    for (int i = 0; i < rank; ++i) {
        d[i] = dims[i];
        b[i] = box[i];
        if (i + 1 < rank) s[i] = strides[i];
    }
    return fn(map, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank,
              const_cast<void*>(base), d, s, b, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

namespace {

template <int kMode, int NT, int kCtas, bool kSplit>
__global__ void __launch_bounds__(kThreads, 1) experts_mma_kernel(const __grid_constant__ MmaArgs p) {
    using S = Shape<NT, kCtas>;
    constexpr bool kFew = kMode == kFewUp || kMode == kFewDown;
    constexpr bool kGather = kMode == kFewUp;   // rows are tokens anywhere in x: warps 2 and 3 copy them
    constexpr int kBoxRows = kFew ? kFewBoxRows : S::kBoxRows;
    constexpr int kStep = 16 * kCtas;   // an MMA's rows come in steps of
    extern __shared__ uint8_t smem_raw[];
    uint8_t* stages = smem_raw + (1024 - (smem_addr(smem_raw) & 1023)) % 1024;
    Barriers* s = reinterpret_cast<Barriers*>(stages + S::kStages * S::kStageBytes);
    Table t;
    t.tile_end = reinterpret_cast<int*>(s + 1);
    t.first = t.tile_end + p.E;
    t.count = t.first + p.E;
    t.list = reinterpret_cast<int16_t*>(t.count + p.E);
    t.expert = t.list + p.T * p.K;
    t.named = reinterpret_cast<uint8_t*>(t.expert + p.T * p.K + EP_FEW_MAX_TOKENS);
    const int warp = uniform_warp(), lane = threadIdx.x & 31;
    const int rank = kCtas == 2 ? static_cast<int>(cluster_ctarank()) : 0;
    const int cta_features = p.gate_half ? kM / 2 : kM, tile_features = cta_features * kCtas;
    const int feature_tiles = (p.F + tile_features - 1) / tile_features;
    // a cluster's CTAs each take a piece of the sum (few tiles, long sums)
    const int split = kSplit ? p.split : 1, piece = kSplit ? static_cast<int>(cluster_ctarank()) : 0;
    const int k_blocks = (p.depth + kDepth - 1) / kDepth, k_each = (k_blocks + split - 1) / split;
    const int kb_begin = piece * k_each, kb_end = min(k_blocks, kb_begin + k_each);
    const int worker = blockIdx.x / (kCtas * split), workers = gridDim.x / (kCtas * split);

    if (threadIdx.x == 0) {
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(&s->full[i], kGather ? 1 + kGatherWarps : 1);
            mbar_init(&s->empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s->acc_full[i], 1);
            mbar_init(&s->acc_empty[i], kReadWarps * kCtas);
        }
        mbar_init(&s->drain, 1);
        s->gave_up = 0;
        fence_mbar_init();
        prefetch_map(&p.a);
        if (!kGather) prefetch_map(&p.b);
    }
    if (warp == 2) tmem_alloc<kCtas>(&s->tmem, S::kColumns);
    // The down product's kernel may start, and route, once every CTA of the
    // up product's has seen its own inputs complete ("Reads before the wait").
    if (kMode != kFewDown) {
        if (!p.wait_late) pdl_wait();
        pdl_launch_dependents();
    }

    if (kFew) {
        // entries by expert, in the order of (token, slot)
        for (int i = threadIdx.x; i < p.T * p.K; i += kThreads) {
            const int64_t e = __ldcg(reinterpret_cast<const long long*>(p.topk_idx) + i);   // (may come before the wait)
            const bool ok = e >= 0 && e < p.E;
            if (!ok && e != -1 && kMode == kFewUp && blockIdx.x == 0) atomicOr(p.status, EP_ERR_INVALID_INDEX);
            t.expert[i] = ok ? static_cast<int16_t>(e) : static_cast<int16_t>(-1);
        }
        const int entries = p.T * p.K;
        if (kMode == kFewUp && blockIdx.x == 0)
            for (int i = threadIdx.x; i < p.done_words; i += kThreads) p.done[i] = 0;
        // Few entries: one warp puts them in place, 32 at a time.  More: every
        // warp its share of them, after counting how many of each expert's
        // lie in the shares before it (counted where the stages will be).
        // 1544 entries: 53 -> 34 us a call; 8 entries by shares: 117 -> 120 us.
        const bool shared = entries > 256;
        const int share = (entries + kThreads - 1) / kThreads * 32;
        const int begin = shared ? min(entries, warp * share) : 0;
        const int end = shared ? min(entries, begin + share) : warp == 0 ? entries : 0;
        uint32_t* const at = reinterpret_cast<uint32_t*>(stages);   // [warps][E]
        if (shared)
            for (int i = threadIdx.x; i < kThreads / 32 * p.E; i += kThreads) at[i] = 0;
        for (int e = threadIdx.x; e < p.E; e += kThreads) t.count[e] = 0;
        __syncthreads();
        for (int i = threadIdx.x; i < entries; i += kThreads)
            if (t.expert[i] >= 0) atomicAdd(&t.count[t.expert[i]], 1);
        for (int i = begin + lane; shared && i < end; i += 32)
            if (t.expert[i] >= 0) atomicAdd(&at[warp * p.E + t.expert[i]], 1u);
        __syncthreads();
        scan_experts<kThreads>(p.E, t.first, s->warp_sum, [&](int e) { return t.count[e]; });
        scan_experts<kThreads>(p.E, t.tile_end, s->warp_sum, [&](int e) { return (t.count[e] + NT - 1) / NT; });
        // first[e] is where expert e's entries end; filled from the last one
        // down it becomes where they begin
        if (shared) {
            for (int e = threadIdx.x; e < p.E; e += kThreads) {
                uint32_t end_at = t.first[e];
                for (int w = kThreads / 32 - 1; w >= 0; --w) {
                    const uint32_t n = at[w * p.E + e];
                    at[w * p.E + e] = end_at;
                    end_at -= n;
                }
                t.first[e] = static_cast<int>(end_at);
            }
            __syncthreads();
        }
        uint32_t* const ends = shared ? at + warp * p.E : reinterpret_cast<uint32_t*>(t.first);
        for (int i0 = begin + (end - begin - 1) / 32 * 32; i0 >= begin && begin < end; i0 -= 32) {
            const int i = i0 + lane, e = i < end ? t.expert[i] : -1;
            const unsigned same = __match_any_sync(0xffffffffu, e);
            if (e >= 0) t.list[ends[e] - __popc(same >> lane)] = static_cast<int16_t>(kGather ? i / p.K : i);
            __syncwarp();
            if (e >= 0 && (same >> lane) == 1u) ends[e] -= __popc(same);
            __syncwarp();
        }
        if (kMode == kFewDown && (shared || warp != 0))
            for (int tok = shared ? threadIdx.x : threadIdx.x - 32; tok < p.T; tok += shared ? kThreads : kThreads - 32) {
                int n = 0;
                for (int k = 0; k < p.K; ++k) n += t.expert[tok * p.K + k] >= 0;
                t.named[tok] = static_cast<uint8_t>(n);
            }
        if (shared) fence_proxy_async_smem();   // before the stages are loaded
    } else {
        expert_blocks<kThreads>(p.expert_offset, p.counts, p.E, p.rows, t.first, t.count, s->warp_rows, p.status);
        scan_experts<kThreads>(p.E, t.tile_end, s->warp_sum, [&](int e) { return (t.count[e] + NT - 1) / NT; });
    }
    tcgen05_before_sync();
    __syncthreads();
    if (kCtas == 2) cluster_sync();   // the pair's barriers are there for either
    tcgen05_after_sync();
    const uint32_t tmem = s->tmem;
    const int tiles = t.tile_end[p.E - 1] * feature_tiles;

    if (kMode == kFewDown && (warp != 0 || worker >= tiles)) pdl_wait();
    if (kMode == kFewDown) pdl_launch_dependents();
    if (kMode == kFewDown && warp >= 4) {
        // tokens of no expert: their residual, or zeros
        for (int tok = blockIdx.x; tok < p.T; tok += gridDim.x) {
            bool any = false;
            for (int k = 0; k < p.K; ++k) any |= t.expert[tok * p.K + k] >= 0;
            if (!any)
                for (int f = threadIdx.x - 128; f < p.F; f += kReadWarps * 32) {
                    const int64_t at = static_cast<int64_t>(tok) * p.F + f;
                    p.out[at] = p.residual ? p.residual[at] : __float2bfloat16(0.0f);
                }
        }
    }

    // Few tokens, down, by the warps that read accumulators: the tokens whose
    // last expert this tile was get their sum over the experts, k ascending,
    // whoever came last.  The tile's rows in every `of`-th 32 are this CTA's.
    const auto sum_tokens = [&](const Tile& r, int first, int of, int which) {
        const int tid = threadIdx.x - 128;
        if (tid == 0) s->completed = 0;
        __threadfence();
        named_barrier(1, kReadWarps * 32);
        for (int j = tid; j < r.rows; j += kReadWarps * 32) {
            if (j / 32 % of != which) continue;
            const int tok = t.list[first + j] / p.K;
            if (!EP_IN((r.f0 / kM) * p.T + tok, p.done_words)) continue;
            const uint32_t before = atomicAdd(&p.done[(r.f0 / kM) * p.T + tok], 1u);
            if (before + 1 == t.named[tok]) {
                __threadfence();
                t.expert[p.T * p.K + atomicAdd(&s->completed, 1)] = static_cast<int16_t>(tok);
            }
        }
        named_barrier(1, kReadWarps * 32);
        // a warp a token, four features a lane, all its experts' rows at once
        const int m = s->completed, feature = r.f0 + lane * 4;
        for (int i = tid / 32; i < m; i += kReadWarps) {
            const int tok = t.expert[p.T * p.K + i];
            if (feature >= p.F || !EP_IN(tok, p.T)) continue;
            const int64_t at = static_cast<int64_t>(tok) * p.F + feature;
            uint2 res = make_uint2(0u, 0u);
            if (p.residual) res = *reinterpret_cast<const uint2*>(p.residual + at);
            float4 part[EP_FEW_MAX_TOPK];
            float weight[EP_FEW_MAX_TOPK];
#pragma unroll
            for (int k = 0; k < EP_FEW_MAX_TOPK; ++k) {
                const int entry = tok * p.K + k;
                const bool there = k < p.K && t.expert[entry] >= 0;
                part[k] = there ? __ldcg(reinterpret_cast<const float4*>(p.part + static_cast<int64_t>(entry) * p.F +
                                                                          feature))
                                : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                weight[k] = there ? p.topk_weights[entry] : 0.0f;
            }
            float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int k = 0; k < EP_FEW_MAX_TOPK; ++k) {
                sum.x = fmaf(weight[k], part[k].x, sum.x);
                sum.y = fmaf(weight[k], part[k].y, sum.y);
                sum.z = fmaf(weight[k], part[k].z, sum.z);
                sum.w = fmaf(weight[k], part[k].w, sum.w);
            }
            if (p.residual) {
                const float2 lo = unpack2(res.x), hi = unpack2(res.y);
                sum.x += lo.x;
                sum.y += lo.y;
                sum.z += hi.x;
                sum.w += hi.y;
            }
            *reinterpret_cast<uint2*>(p.out + at) = make_uint2(pack2(sum.x, sum.y), pack2(sum.z, sum.w));
        }
        named_barrier(1, kReadWarps * 32);
    };

    if (warp == 0) {
        Ring<S::kStages> ring;
        int issued = 0;
        bool ok = true;
        for (int g = worker; g < tiles && ok; g += workers) {
            const Tile r = tile_at<NT, kStep>(g, t, p.E, feature_tiles, tile_features);
            const int share = r.width / kCtas;   // the row operand's rows of each CTA
            const int first = t.first[r.e] + r.row0 + rank * share;
            const auto boxes_of = [&](int who) {
                return (max(0, min(share, r.rows - who * share)) + kBoxRows - 1) / kBoxRows;
            };
            const int boxes = boxes_of(rank);
            const uint32_t bytes = kGather ? kABytes : kCtas * kABytes + (boxes_of(0) + (kCtas == 2 ? boxes_of(1) : 0)) *
                                                         (kBoxRows * kDepth * 2);
            const int f0 = r.f0 + rank * cta_features;
            const auto load_weights = [&](int stage, int kb) {
                uint8_t* const sa = stages + stage * S::kStageBytes;
                uint32_t bar = smem_addr(&s->full[stage]);
                if (kCtas == 2) bar = map_to_rank(bar, 0);
                if (elect_one()) {
                    if (rank == 0) mbar_arrive_expect_tx(&s->full[stage], bytes);
                    if (kMode == kInputGrad) {
                        tma_load_3d<kCtas>(sa, &p.a, bar, f0, kb * kDepth, r.e);
                        tma_load_3d<kCtas>(sa + kABytes / 2, &p.a, bar, f0 + 64, kb * kDepth, r.e);
                    } else if (p.gate_half) {
                        tma_load_5d<kCtas>(sa, &p.a, bar, kb * kDepth, 0, 0, f0 / 8, r.e);
                    } else {
                        tma_load_3d<kCtas>(sa, &p.a, bar, kb * kDepth, f0, r.e);
                    }
                }
                __syncwarp();
            };
            const auto load_rows = [&](int stage, int kb) {
                if (kTestDropFirstLoad && worker == 0 && issued == 0) return;
                uint8_t* const sb = stages + stage * S::kStageBytes + kABytes;
                uint32_t bar = smem_addr(&s->full[stage]);
                if (kCtas == 2) bar = map_to_rank(bar, 0);
                if (elect_one()) {
                    for (int i = 0; i < boxes; ++i)
                        tma_load_2d<kCtas>(sb + i * kBoxRows * kDepth * 2, &p.b, bar, kb * kDepth, first + i * kBoxRows);
                }
                __syncwarp();
            };
            // the down product's first weights come while the up product ends
            int early = 0;
            if (kMode == kFewDown && issued == 0) {
                early = min(S::kStages, kb_end - kb_begin);
                for (int i = 0; i < early; ++i) load_weights(i, kb_begin + i);
                pdl_wait();
            }
            for (int kb = kb_begin; kb < kb_end; ++kb, ++issued, ring.next()) {
                if (issued >= early) {   // (not the first tile: early is 0)
                    ok = warp_wait(&s->empty[ring.stage], ring.parity ^ 1);
                    if (!ok) break;
                    load_weights(ring.stage, kb);
                }
                if (!kGather) load_rows(ring.stage, kb);
            }
        }
        if (!ok) atomicOr(p.status, EP_ERR_TIMEOUT);
        // no copy may still be in flight when the CTA ends (a pair's end: rank 0 sees both CTAs')
        if (rank == 0)
            for (int i = max(0, issued - S::kStages); i < issued; ++i)
                if (!warp_wait(&s->full[i % S::kStages], (i / S::kStages) & 1)) break;
    } else if (warp == 1 && rank == 0) {
        Ring<S::kStages> ring;
        Ring<2> accs;
        constexpr bool kMn = kMode == kInputGrad;
        const uint64_t desc_a = operand_desc(smem_addr(stages), kMn ? kABytes / 2 : 16);
        const uint64_t desc_b = operand_desc(smem_addr(stages) + kABytes, 16);
        bool ok = true;
        for (int g = worker; g < tiles && ok; g += workers, accs.next()) {
            const Tile r = tile_at<NT, kStep>(g, t, p.E, feature_tiles, tile_features);
            const uint32_t idesc = instr_desc(false, kMn, false, kM * kCtas, r.width);
            const uint32_t d = tmem + accs.stage * NT;
            ok = warp_wait(&s->acc_empty[accs.stage], accs.parity ^ 1);
            tcgen05_after_sync();
            for (int kb = kb_begin; kb < kb_end && ok; ++kb, ring.next()) {
                ok = warp_wait(&s->full[ring.stage], ring.parity);
                if (!ok) break;
                tcgen05_after_sync();
                if (elect_one()) {
                    const uint64_t a = desc_at(desc_a, ring.stage * S::kStageBytes);
                    const uint64_t b = desc_at(desc_b, ring.stage * S::kStageBytes);
#pragma unroll
                    for (int k = 0; k < kDepth / 16; ++k)
                        mma<kCtas, false>(d, desc_at(a, k * (kMn ? 2048 : 32)), desc_at(b, k * 32), idesc,
                                          kb > kb_begin || k > 0);
                    mma_commit<kCtas>(&s->empty[ring.stage]);
                    if (kb == kb_end - 1) mma_commit<kCtas>(&s->acc_full[accs.stage]);
                }
                __syncwarp();
            }
        }
        if (!ok) {
            atomicOr(p.status, EP_ERR_TIMEOUT);
            if (elect_one()) mma_commit<kCtas>(&s->drain);
            __syncwarp();
            warp_wait(&s->drain, 0);
        }
    } else if (kGather && (warp == 2 || warp == 3)) {
        // The tokens' rows, 16 bytes a lane, 8 rows at a time, into the places
        // the swizzle gives them.  A stage's copies are waited for when the
        // kLag next ones are on their way (1: 128 tokens of all experts 3.17 ->
        // 3.39 ms; 2, 4 and 5: 6 tokens alike, 143 tokens 61.0, 59.8, 59.6 us, 154
        // tokens 48.0, 48.6, 49.3 against 60.3 and 47.6).
        constexpr int kLag = 3, kCopies = NT / 8;
        static_assert(kLag < S::kStages, "the stage waited for is never the one to be filled");
        Ring<S::kStages> ring, landed;
        const int tid = threadIdx.x - 64, chunk = tid & 7, row0 = tid >> 3;
        const uint32_t place = kABytes + row0 * 128 + ((chunk ^ row0) << 4);
        int in_flight = 0;
        bool ok = true;
        const auto hand_over = [&] {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0 && !(kTestDropFirstLoad && worker == 0 && landed.stage == 0 && landed.parity == 0))
                mbar_arrive(&s->full[landed.stage]);
            landed.next();
            --in_flight;
        };
        for (int g = worker; g < tiles && ok; g += workers) {
            const Tile r = tile_at<NT, kStep>(g, t, p.E, feature_tiles, tile_features);
            const int first = t.first[r.e] + r.row0;
            int tok[kCopies];
#pragma unroll
            for (int i = 0; i < kCopies; ++i) {
                tok[i] = -1;
                if (i * 8 + row0 < r.rows) tok[i] = t.list[first + i * 8 + row0];
                if (tok[i] >= 0 && !EP_IN(tok[i], p.T)) tok[i] = -1;
            }
            for (int kb = kb_begin; kb < kb_end; ++kb, ring.next()) {
                ok = warp_wait(&s->empty[ring.stage], ring.parity ^ 1);
                if (!ok) break;
                const uint32_t sb = smem_addr(stages + ring.stage * S::kStageBytes) + place;
                const int column = kb * kDepth + chunk * 8;
                const bool inside = column < p.depth;   // else zeros
                const __nv_bfloat16* const from = p.x + (inside ? column : 0);
#pragma unroll
                for (int i = 0; i < kCopies; ++i) {
                    if (tok[i] >= 0)
                        copy16_async(sb + i * 1024, from + static_cast<int64_t>(tok[i]) * p.depth, inside);
                }
                copies_commit();
                if (++in_flight > kLag) {
                    copies_wait<kLag>();
                    hand_over();
                }
            }
        }
        if (!ok) atomicOr(p.status, EP_ERR_TIMEOUT);
        while (in_flight > 0) {
            if (in_flight == 3)
                copies_wait<2>();
            else if (in_flight == 2)
                copies_wait<1>();
            else
                copies_wait<0>();
            hand_over();
        }
    } else if (warp >= 4) {
        const int q = warp & 3, turn = (warp - 4) / 4;
        Ring<2> accs;
        for (int g = worker; g < tiles; g += workers, accs.next()) {
            Tile r = tile_at<NT, kStep>(g, t, p.E, feature_tiles, tile_features);
            r.f0 += rank * cta_features;
            const int first = t.first[r.e] + r.row0;
            const uint32_t acc = tmem + accs.stage * NT + (static_cast<uint32_t>(q * 32) << 16);
            const float bias = kMode == kInputGrad ? 0.0f : bias_of(p, r, q, lane);
            Ahead ahead;
            ask_ahead<kMode>(p, t, r, first, q, lane, turn * 32, &ahead);
            const bool ready = warp_wait(&s->acc_full[accs.stage], accs.parity);
            if (!ready) {
                atomicOr(p.status, EP_ERR_TIMEOUT);
                s->gave_up = 1;
            }
            if (kMode == kFewDown) named_barrier(1, kReadWarps * 32);   // its barriers below are for all of these warps
            if (kMode == kFewDown ? *reinterpret_cast<volatile int*>(&s->gave_up) != 0 : !ready) break;
            tcgen05_after_sync();
            const int last = (r.width - 1) / 32;   // 32-column step
            if (kSplit) {   // the only tile: this piece's sums, [column][feature], where the stages were
                for (int step = turn; step <= last; step += 2) {
                    float v[32];
                    tmem_load32(acc + step * 32, v);
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        reinterpret_cast<float*>(stages)[(step * 32 + j) * kM + q * 32 + lane] = v[j];
                }
                continue;
            }
            for (int step = turn; step == turn || step <= last; step += 2) {
                const int c0 = step * 32;
                float v[32];
                __syncwarp();
                if (step <= last) tmem_load32(acc + c0, v);
                if (step + 2 > last) {
                    tcgen05_before_sync();
                    __syncwarp();
                    if (lane == 0) {
                        if (kCtas == 1)
                            mbar_arrive(&s->acc_empty[accs.stage]);
                        else
                            mbar_arrive_cluster_relaxed(map_to_rank(smem_addr(&s->acc_empty[accs.stage]), 0));
                    }
                }
                const Ahead now = ahead;
                if (step + 2 <= last) ask_ahead<kMode>(p, t, r, first, q, lane, c0 + 64, &ahead);
                if (step <= last) finish_columns<kMode>(p, t, r, first, q, lane, bias, c0, v, now);
            }
            if (kMode == kFewDown) sum_tokens(r, first, 1, 0);
        }
    }
    if (kSplit) {
        // the pieces' sums are added in their order, every split-th 32 columns
        // by each CTA
        cluster_sync();
        if (warp >= 4 && worker < tiles) {
            const int q = warp & 3, turn = (warp - 4) / 4;
            const Tile r = tile_at<NT, kStep>(worker, t, p.E, feature_tiles, tile_features);
            const int first = t.first[r.e] + r.row0;
            const float bias = kMode == kInputGrad ? 0.0f : bias_of(p, r, q, lane);
            for (int step = piece + split * turn; step * 32 < r.width; step += 2 * split) {
                Ahead ahead;
                ask_ahead<kMode>(p, t, r, first, q, lane, step * 32, &ahead);
                float v[32] = {};
                for (int from = 0; from < split; ++from) {
                    const uint32_t base = map_to_rank(smem_addr(stages), from) + (step * 32 * kM + q * 32 + lane) * 4;
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] += load_cluster(base + j * kM * 4);
                }
                finish_columns<kMode>(p, t, r, first, q, lane, bias, step * 32, v, ahead);
            }
            if (kMode == kFewDown) sum_tokens(r, first, split, piece);
        }
    }
    if (p.wait_late) pdl_wait();
    __syncthreads();
    // no CTA of a cluster ends while another may still reach it
    if (kCtas == 2 || kSplit) cluster_sync();
    if (warp == 2) tmem_free<kCtas>(tmem, S::kColumns);
}

template <int NT, int kCtas>
size_t smem_bytes(int E, int entries) {
    using S = Shape<NT, kCtas>;
    return 1024 + S::kStages * S::kStageBytes + sizeof(Barriers) + static_cast<size_t>(E) * 12 +
           (entries > 0 ? static_cast<size_t>(entries) * 4 + EP_FEW_MAX_TOKENS * 3 : 0);
}

// tiles_bound: at least as many tiles as there can be, for the grid.  With
// fewer than half as many tiles as SMs a cluster of up to 8 CTAs shares each
// tile's sum, 16 stages or more each: one CTA reads no more than about a
// seventieth of what the memory gives.  (A cluster and the addition cost about
// 2 us, what 10 stages take: 20 stages on two CTAs 14 -> 18 us.)
template <int kMode, int NT, int kCtas, bool kSplit = false>
cudaError_t launch(MmaArgs a, int tiles_bound, cudaStream_t stream) {
    const int sms = device_info().num_sms;
    if constexpr (kCtas == 1 && !kSplit) {
        const int k_blocks = (a.depth + kDepth - 1) / kDepth;
        a.split = 1;
        while (a.split < 8 && tiles_bound * a.split * 2 <= sms && k_blocks >= 32 * a.split) a.split *= 2;
        if (a.split > 1) return launch<kMode, NT, 1, true>(a, tiles_bound, stream);
    }
    const size_t smem = smem_bytes<NT, kCtas>(a.E, a.T * a.K);
    const auto kernel = experts_mma_kernel<kMode, NT, kCtas, kSplit>;
    static std::atomic<bool> ready[kMaxDevices];
    const cudaError_t e = allow_all_smem(reinterpret_cast<const void*>(kernel), ready);
    if (e != cudaSuccess) return e;
    const int cluster = kCtas * (kSplit ? a.split : 1), workers = std::max(1, std::min(sms / cluster, tiles_bound));
    return launch_experts(kernel, dim3(workers * cluster), dim3(kThreads), smem, stream, cluster, a);
}

// Pairs of CTAs halve the row operand's copies into shared memory, whose
// bandwidth (copies in, operands out) bounds one CTA's 128 x 256 tile.  A call
// that has no more tiles than pairs takes single CTAs, twice as many, of half
// as many rows: more of them, and room for six stages instead of four.
template <int kMode>
cudaError_t launch_rows(const MmaArgs& a, cudaStream_t stream) {
    constexpr int kPairRows = 256, kRows = 128;
    const int per = a.gate_half ? kM / 2 : kM;
    const int pairs = bound_tiles(a.rows / kPairRows + a.E, (a.F + 2 * per - 1) / (2 * per));
    if (pairs * 2 > device_info().num_sms) return launch<kMode, kPairRows, 2>(a, pairs, stream);
    return launch<kMode, kRows, 1>(a, bound_tiles(a.rows / kRows + a.E, (a.F + per - 1) / per), stream);
}

// ---------------------------------------------------------------------------
// Weight gradient: dW[e][n, k] = sum over e's rows of dz[row, n] * x[row, k].
// Both operands are read as they lie, rows of the sum outermost (MN-major
// descriptors), 128 n x 256 k a tile.  The last stage of an expert may hold
// rows of the next one, or padding with anything in it: two warps clear those
// rows of both operands in shared memory before the MMAs read them.  The tensor
// cores' fp32 additions truncate, which shows where one accumulator takes very
// many rows: dw is off by 1.7e-3 of its norm (its rounding to bf16) up to 2^17
// rows an expert, 2.0e-3 at 2^20, 5.2e-3 at 2^22, 1.9e-2 at 2^24 (a cluster of 8 on
// the sum: 2.9e-3).  32
// experts x 1024 rows, dw [4096, 7168] each: 1.22 ms, 1.58 PFLOP/s (8 experts x
// 2048 rows: tensor pipe 89% busy); one CTA a tile 1.50 ms.  Few tiles and many
// rows: a cluster's CTAs each take a piece of the rows (kSplit, as above).
// ---------------------------------------------------------------------------

constexpr int kGradK = 256;      // columns of a tile

struct GradArgs {
    CUtensorMap dz, x;           // boxes of 64 columns x 64 rows
    CUtensorMap out;             // dw, boxes of 64 columns x 32 rows
    int Nw, K, E;
    int64_t rows;
    const int32_t* expert_offset;
    const int32_t* counts;
    int32_t* status;
    int split, wait_late;        // as in MmaArgs
};

template <int kCtas>
struct GradShape {
    static constexpr int kColumnsOfX = kGradK / kCtas;   // in one CTA
    static constexpr int kStageBytes = (kM + kColumnsOfX) * kDepth * 2;
    static constexpr int kOutBytes = kReadWarps * 4096;   // a box of dw for each warp of the epilogue
    static constexpr int kStages = (208 * 1024 - kOutBytes) / kStageBytes;
    static constexpr int kColumns = 2 * kGradK;
};

template <int kCtas, bool kSplit>
__global__ void __launch_bounds__(kThreads, 1) weight_grad_kernel(const __grid_constant__ GradArgs p) {
    using S = GradShape<kCtas>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* stages = smem_raw + (1024 - (smem_addr(smem_raw) & 1023)) % 1024;
    uint8_t* boxes = stages + S::kStages * S::kStageBytes;
    Barriers* s = reinterpret_cast<Barriers*>(boxes + S::kOutBytes);
    int* s_first = reinterpret_cast<int*>(s + 1);
    int* s_count = s_first + p.E;
    const int warp = uniform_warp(), lane = threadIdx.x & 31;
    const int rank = kCtas == 2 ? static_cast<int>(cluster_ctarank()) : 0;
    const int n_tiles = (p.Nw + kM * kCtas - 1) / (kM * kCtas), k_tiles = (p.K + kGradK - 1) / kGradK;
    const int tiles = p.E * n_tiles * k_tiles;
    const int split = kSplit ? p.split : 1, piece = kSplit ? static_cast<int>(cluster_ctarank()) : 0;
    const int worker = blockIdx.x / (kCtas * split), workers = gridDim.x / (kCtas * split);

    if (threadIdx.x == 0) {
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(&s->full[i], 1);
            mbar_init(&s->empty[i], 1);
            mbar_init(&s->tail_full[i], 1);
            mbar_init(&s->cleared[i], 2 * kCtas);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s->acc_full[i], 1);
            mbar_init(&s->acc_empty[i], kReadWarps * kCtas);
        }
        mbar_init(&s->drain, 1);
        fence_mbar_init();
        prefetch_map(&p.dz);
        prefetch_map(&p.x);
    }
    if (warp == 2) tmem_alloc<kCtas>(&s->tmem, S::kColumns);
    if (!p.wait_late) pdl_wait();
    pdl_launch_dependents();
    expert_blocks<kThreads>(p.expert_offset, p.counts, p.E, p.rows, s_first, s_count, s->warp_rows, p.status);
    tcgen05_before_sync();
    __syncthreads();
    if (kCtas == 2) cluster_sync();   // the pair's barriers are there for either
    tcgen05_after_sync();
    const uint32_t tmem = s->tmem;
    const auto expert_of = [&](int g) { return g / (n_tiles * k_tiles); };
    const auto n0_of = [&](int g) { return g % (n_tiles * k_tiles) % n_tiles * (kM * kCtas); };
    const auto k0_of = [&](int g) { return g % (n_tiles * k_tiles) / n_tiles * kGradK; };
    // The rows of an expert that this CTA (or pair) sums: [lo, hi).
    const auto lo_of = [&](int cnt) {
        return kSplit ? min(cnt, ((cnt + kDepth - 1) / kDepth + split - 1) / split * kDepth * piece) : 0;
    };
    const auto hi_of = [&](int cnt) {
        return kSplit ? min(cnt, ((cnt + kDepth - 1) / kDepth + split - 1) / split * kDepth * (piece + 1)) : cnt;
    };

    // 32 rows x 64 columns of dw through shared memory, by one warp: a warp
    // storing 16 bytes of 32 rows at a time kept its loads waiting.  take(c, v):
    // this lane's row, columns c .. c + 31 of the tile (v comes as zeros).
    const auto store_box = [&](int c0, int row0, int k0, int e, auto take) {
        uint8_t* const box = boxes + (warp - 4) * 4096;
        if (lane == 0) bulk_wait_read<0>();   // the store before
        __syncwarp();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float v[32] = {};
            take(c0 + 32 * h, v);
#pragma unroll
            for (int c = 0; c < 32; c += 8)
                *reinterpret_cast<uint4*>(box + lane * 128 + ((4 * h + c / 8) ^ (lane & 7)) * 16) =
                    make_uint4(pack2(v[c], v[c + 1]), pack2(v[c + 2], v[c + 3]), pack2(v[c + 4], v[c + 5]),
                               pack2(v[c + 6], v[c + 7]));
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && EP_IN(e, p.E) && EP_IN(row0, p.Nw) && EP_IN(k0 + c0, p.K)) {
            tma_store_3d(&p.out, box, k0 + c0, row0, e);
            bulk_commit();
        }
    };

    if (warp == 0) {
        Ring<S::kStages> ring;
        int issued = 0;
        uint32_t tail_bits = 0, full_bits = 0, last_tail = 0;   // parities of the stages' next loads
        bool ok = true;
        for (int g = worker; g < tiles && ok; g += workers) {
            const int e = expert_of(g), n0 = n0_of(g), k0 = k0_of(g), cnt = s_count[e], first = s_first[e];
            const auto a_boxes = [&](int who) { return max(0, min(2, (p.Nw - n0 - who * kM + 63) / 64)); };
            const auto b_boxes = [&](int who) {
                return max(0, min(S::kColumnsOfX / 64, (p.K - k0 - who * S::kColumnsOfX + 63) / 64));
            };
            const int mine_a = a_boxes(rank), mine_b = b_boxes(rank);
            const int all = a_boxes(0) + b_boxes(0) + (kCtas == 2 ? a_boxes(1) + b_boxes(1) : 0);
            const int hi = hi_of(cnt);
            for (int r = lo_of(cnt); r < hi; r += kDepth, ++issued, ring.next()) {
                ok = warp_wait(&s->empty[ring.stage], ring.parity ^ 1);
                if (!ok) break;
                const uint32_t bit = 1u << ring.stage;
                const bool tail = r + kDepth > cnt;
                (tail ? tail_bits : full_bits) ^= bit;
                last_tail = tail ? last_tail | bit : last_tail & ~bit;
                if (elect_one()) {
                    uint8_t* const sa = stages + ring.stage * S::kStageBytes;
                    uint8_t* const sb = sa + kABytes;
                    const int nx = n0 + rank * kM, kx = k0 + rank * S::kColumnsOfX;
                    const bool drop = kTestDropFirstLoad && worker == 0 && issued == 0;
                    if (tail) {   // each CTA's own barrier: its warps clear rows first
                        const uint32_t bar = smem_addr(&s->tail_full[ring.stage]);
                        mbar_arrive_expect_tx(&s->tail_full[ring.stage], (mine_a + mine_b) * 8192);
                        for (int i = 0; i < mine_a; ++i)
                            tma_load_2d<1>(sa + i * 8192, &p.dz, bar, nx + 64 * i, first + r);
                        for (int i = 0; i < mine_b && !drop; ++i)
                            tma_load_2d<1>(sb + i * 8192, &p.x, bar, kx + 64 * i, first + r);
                    } else {
                        uint32_t bar = smem_addr(&s->full[ring.stage]);
                        if (kCtas == 2) bar = map_to_rank(bar, 0);
                        if (rank == 0) mbar_arrive_expect_tx(&s->full[ring.stage], all * 8192);
                        for (int i = 0; i < mine_a; ++i)
                            tma_load_2d<kCtas>(sa + i * 8192, &p.dz, bar, nx + 64 * i, first + r);
                        for (int i = 0; i < mine_b && !drop; ++i)
                            tma_load_2d<kCtas>(sb + i * 8192, &p.x, bar, kx + 64 * i, first + r);
                    }
                }
                __syncwarp();
            }
        }
        if (!ok) atomicOr(p.status, EP_ERR_TIMEOUT);
        // no copy may still be in flight when the CTA ends (a pair's end: rank 0 sees both CTAs')
        for (int st = 0; st < S::kStages && st < issued; ++st) {
            const bool tail = (last_tail >> st) & 1;
            if (!tail && rank != 0) continue;
            if (!warp_wait(tail ? &s->tail_full[st] : &s->full[st], (((tail ? tail_bits : full_bits) >> st) & 1) ^ 1))
                break;
        }
    } else if (warp == 1 && rank == 0) {
        const uint32_t idesc = instr_desc(false, true, true, kM * kCtas, kGradK);
        const uint64_t desc_a = operand_desc(smem_addr(stages), 8192);
        const uint64_t desc_b = operand_desc(smem_addr(stages) + kABytes, 8192);
        Ring<S::kStages> ring;
        Ring<2> accs;
        uint32_t tail_bits = 0, full_bits = 0;
        bool ok = true;
        for (int g = worker; g < tiles && ok; g += workers) {
            const int cnt = s_count[expert_of(g)], lo = lo_of(cnt), hi = hi_of(cnt);
            if (lo >= hi) continue;
            const uint32_t d = tmem + accs.stage * kGradK;
            ok = warp_wait(&s->acc_empty[accs.stage], accs.parity ^ 1);
            tcgen05_after_sync();
            for (int r = lo; r < hi && ok; r += kDepth, ring.next()) {
                const bool tail = r + kDepth > cnt;
                ok = warp_wait(tail ? &s->cleared[ring.stage] : &s->full[ring.stage],
                               ((tail ? tail_bits : full_bits) >> ring.stage) & 1);
                (tail ? tail_bits : full_bits) ^= 1u << ring.stage;
                if (!ok) break;
                tcgen05_after_sync();
                if (elect_one()) {
                    const uint64_t a = desc_at(desc_a, ring.stage * S::kStageBytes);
                    const uint64_t b = desc_at(desc_b, ring.stage * S::kStageBytes);
#pragma unroll
                    for (int k = 0; k < kDepth / 16; ++k)
                        mma<kCtas, false>(d, desc_at(a, k * 2048), desc_at(b, k * 2048), idesc, r > lo || k > 0);
                    mma_commit<kCtas>(&s->empty[ring.stage]);
                    if (r + kDepth >= hi) mma_commit<kCtas>(&s->acc_full[accs.stage]);
                }
                __syncwarp();
            }
            accs.next();
        }
        if (!ok) {
            atomicOr(p.status, EP_ERR_TIMEOUT);
            if (elect_one()) mma_commit<kCtas>(&s->drain);
            __syncwarp();
            warp_wait(&s->drain, 0);
        }
    } else if (warp == 2 || warp == 3) {
        int it = 0;
        uint32_t tail_bits = 0;
        for (int g = worker; g < tiles; g += workers) {
            const int cnt = s_count[expert_of(g)], lo = lo_of(cnt), hi = hi_of(cnt), valid = cnt % kDepth;
            it += (hi - lo + kDepth - 1) / kDepth;
            if (valid == 0 || lo >= hi || hi < cnt) continue;
            const int st = (it - 1) % S::kStages;
            if (!warp_wait(&s->tail_full[st], (tail_bits >> st) & 1)) {
                atomicOr(p.status, EP_ERR_TIMEOUT);
                break;
            }
            tail_bits ^= 1u << st;
            // whole 128-byte rows of every 64-column box, so the swizzle does not matter
            const int clear = (kDepth - valid) * 8;
            uint8_t* base = stages + st * S::kStageBytes + valid * 128;
            for (int box = 0; box < (kM + S::kColumnsOfX) / 64; ++box)
                for (int i = (warp - 2) * 32 + lane; i < clear; i += 64)
                    *reinterpret_cast<uint4*>(base + box * 8192 + i * 16) = make_uint4(0, 0, 0, 0);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                if (kCtas == 1)
                    mbar_arrive(&s->cleared[st]);
                else
                    mbar_arrive_cluster(map_to_rank(smem_addr(&s->cleared[st]), 0));
            }
        }
    } else if (warp >= 4) {
        const int q = warp & 3, turn = (warp - 4) / 4;
        Ring<2> accs;
        for (int g = worker; g < tiles; g += workers) {
            const int e = expert_of(g), n0 = n0_of(g) + rank * kM, k0 = k0_of(g), cnt = s_count[e];
            const int row0 = n0 + q * 32;
            const bool sums = lo_of(cnt) < hi_of(cnt);
            if (sums) {
                if (!warp_wait(&s->acc_full[accs.stage], accs.parity)) {
                    atomicOr(p.status, EP_ERR_TIMEOUT);
                    break;
                }
                tcgen05_after_sync();
            }
            const uint32_t acc = tmem + accs.stage * kGradK + (static_cast<uint32_t>(q * 32) << 16);
            const int width = row0 < p.Nw ? min(kGradK, p.K - k0) : 0;   // the rows past Nw in a box are not stored
            if (kSplit) {   // the only tile: this piece's sums, [column][row], where the stages were
                for (int c0 = turn * 32; c0 < width; c0 += 64) {
                    float v[32] = {};
                    if (sums) tmem_load32(acc + c0, v);
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        reinterpret_cast<float*>(stages)[(c0 + j) * kM + q * 32 + lane] = v[j];
                }
                continue;
            }
            const auto release = [&] {   // the accumulator has been read
                tcgen05_before_sync();
                __syncwarp();
                if (lane == 0) {
                    if (kCtas == 1)
                        mbar_arrive(&s->acc_empty[accs.stage]);
                    else
                        mbar_arrive_cluster_relaxed(map_to_rank(smem_addr(&s->acc_empty[accs.stage]), 0));
                }
            };
            if (sums && turn * 64 >= width) release();
            for (int c0 = turn * 64; c0 < width; c0 += 128) {
                store_box(c0, row0, k0, e, [&](int c, float (&v)[32]) {
                    if (sums) tmem_load32(acc + c, v);
                    if (sums && c0 + 128 >= width && c > c0) release();
                });
            }
            if (sums) accs.next();
        }
        if (lane == 0) bulk_wait_all<0>();
        __syncwarp();
    }
    if (kSplit) {
        cluster_sync();
        if (warp >= 4 && worker < tiles) {
            const int q = warp & 3, turn = (warp - 4) / 4;
            const int n0 = n0_of(worker), k0 = k0_of(worker), row0 = n0 + q * 32;
            const int width = row0 < p.Nw ? min(kGradK, p.K - k0) : 0;
            for (int step = piece + split * turn; step * 64 < width; step += 2 * split)
                store_box(step * 64, row0, k0, expert_of(worker), [&](int c, float (&v)[32]) {
                    if (c < width)
                        for (int from = 0; from < split; ++from) {
                            const uint32_t base =
                                map_to_rank(smem_addr(stages), from) + (c * kM + q * 32 + lane) * 4;
#pragma unroll
                            for (int j = 0; j < 32; ++j) v[j] += load_cluster(base + j * kM * 4);
                        }
                });
            if (lane == 0) bulk_wait_all<0>();
            __syncwarp();
        }
    }
    if (p.wait_late) pdl_wait();
    __syncthreads();
    // no CTA of a cluster ends while another may still reach it
    if (kCtas == 2 || kSplit) cluster_sync();
    if (warp == 2) tmem_free<kCtas>(tmem, S::kColumns);
}

template <int kCtas, bool kSplit = false>
cudaError_t launch_grad(const GradArgs& a, int64_t tiles, cudaStream_t stream) {
    using S = GradShape<kCtas>;
    const auto kernel = weight_grad_kernel<kCtas, kSplit>;
    const size_t smem = 1024 + S::kStages * S::kStageBytes + S::kOutBytes + sizeof(Barriers) + 8 * static_cast<size_t>(a.E);
    static std::atomic<bool> ready[kMaxDevices];
    const cudaError_t e = allow_all_smem(reinterpret_cast<const void*>(kernel), ready);
    if (e != cudaSuccess) return e;
    const int cluster = kCtas * (kSplit ? a.split : 1);
    const int workers = static_cast<int>(std::min<int64_t>(device_info().num_sms / cluster, tiles));
    return launch_experts(kernel, dim3(std::max(1, workers) * cluster), dim3(kThreads), smem, stream, cluster, a);
}

}  // namespace

cudaError_t launch_expert_gemm_bf16(const ExpertGemmParams& p, cudaStream_t stream) {
    MmaArgs a = product_args(p);
    if (!(a.gate_half ? gated_map(&a.a, p.w, p.E, p.N, p.K) : weight_map(&a.a, p.w, p.E, p.Nw, p.K, kM)) ||
        !row_map(&a.b, p.x, p.rows, p.K, kDepth))
        return cudaErrorInvalidValue;
    return launch_rows<kProduct>(a, stream);
}

cudaError_t launch_input_grad(const ExpertBackwardParams& p, const __nv_bfloat16* dz, bool wait_late,
                              cudaStream_t stream) {
    MmaArgs a{};
    if (!weight_map(&a.a, p.w, p.E, p.Nw, p.K, kDepth) || !row_map(&a.b, dz, p.rows, p.Nw, kDepth))
        return cudaErrorInvalidValue;
    a.depth = p.Nw;
    a.F = p.K;
    a.E = p.E;
    a.rows = p.rows;
    a.expert_offset = p.expert_offset;
    a.counts = p.counts;
    a.y = p.dx;
    a.status = p.status;
    a.wait_late = wait_late;
    return launch_rows<kInputGrad>(a, stream);
}

cudaError_t launch_weight_grad(const ExpertBackwardParams& p, const __nv_bfloat16* dz, bool wait_late,
                               cudaStream_t stream) {
    GradArgs a{};
    a.wait_late = wait_late;
    // no rows: nothing is loaded, but a map needs an extent
    const int64_t rows = std::max<int64_t>(p.rows, 1);
    if (!row_map(&a.dz, p.rows > 0 ? dz : p.dw, rows, p.Nw, kDepth) ||
        !row_map(&a.x, p.rows > 0 ? p.x : p.dw, rows, p.K, kDepth) || !weight_map(&a.out, p.dw, p.E, p.Nw, p.K, 32))
        return cudaErrorInvalidValue;
    a.Nw = p.Nw;
    a.K = p.K;
    a.E = p.E;
    a.rows = p.rows;
    a.expert_offset = p.expert_offset;
    a.counts = p.counts;
    a.status = p.status;
    const auto tiles = [&](int n) {
        return static_cast<int64_t>(p.E) * ((p.Nw + n - 1) / n) * ((p.K + kGradK - 1) / kGradK);
    };
    if (tiles(kM) > INT32_MAX) return cudaErrorInvalidValue;
    // pairs, as for the rows' products, unless they would leave SMs idle
    if (tiles(2 * kM) * 2 > device_info().num_sms) return launch_grad<2>(a, tiles(2 * kM), stream);
    // few tiles: pieces of 8 stages of rows or more
    const int64_t blocks = p.rows / p.E / kDepth;
    a.split = 1;
    while (a.split < 8 && tiles(kM) * a.split * 2 <= device_info().num_sms && blocks >= 16 * a.split) a.split *= 2;
    return a.split > 1 ? launch_grad<1, true>(a, tiles(kM), stream) : launch_grad<1>(a, tiles(kM), stream);
}

cudaError_t launch_few_tokens(const FewTokensParams& p, cudaStream_t stream) {
    constexpr int NT = 64;
    MmaArgs up{};
    const bool gated = p.act == EP_ACT_SWIGLU;
    if (!(gated ? gated_map(&up.a, p.w_up, p.E, p.I, p.H) : weight_map(&up.a, p.w_up, p.E, p.Nw, p.H, kM)))
        return cudaErrorInvalidValue;
    up.depth = p.H;
    up.F = p.I;
    up.gate_half = gated ? p.I : 0;
    up.E = p.E;
    up.act = p.act;
    up.x = p.x;
    up.topk_idx = p.topk_idx;
    up.topk_weights = p.topk_weights;
    up.T = p.T;
    up.K = p.K;
    up.rows = static_cast<int64_t>(p.T) * p.K;
    up.bias = p.bias_up;
    up.y = p.h;
    up.done = p.done;
    up.done_words = (p.H + kM - 1) / kM * p.T;
    up.status = p.status;
    MmaArgs down = up;
    if (!weight_map(&down.a, p.w_down, p.E, p.H, p.I, kM) ||
        !row_map(&down.b, p.h, static_cast<int64_t>(p.T) * p.K, p.I, kFewBoxRows))
        return cudaErrorInvalidValue;
    down.depth = p.I;
    down.F = p.H;
    down.gate_half = 0;
    down.act = EP_ACT_NONE;
    down.bias = p.bias_down;
    down.y = nullptr;
    down.part = p.part;
    down.residual = p.residual;
    down.out = p.out;
    const int entries = p.T * p.K, active = std::min(p.E, entries);
    const int per = gated ? kM / 2 : kM;
    cudaError_t e = launch<kFewUp, NT, 1>(up, bound_tiles(active + entries / NT, (p.I + per - 1) / per), stream);
    if (e != cudaSuccess) return e;
    return launch<kFewDown, NT, 1>(down, bound_tiles(active + entries / NT, (p.H + kM - 1) / kM), stream);
}

}  // namespace epg
