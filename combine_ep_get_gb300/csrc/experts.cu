// The experts between dispatch and combine: matrix product with its epilogue,
// its gradients, and the whole layer for a few tokens (the contract is in
// include/ep_get.h).  Plain tiled kernels: 64 x 64 outputs a block, 16 terms
// at a time through shared memory, fp32 multiply-adds.
#include <cuda_fp8.h>

#include "experts.cuh"

namespace epg {
namespace {

constexpr int kT = 64, kD = 16;

// acc[i][j] += sum over k < depth of a(m, k) * b(n, k), m = 4 * ty + i, n = 4 * tx + j
template <class A, class B>
__device__ __forceinline__ void tile_product(float (&acc)[4][4], int64_t depth, A a, B b) {
    __shared__ float sa[kD][kT + 1], sb[kD][kT + 1];
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    for (int64_t k0 = 0; k0 < depth; k0 += kD) {
        for (int i = tid; i < kT * kD; i += 256) {
            const int r = i / kD, k = i % kD;
            sa[k][r] = k0 + k < depth ? a(r, k0 + k) : 0.0f;
            sb[k][r] = k0 + k < depth ? b(r, k0 + k) : 0.0f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kD; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sa[k][4 * ty + i], sb[k][4 * tx + j], acc[i][j]);
        __syncthreads();
    }
}

__device__ __forceinline__ float bf(const __nv_bfloat16* p, int64_t i) { return __bfloat162float(p[i]); }

template <bool kFp8>
__device__ __forceinline__ float load(const uint8_t* p, int64_t i) {
    if (kFp8) {
        __nv_fp8_e4m3 v;
        v.__x = p[i];
        return static_cast<float>(v);
    }
    return bf(reinterpret_cast<const __nv_bfloat16*>(p), i);
}

// grid (column tiles, E): every block walks its expert's row tiles
template <bool kFp8>
__global__ void __launch_bounds__(256) product_kernel(const __grid_constant__ ExpertGemmParams p) {
    const int e = blockIdx.y, n0 = blockIdx.x * kT, tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    int64_t first;
    const int cnt = expert_rows(p.expert_offset, p.counts, e, p.rows, &first, p.status);
    const bool gated = p.act == EP_ACT_SWIGLU;
    for (int m0 = 0; m0 < cnt; m0 += kT) {
        float acc[2][4][4] = {};
        const auto a = [&](int r, int64_t k) {
            if (m0 + r >= cnt) return 0.0f;
            const int64_t d = first + m0 + r;
            const float v = load<kFp8>(p.x, d * p.K + k);
            return kFp8 ? v * p.x_sf[d * p.sf_row + k / 128 * p.sf_block] : v;
        };
        for (int half = 0; half < (gated ? 2 : 1); ++half)
            tile_product(acc[half], p.K, a, [&](int c, int64_t k) {
                if (n0 + c >= p.N) return 0.0f;
                const int64_t n = half * p.N + n0 + c;
                const float v = load<kFp8>(p.w, (static_cast<int64_t>(e) * p.Nw + n) * p.K + k);
                return kFp8 ? v * p.w_sf[(e * (p.Nw / 128) + n / 128) * (p.K / 128) + k / 128] : v;
            });
        for (int i = 0; i < 4; ++i)
            for (int j = 0; j < 4; ++j) {
                const int r = m0 + 4 * ty + i, n = n0 + 4 * tx + j;
                if (r >= cnt || n >= p.N) continue;
                const int64_t d = first + r;
                float z[2] = {acc[0][i][j], acc[1][i][j]};
                for (int half = 0; half < (gated ? 2 : 1); ++half) {
                    if (p.bias) z[half] += p.bias[static_cast<int64_t>(e) * p.Nw + half * p.N + n];
                    if (p.z) p.z[d * p.Nw + half * p.N + n] = __float2bfloat16(z[half]);
                }
                float v = gated ? silu(z[0]) * z[1] : activate(z[0], p.act);
                if (p.row_weight) v *= p.row_weight[d];
                if (p.residual) v += bf(p.residual, d * p.N + n);
                p.y[d * p.N + n] = __float2bfloat16(v);
            }
    }
}

}  // namespace

cudaError_t launch_expert_gemm(const ExpertGemmParams& p, bool fp8, cudaStream_t stream) {
    if (!fp8) return launch_expert_gemm_bf16(p, stream);
    const dim3 grid((p.N + kT - 1) / kT, p.E);
    product_kernel<true><<<grid, 256, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace epg
