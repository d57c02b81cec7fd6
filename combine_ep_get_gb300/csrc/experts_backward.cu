// Gradients of the experts' product: the activation's backward pass with the
// bias' and the row weights' gradients, then the two matrix products
// (experts_mma.cu).
//
// The activation's pass reads dy and z and writes dz, each once: it is bound
// by memory (SWIGLU, 16384 rows x 2048: 336 MB in 55 us, 6.1 TB/s; 80
// registers, three blocks an SM, against 60 us for two and 80 us for four) or,
// GELU with a row weight, by its arithmetic (17004 rows x 1296: 36 us).  dz is
// rounded to bf16 for the tensor cores, once, and both products take the
// rounded one (dx and dw are then off by 2.3e-3 of their norms, 1.7e-3 of it
// their own rounding); its sums do not.  A block takes 32 rows of one expert x 256 columns (a strip),
// each thread 8 neighbouring columns (16-byte loads and stores) of every
// eighth row.  The bias' gradient is the sum of dz down the rows: 32 rows in
// a block's registers, before dz is rounded, the blocks' sums then added in
// order by a second kernel.  The row weights' gradient is the sum along a row
// of dy * act(z): a strip's sum by shuffles, the strips' sums added in order
// by the same second kernel.  No atomics: results do not depend on timing.
#include "experts.cuh"

namespace epg {
namespace {

constexpr int kThreads = 256;
constexpr int kVecs = kBackwardStrip / 8;      // 8-column vectors of a strip
constexpr int kRowLanes = kThreads / kVecs;    // rows at a time
constexpr int kAhead = kBackwardTileRows / kRowLanes;   // rows of a thread
static_assert(kVecs == 32, "a warp has a row of the strip");

__device__ __forceinline__ void unpack8(uint4 v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

struct Tables {
    int* tile_end;   // [E] row tiles of experts 0 .. e
    int* first;
    int* count;
};

__device__ __forceinline__ Tables row_tables(const ExpertBackwardParams& p, int* smem, int* warp_sum) {
    __shared__ int64_t warp_rows[kThreads / 32];
    Tables t;
    t.tile_end = smem;
    t.first = smem + p.E;
    t.count = t.first + p.E;
    const bool fit =
        expert_blocks<kThreads>(p.expert_offset, p.counts, p.E, p.rows, t.first, t.count, warp_rows, p.status);
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.blocks_fit = fit;
    scan_experts<kThreads>(p.E, t.tile_end, warp_sum,
                           [&](int e) { return (t.count[e] + kBackwardTileRows - 1) / kBackwardTileRows; });
    return t;
}

// act(z) and its derivative together (of the gated one's gate).
template <int kAct>
__device__ __forceinline__ void activate_both(float z, float* a, float* slope) {
    if (kAct == EP_ACT_RELU) {
        *a = z < 0.0f ? 0.0f : z;
        *slope = z > 0.0f ? 1.0f : 0.0f;
    } else if (kAct == EP_ACT_GELU) {
        float density;
        const float cdf = normal_cdf(z, &density);
        *a = z * cdf;
        *slope = fmaf(z, density, cdf);
    } else if (kAct == EP_ACT_SILU || kAct == EP_ACT_SWIGLU) {
        const float s = sigmoid(z);
        *a = z * s;
        *slope = s * (1.0f + z * (1.0f - s));
    } else {
        *a = z;
        *slope = 1.0f;
    }
}

template <int kAct>
__global__ void __launch_bounds__(kThreads, 3) activation_backward_kernel(const __grid_constant__ ExpertBackwardParams p) {
    constexpr bool kGated = kAct == EP_ACT_SWIGLU;
    extern __shared__ int tables[];
    __shared__ int warp_sum[kThreads / 32];
    __shared__ float sums[kRowLanes][kBackwardStrip];
    pdl_wait();
    pdl_launch_dependents();
    const Tables t = row_tables(p, tables, warp_sum);
    const int strips = (p.N + kBackwardStrip - 1) / kBackwardStrip;
    const int row_tiles = t.tile_end[p.E - 1];
    const int vec = threadIdx.x % kVecs, row_lane = threadIdx.x / kVecs;
    const bool need_z = kAct != EP_ACT_NONE || p.d_row_weight;
    for (int64_t g = blockIdx.x; g < static_cast<int64_t>(row_tiles) * strips; g += gridDim.x) {
        const int tile = static_cast<int>(g / strips), strip = static_cast<int>(g % strips);
        int lo = 0, hi = p.E - 1;
        while (lo < hi) {
            const int mid = (lo + hi) / 2;
            if (t.tile_end[mid] > tile)
                hi = mid;
            else
                lo = mid + 1;
        }
        const int row0 = (tile - (lo > 0 ? t.tile_end[lo - 1] : 0)) * kBackwardTileRows;
        const int rows = min(kBackwardTileRows, t.count[lo] - row0);
        const int64_t first = static_cast<int64_t>(t.first[lo]) + row0;
        const int n = strip * kBackwardStrip + vec * 8;
        // a thread's rows are all asked for before the first is used; rows and
        // columns that are not there are zeros
        uint4 dy_v[kAhead], z_v[kAhead], u_v[kAhead];
        float w_v[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int r = row_lane + j * kRowLanes;
            const int64_t d = first + r;
            const bool here = n < p.N && r < rows && EP_IN(d, p.rows);
            const uint4 zero = make_uint4(0, 0, 0, 0);
            dy_v[j] = here ? ld_stream_v4(p.dy + d * p.N + n) : zero;
            z_v[j] = here && need_z ? ld_stream_v4(p.z + d * p.Nw + n) : zero;
            if (kGated) u_v[j] = here ? ld_stream_v4(p.z + d * p.Nw + p.N + n) : zero;
            w_v[j] = here && p.row_weight ? p.row_weight[d] : 1.0f;
        }
        float sum[kGated ? 2 : 1][8] = {};
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int r = row_lane + j * kRowLanes;
            const int64_t d = first + r;
            const bool here = n < p.N && r < rows && EP_IN(d, p.rows);
            float dy[8], z[8], u[8], dz[8], du[8], dot = 0.0f;
            unpack8(dy_v[j], dy);
            unpack8(z_v[j], z);
            if (kGated) unpack8(u_v[j], u);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float da = dy[i] * w_v[j];
                float a, slope;
                activate_both<kAct>(z[i], &a, &slope);
                if (kGated) {
                    dz[i] = da * u[i] * slope;
                    du[i] = da * a;
                    sum[kGated ? 1 : 0][i] += du[i];
                    a *= u[i];
                } else {
                    dz[i] = da * slope;
                }
                sum[0][i] += dz[i];
                dot = fmaf(dy[i], a, dot);
            }
            if (p.dz && here) {
                st_v4(p.dz + d * p.Nw + n, pack8(dz));
                if (kGated) st_v4(p.dz + d * p.Nw + p.N + n, pack8(du));
            }
            if (p.d_row_weight) {   // a row of the strip is one warp's
                for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
                if (vec == 0 && r < rows && EP_IN(d, p.rows)) p.weight_part[strip * p.rows + d] = dot;
            }
        }
        if (p.dbias)
            for (int half = 0; half < (kGated ? 2 : 1); ++half) {
                __syncthreads();
#pragma unroll
                for (int i = 0; i < 8; ++i) sums[row_lane][vec * 8 + i] = sum[half][i];
                __syncthreads();
                for (int c = threadIdx.x; c < kBackwardStrip; c += kThreads)
                    if (strip * kBackwardStrip + c < p.N && EP_IN(tile, p.rows / kBackwardTileRows + p.E)) {
                        float v = 0.0f;
                        for (int i = 0; i < kRowLanes; ++i) v += sums[i][c];
                        p.bias_part[static_cast<int64_t>(tile) * p.Nw + half * p.N + strip * kBackwardStrip + c] = v;
                    }
            }
    }
}

// The partial sums, in order: blocks of `columns` columns of every expert's
// dbias, kThreads / columns threads taking turns at a column's row tiles, then
// row_blocks blocks for every expert's rows of d_row_weight.
__global__ void __launch_bounds__(kThreads) backward_sums_kernel(const __grid_constant__ ExpertBackwardParams p,
                                                                 int columns, int bias_blocks, int row_blocks) {
    __shared__ int warp_sum[kThreads / 32];
    __shared__ float sums[kThreads];
    pdl_wait();
    pdl_launch_dependents();
    const int column_blocks = (p.Nw + columns - 1) / columns;
    const bool fit = p.rows == 0 || *p.blocks_fit;   // (without rows there was no pass before)
    int64_t first;
    if (static_cast<int>(blockIdx.x) >= bias_blocks) {
        const int block = blockIdx.x - bias_blocks, e = block / row_blocks;
        const int cnt = fit ? expert_rows(p.expert_offset, p.counts, e, p.rows, &first, p.status) : 0;
        const int strips = (p.N + kBackwardStrip - 1) / kBackwardStrip;
        for (int r = block % row_blocks * kThreads + threadIdx.x; r < cnt; r += row_blocks * kThreads) {
            float v = 0.0f;
            for (int i = 0; i < strips; ++i) v += p.weight_part[i * p.rows + first + r];
            if (EP_IN(first + r, p.rows)) p.d_row_weight[first + r] = v;
        }
        return;
    }
    const int e = blockIdx.x / column_blocks, c = threadIdx.x % columns, part = threadIdx.x / columns;
    const int n = blockIdx.x % column_blocks * columns + c, parts = kThreads / columns;
    // row tiles of the experts before this one
    int before = 0;
    for (int i = threadIdx.x; i < e; i += kThreads)
        before += (expert_rows(p.expert_offset, p.counts, i, p.rows, &first, p.status) + kBackwardTileRows - 1) /
                  kBackwardTileRows;
    for (int o = 16; o > 0; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
    if ((threadIdx.x & 31) == 0) warp_sum[threadIdx.x / 32] = before;
    __syncthreads();
    before = 0;
    for (int w = 0; w < kThreads / 32; ++w) before += warp_sum[w];
    const int rows = fit ? expert_rows(p.expert_offset, p.counts, e, p.rows, &first, p.status) : 0;
    const int tiles = (rows + kBackwardTileRows - 1) / kBackwardTileRows;
    float v = 0.0f;
    if (n < p.Nw)
#pragma unroll 8
        for (int i = part; i < tiles; i += parts)
            if (EP_IN(before + i, p.rows / kBackwardTileRows + p.E))
                v += p.bias_part[static_cast<int64_t>(before + i) * p.Nw + n];
    if (parts > 1) {
        sums[threadIdx.x] = v;
        __syncthreads();
        if (part > 0) return;
        for (int i = 1; i < parts; ++i) v += sums[i * columns + c];
    }
    if (n < p.Nw && EP_IN(e, p.E)) p.dbias[static_cast<int64_t>(e) * p.Nw + n] = v;
}

}  // namespace

cudaError_t launch_expert_backward(const ExpertBackwardParams& given, cudaStream_t stream) {
    ExpertBackwardParams p = given;
    // without activation and row weight dz is dy
    const bool plain = p.act == EP_ACT_NONE && !p.row_weight;
    const __nv_bfloat16* dz = plain ? p.dy : p.dz;
    if (plain || (!p.dx && !p.dw)) p.dz = nullptr;
    if (p.rows > 0 && (p.dz || p.dbias || p.d_row_weight)) {
        void (*const kernels[])(ExpertBackwardParams) = {
            activation_backward_kernel<EP_ACT_NONE>, activation_backward_kernel<EP_ACT_RELU>,
            activation_backward_kernel<EP_ACT_GELU>, activation_backward_kernel<EP_ACT_SILU>,
            activation_backward_kernel<EP_ACT_SWIGLU>};
        const int64_t tiles =
            (p.rows / kBackwardTileRows + p.E) * static_cast<int64_t>((p.N + kBackwardStrip - 1) / kBackwardStrip);
        // one wave: the table of row tiles is built once a block
        const int grid = static_cast<int>(tiles < device_info().num_sms * 3 ? tiles : device_info().num_sms * 3);
        const cudaError_t e = launch_experts(kernels[p.act], dim3(grid), dim3(kThreads),
                                              static_cast<size_t>(p.E) * 12, stream, 1, p);
        if (e != cudaSuccess) return e;
    }
    if (p.dbias || p.d_row_weight) {
        // few row tiles an expert: a thread a column; many: eight threads
        const int64_t tiles = p.rows / kBackwardTileRows / p.E;
        const int columns = tiles < 8 ? 256 : tiles < 32 ? 64 : 32;
        const int64_t bias_blocks = p.dbias ? static_cast<int64_t>(p.E) * ((p.Nw + columns - 1) / columns) : 0;
        const int row_blocks = p.E < 64 ? 16 : p.E < 1024 ? 1024 / p.E : 1;
        const int64_t blocks = bias_blocks + (p.d_row_weight ? static_cast<int64_t>(row_blocks) * p.E : 0);
        if (blocks > INT32_MAX) return cudaErrorInvalidValue;
        const cudaError_t e = launch_experts(backward_sums_kernel, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0,
                                         stream, 1, p, columns, static_cast<int>(bias_blocks), row_blocks);
        if (e != cudaSuccess) return e;
    }
    // Both products need only dz.  A kernel between them and dz's has waited
    // for dz before it let them start, so they need not wait for it to end
    // until they end themselves ("Reads before the wait" in experts.cuh): each
    // fills the SMs that the one before frees.
    bool late = p.dbias || p.d_row_weight;
    if (p.dx) {
        const cudaError_t e = launch_input_grad(p, dz, late, stream);
        if (e != cudaSuccess) return e;
        late = true;
    }
    return p.dw ? launch_weight_grad(p, dz, late, stream) : cudaSuccess;
}

}  // namespace epg
