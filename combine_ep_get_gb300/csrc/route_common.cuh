// Device helpers of the router's kernels: a warp holds one token's row of
// logits, expert j * 32 + lane in element j.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "experts.cuh"   // exp2_approx, reciprocal_approx
#include "route.cuh"

namespace epg {

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
__device__ __forceinline__ void from_float(float* p, float v) { *p = v; }
__device__ __forceinline__ void from_float(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void from_float(__half* p, float v) { *p = __float2half_rn(v); }

constexpr float kInf = __builtin_huge_valf();

// A row's logits; -inf behind the last expert.  kFull: there are 32 kPer experts.
template <int kPer, bool kFull = false, typename L>
__device__ __forceinline__ void load_row(const L* row, int E, int lane, float (&v)[kPer]) {
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int e = j * 32 + lane;
        v[j] = kFull || e < E ? to_float(row[e]) : -kInf;
    }
}

// The largest value of a warp, NaN aside.
__device__ __forceinline__ float warp_max(float v) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Two sums at once: a sum's five exchanges wait for one another.
__device__ __forceinline__ void warp_sums(float& a, float& b) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float x = __shfl_xor_sync(0xffffffffu, a, o), y = __shfl_xor_sync(0xffffffffu, b, o);
        a += x;
        b += y;
    }
}

// sigmoid(l) exp(-shift), shift <= 0: with the largest logit of a sum as shift
// where that is far below zero, so that ratios of sigmoids stay exact where the
// sigmoids themselves would be subnormal or zero.
__device__ __forceinline__ float sigmoid_shifted(float l, float shift) {
    const float e = expf(-fabsf(l));
    const float top = l < 0.0f ? (shift == 0.0f ? e : expf(l - shift)) : 1.0f;
    return top / (1.0f + e);
}
__device__ __forceinline__ float shift_of(float largest) { return largest < -16.0f ? largest : 0.0f; }

// The same as the hardware's 2^x and 1/x give it, without a shift: (sigmoid(l), 1 - sigmoid(l)), each good to 4e-7 of
// itself and 2^-24 |l|, what l's own last place moves it by.
__device__ __forceinline__ float sigmoid_fast(float l, float* rest) {
    const float e = exp2_approx(-kLog2E * fabsf(l)), r = reciprocal_approx(1.0f + e), small = e * r;
    *rest = l < 0.0f ? r : small;
    return l < 0.0f ? small : r;
}

// Sequence of token t: the last q with offset[q] <= t, -1 or S for tokens
// before the first or behind the last one.
__device__ __forceinline__ int sequence_of(const int32_t* offset, int S, int t) {
    if (!offset) return 0;
    int lo = -1, hi = S;     // offset[lo] <= t (or lo = -1), offset[hi + 1] > t (or hi = S)
    while (lo < hi) {
        const int mid = lo + (hi - lo + 1) / 2;
        if (offset[mid] <= t)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// The same by a warp, all lanes alike.
__device__ __forceinline__ int warp_sequence_of(const int32_t* offset, int S, int t, int lane) {
    if (!offset) return 0;
    if (S >= 32) return sequence_of(offset, S, t);
    return __popc(__ballot_sync(0xffffffffu, lane <= S && offset[lane <= S ? lane : S] <= t)) - 1;
}

// Calls f with the type of the logits, the elements of a row in a lane, and whether a row fills them.
template <typename F>
cudaError_t with_row_type(int dtype, int E, F f) {
    const auto sized = [&](auto* type) {
        const auto full = [&](auto per) {
            return E == 32 * decltype(per)::value ? f(type, per, std::true_type()) : f(type, per, std::false_type());
        };
        if (E <= 32) return full(std::integral_constant<int, 1>());
        if (E <= 64) return full(std::integral_constant<int, 2>());
        if (E <= 128) return full(std::integral_constant<int, 4>());
        if (E <= 256) return full(std::integral_constant<int, 8>());
        if (E <= 512) return f(type, std::integral_constant<int, 16>(), std::false_type());
        if (E <= 1024) return f(type, std::integral_constant<int, 32>(), std::false_type());
        return f(type, std::integral_constant<int, 64>(), std::false_type());
    };
    if (dtype == EP_FP32) return sized(static_cast<const float*>(nullptr));
    if (dtype == EP_FP16) return sized(static_cast<const __half*>(nullptr));
    return sized(static_cast<const __nv_bfloat16*>(nullptr));
}

}  // namespace epg
