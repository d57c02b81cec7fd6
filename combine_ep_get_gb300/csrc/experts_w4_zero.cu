// The experts' products with 4-bit weights, compiled for int4 codes with zero points.
#include "experts_w4_kernel.cuh"

namespace epg {
namespace w4 {

cudaError_t launch_zero(const Args& a, int group, Which which, dim3 grid, size_t smem, cudaStream_t stream) {
    return launch_form<kIntZero>(a, group, which, grid, smem, stream);
}

}  // namespace w4
}  // namespace epg
