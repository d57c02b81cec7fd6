// The experts' products with 4-bit weights, compiled for E2M1 codes.
#include "experts_w4_kernel.cuh"

namespace epg {
namespace w4 {

cudaError_t launch_fp(const Args& a, int group, Which which, dim3 grid, size_t smem, cudaStream_t stream) {
    return launch_form<EP_W4_FP>(a, group, which, grid, smem, stream);
}

}  // namespace w4
}  // namespace epg
