// The experts' products with 4-bit weights, compiled for int4 codes around 8.
#include "experts_w4_kernel.cuh"

namespace epg {
namespace w4 {

cudaError_t launch_int(const Args& a, int group, Which which, dim3 grid, size_t smem, cudaStream_t stream) {
    return launch_form<EP_W4_INT>(a, group, which, grid, smem, stream);
}

}  // namespace w4
}  // namespace epg
