// The kernels for bf16 weights of the products of few rows.
#include "few_kernel.cuh"

namespace sgemm_gb300 {

template <>
int launch_few<0>(int nt, const few::Params &p, int grid_x, int grid_y, int smem, cudaStream_t s, bool dep) {
    return launch_tiles<0, false>(nt, p, grid_x, grid_y, smem, s, dep);
}

}  // namespace sgemm_gb300
