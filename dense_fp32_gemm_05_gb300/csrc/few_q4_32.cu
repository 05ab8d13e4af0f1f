// The kernels for 4-bit weights in groups of 32 of the products of few rows.
#include "few_kernel.cuh"

namespace sgemm_gb300 {

template <>
int launch_few<32>(int nt, const few::Params &p, int grid_x, int grid_y, int smem, cudaStream_t s, bool dep) {
    return p.z[0] ? launch_tiles<32, true>(nt, p, grid_x, grid_y, smem, s, dep)
                  : launch_tiles<32, false>(nt, p, grid_x, grid_y, smem, s, dep);
}

}  // namespace sgemm_gb300
