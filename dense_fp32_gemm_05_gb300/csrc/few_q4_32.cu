// The kernels for 4-bit weights in groups of 32, for products of few rows.
#include "few_kernel.cuh"

namespace sgemm_gb300 {

template <>
int launch_few<32>(const FewLaunch &l, cudaStream_t s) {
    return l.p.z[0] ? launch_tiles<32, true>(l, s) : launch_tiles<32, false>(l, s);
}

}  // namespace sgemm_gb300
