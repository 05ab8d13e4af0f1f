// The kernels for bf16 weights, for products of few rows.
#include "few_kernel.cuh"

namespace sgemm_gb300 {

template <>
int launch_few<0>(const FewLaunch &l, cudaStream_t s) {
    return launch_tiles<0, false>(l, s);
}

}  // namespace sgemm_gb300
