// The kernels for bf16 weights, for products of few rows.
#include "few_kernel.cuh"

namespace sgemm_gb300 {

// (a block's few tokens, 16 at most, are one or two tiles of columns)
template <>
int launch_few<0>(const FewLaunch &l, cudaStream_t s) {
    return l.nt == 1 ? launch_kernel<0, false, 1>(l, s) : l.nt == 2 ? launch_kernel<0, false, 2>(l, s) : SGEMM_ERR_UNSUPPORTED;
}

}  // namespace sgemm_gb300
