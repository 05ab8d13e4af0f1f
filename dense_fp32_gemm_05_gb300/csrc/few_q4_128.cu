// The kernels for 4-bit weights in groups of 128, for products of few rows; and what the kernels of
// every type share of the GPU.
#include <atomic>

#include "few_kernel.cuh"

namespace sgemm_gb300 {

template <>
int launch_few<128>(const FewLaunch &l, cudaStream_t s) {
    return l.p.z[0] ? launch_tiles<128, true>(l, s) : launch_tiles<128, false>(l, s);
}

// A CTA has the most shared memory that a plan gives it; registers are as all kernels of so
// many tiles have them (two CTAs an SM, or one).
int few_clusters(int dev, int nt, int ks) {
    static std::atomic<int> known[64][2][9];       // one more than the answer
    const int wide = nt > 2;
    std::atomic<int> *at = dev < 64 && ks <= 8 ? &known[dev][wide][ks] : nullptr;
    if (at && at->load(std::memory_order_relaxed)) return at->load(std::memory_order_relaxed) - 1;
    const auto kern = wide ? few::few_kernel<128, false, 4> : few::few_kernel<128, false, 1>;
    const size_t smem = 1024 + (size_t)few_most_smem(nt);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)ks);
    cfg.blockDim = dim3((unsigned)few::THREADS);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)ks;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 225 * 1024) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    if (at) at->store(n + 1, std::memory_order_relaxed);
    return n;
}

}  // namespace sgemm_gb300
