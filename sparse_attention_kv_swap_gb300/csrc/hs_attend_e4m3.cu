// hs_attend over e4m3 codes (one translation unit per code: they compile in parallel).
#include "hs_attend.cuh"

namespace hs {

cudaError_t attend_run_e4m3(const AttendShape& sh, int D, cudaStream_t s) {
    return attend::run<HS_KV_E4M3>(sh, D, s);
}

int attend_resident(int P, size_t smem) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(P);
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = P;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int clusters = 0;
    if (attend::open_kernel<HS_KV_E4M3, 128, 1, false>(P, smem) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&clusters, attend::attend_kernel<HS_KV_E4M3, 128, 1, false>,
                                       &cfg) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    return clusters * P;
}

}  // namespace hs
