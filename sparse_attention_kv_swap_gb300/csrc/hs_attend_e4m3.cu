// hs_attend over e4m3 codes (one translation unit per code: they compile in parallel).
#include "hs_attend.cuh"

namespace hs {

cudaError_t attend_run_e4m3(const AttendShape& sh, int D, cudaStream_t s) {
    return attend::run<HS_KV_E4M3>(sh, D, s);
}

int attend_resident(int P, size_t smem) {
    auto* kernel = attend::attend_kernel<HS_KV_E4M3, 128, 1, false>;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    int clusters = 0;
    if (attend::configure<HS_KV_E4M3, 128, 1, false>(P, 1, 256, smem, nullptr, &cfg, attr) !=
            cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    return clusters * P;
}

}  // namespace hs
