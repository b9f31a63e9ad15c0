// hs_attend over e4m3 codes (one translation unit per code: they compile in parallel).
#include "hs_attend.cuh"

namespace hs {

cudaError_t attend_run_e4m3(const AttendShape& sh, int D, cudaStream_t s) {
    return attend::run<HS_KV_E4M3>(sh, D, s);
}

}  // namespace hs
