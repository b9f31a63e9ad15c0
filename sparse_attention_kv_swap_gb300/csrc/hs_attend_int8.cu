// hs_attend over int8 codes (one translation unit per code: they compile in parallel).
#include "hs_attend.cuh"

namespace hs {

cudaError_t attend_run_int8(const AttendShape& sh, int D, cudaStream_t s) {
    return attend::run<HS_KV_INT8>(sh, D, s);
}

}  // namespace hs
