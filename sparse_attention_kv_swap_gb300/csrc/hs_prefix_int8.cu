// hs_attend_prefix over int8 codes (one translation unit per code: they compile in parallel).
#include "hs_prefix.cuh"

namespace hs {

cudaError_t prefix_run_int8(const PrefixArgs& a, const CUtensorMap& map, int D, cudaStream_t s) {
    return prefix::run<HS_KV_INT8>(a, map, D, s);
}

}  // namespace hs
