// hs_attend_prefix over e4m3 codes (one translation unit per code: they compile in parallel).
#include "hs_prefix.cuh"

namespace hs {

cudaError_t prefix_run_e4m3(const PrefixArgs& a, const CUtensorMap& map, int D, cudaStream_t s) {
    return prefix::run<HS_KV_E4M3>(a, map, D, s);
}

}  // namespace hs
