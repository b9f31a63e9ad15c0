// Shared by the calls that a decode step makes around the swap-in: norms and rotation of
// new queries and keys, bounds on blocks of keys and the selection by them, and
// attention over a shared prefix.  Contracts and layouts are in include/hisparse_swap.h.
#pragma once

#include "hs_kv.cuh"

namespace hs {

// Launchers (each returns the launch's error code).
cudaError_t launch_norm_rope(const hs_norm_rope_args& a, cudaStream_t s);

struct BoundArgs {
    const uint8_t* k;  // 16-bit elements
    int64_t stride[3];
    int32_t fp16, Hkv, D, T, batch, max_count, R, L, NB;
    const int32_t* req;
    const int32_t* start;
    const int32_t* count;
    uint8_t* bounds;
    int32_t windows;  // blocks that max_count tokens can touch
    int32_t slabs;    // of 256 channels of a token
    int32_t vec_k, vec_bounds;
};
cudaError_t launch_bound(BoundArgs a, cudaStream_t s);

// CTAs that score one batch entry's blocks, and the blocks of each: kSelectChunk or more, which bounds the
// workspace.
constexpr int kSelectChunk = 8;
struct SelectShape {
    int chunks, blocks;
};
SelectShape select_shape(int32_t batch, int32_t steps, int32_t row, int32_t NB);
cudaError_t launch_select(const hs_select_args& a, cudaStream_t s);

// Rows of queries that a pipeline of the prefix kernel takes at a time, and tokens of a tile.
constexpr int kPrefixRows = 128;
constexpr int kPrefixTokens = 64;
size_t prefix_workspace(const hs_kv_format& f);
cudaError_t launch_prefix(const hs_kv_format& f, const hs_prefix_args& a, cudaStream_t s);

}  // namespace hs
