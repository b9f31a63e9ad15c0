// Eviction by accumulated attention weight (sm_103a): adding a call's weights
// to the sums of each request, and choosing the tokens that a request keeps.
//
// Choosing is a selection of the k largest of n weights, not a sort: weights
// map to unsigned keys that order like them, three counts over the keys (by 11,
// 11 and 10 bits, most significant first) find the k-th largest key, and one
// ordered pass writes the positions above it plus the first ties.  A CTA
// counts into its shared memory; for long sequences a thread-block cluster
// serves a request and its CTAs read each other's counts over distributed
// shared memory.  A thread keeps its keys in registers from the first pass
// on (sequences up to 131072), so the weights are read once.  The kernel is
// bound by the latency of its passes and barriers, not by the 4 * n bytes:
// 7.4 us for one sequence of 1000, 8.5 for 64 of 4096 (1 MB); 17.8 for 8 of
// 131072 (4 MB) in clusters of 8, of which reading each other's counts is 5
// (6.6 with 32-bit counts, 64 KB a CTA and pass).
#include <cooperative_groups.h>

#include "hs_kv.cuh"

namespace hs {
namespace {

namespace cg = cooperative_groups;

constexpr int kEvictThreads = 1024;
constexpr int kEvictWarps = kEvictThreads / 32;
constexpr int kAhead = 4;                        // CTAs whose counts are read at a time
constexpr int kBins = 2048;
constexpr int kOwnBins = 2;                      // bins a thread looks through
static_assert(kOwnBins * kEvictThreads == kBins, "every bin has a thread");
constexpr int kChunk = 128;                      // positions a warp takes at a time, 4 a lane
constexpr int kMaxChunks = 4;                    // a warp holds in registers

// Key of a weight: larger weights have larger keys, NaN the smallest, the two
// zeros the same.
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);
    if (!(x == x)) return 0u;
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// The weight of a key (the NaN of key 0 and a zero come back without their sign bits).
__device__ __forceinline__ float weight_of(uint32_t key) {
    if (key == 0u) return __uint_as_float(0x7fc00000u);
    return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}

struct EvictArgs {
    const float* acc;
    const int32_t* req;
    const int32_t* seq_lens;
    int32_t recent, budget, R, L;
    int32_t* keep;
    int32_t* kept;
    float* kept_acc;
};

// CH: chunks of a warp's segment that are held in registers; 0: read anew in every pass.
template <int CH>
__global__ void __launch_bounds__(kEvictThreads) evict_kernel(const EvictArgs a) {
    __shared__ __align__(16) uint32_t s_hist[3][kBins];  // this CTA's counts, pass by pass
    // For the cluster: the counts of a thread's bins in one word, where the CTA's keys are few
    // enough (those in registers are).
    constexpr bool kPacked = CH > 0;
    static_assert(kMaxChunks * kChunk * kEvictWarps < 1 << 16, "a CTA's keys fit a count");
    __shared__ uint32_t s_pair[kPacked ? 3 : 1][kEvictThreads];
    __shared__ __align__(8) int s_cta[2];  // this CTA's keys above the edge, and equal to it
    __shared__ int s_tmp[33];
    __shared__ int s_pick[2];       // the chosen bin, and how many are wanted from it
    cg::cluster_group cluster = cg::this_cluster();
    const int P = (int)cluster.num_blocks();
    const int rank = (int)cluster.block_rank();
    const int b = blockIdx.x / P;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    wait_for_previous();
    release_next();
    const int q = ld(a.req + b);
    int n = ld(a.seq_lens + b);
    n = q < 0 || q >= a.R || n < 0 ? 0 : min(n, a.L);
    const float* acc = a.acc + (long long)(n > 0 ? q : 0) * a.L;
    int32_t* keep = a.keep + (long long)b * a.budget;
    float* kept_acc = a.kept_acc ? a.kept_acc + (long long)b * a.budget : nullptr;
    const int kept = min(n, a.budget);
    const int gid = rank * kEvictThreads + tid, all = P * kEvictThreads;
    if (gid == 0) a.kept[b] = kept;
    for (int j = kept + gid; j < a.budget; j += all) {
        keep[j] = -1;
        if (kept_acc) kept_acc[j] = 0.f;
    }
    if (n <= a.budget) {  // the same for the whole cluster
        for (int j = gid; j < n; j += all) {
            keep[j] = j;
            if (kept_acc) kept_acc[j] = acc[j];
        }
        return;
    }
    const int m = n - a.recent;           // candidates
    const int k = a.budget - a.recent;    // to keep of them, k < m
    if (k > 0) {
        // The warp's segment, in chunks of 128 positions, 4 consecutive ones a lane.
        const int chunks = ((m + kChunk - 1) / kChunk + P * kEvictWarps - 1) / (P * kEvictWarps);
        const int lo = (rank * kEvictWarps + warp) * chunks * kChunk;
        uint32_t x[CH > 0 ? CH : 1][4];
        // Past the last candidate the key is 0, the smallest, and the position behind those of all
        // candidates: such a key is never among the k kept, so the passes need not tell.
        auto fetch = [&](int c, uint32_t (&v)[4]) {
            const int t = lo + c * kChunk + lane * 4;
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = t + i < m ? key_of(ld(acc + t + i)) : 0u;
        };
        // Calls f(chunk, its 4 keys) for the warp's chunks in order.
        auto each = [&](auto f) {
            if constexpr (CH > 0) {
#pragma unroll
                for (int c = 0; c < CH; ++c)
                    if (c < chunks) f(c, x[c]);
            } else {
                for (int c = 0; c < chunks; ++c) {
                    fetch(c, x[0]);
                    f(c, x[0]);
                }
            }
        };
        if constexpr (CH > 0) {
#pragma unroll
            for (int c = 0; c < CH; ++c)
                if (c < chunks) fetch(c, x[c]);
        }
        for (int i = tid; i < 3 * kBins; i += kEvictThreads) (&s_hist[0][0])[i] = 0;
        __syncthreads();

        // The k-th largest key digit by digit.
        uint32_t edge = 0;   // the digits found so far; at the end, the key
        int want = k;        // how many of the keys with those digits are kept
#pragma unroll 1
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
            const int bins = pass == 2 ? 1024 : 2048;
            uint32_t* hist = s_hist[pass];
            each([&](int, const uint32_t (&v)[4]) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (pass == 0 || v[i] >> (pass == 1 ? 21 : 10) == edge)
                        atomicAdd(&hist[v[i] >> shift & (bins - 1)], 1u);
            });
            // A thread's bins, counted from the top, over the cluster.
            const int top = kBins - (tid + 1) * kOwnBins;
            if (kPacked && P > 1) {
                __syncthreads();
                s_pair[pass][tid] = hist[top] | hist[top + 1] << 16;
            }
            cluster.sync();
            int mine[kOwnBins] = {};
#pragma unroll 1
            for (int r0 = 0; r0 < P; r0 += kAhead) {
                uint2 h[kAhead];  // on their way together: a remote load takes long
#pragma unroll
                for (int r = 0; r < kAhead; ++r) {
                    h[r] = make_uint2(0, 0);
                    if (r0 + r >= P) continue;
                    if (kPacked && P > 1) {
                        h[r].x = cluster.map_shared_rank(s_pair[pass], r0 + r)[tid];
                        h[r].y = h[r].x >> 16, h[r].x &= 0xffff;
                    } else {
                        h[r] = *reinterpret_cast<const uint2*>(
                            cluster.map_shared_rank(hist, r0 + r) + top);
                    }
                }
#pragma unroll
                for (int r = 0; r < kAhead; ++r) mine[0] += h[r].y, mine[1] += h[r].x;
            }
            int all_keys;
            int above =
                block_exclusive_scan(mine[0] + mine[1], s_tmp, &all_keys);
#pragma unroll
            for (int i = 0; i < kOwnBins; ++i) {
                if (above < want && want <= above + mine[i]) {
                    s_pick[0] = top + kOwnBins - 1 - i;
                    s_pick[1] = want - above;
                }
                above += mine[i];
            }
            __syncthreads();
            const int pick = s_pick[0];
            want = s_pick[1];
            edge = (edge << (pass == 2 ? 10 : 11)) | (uint32_t)pick;
        }

        // The warps' counts, then the positions in order.
        int na = 0, ne = 0;
        each([&](int, const uint32_t (&v)[4]) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                na += v[i] > edge;
                ne += v[i] == edge;
            }
        });
        na = __reduce_add_sync(0xffffffffu, na);
        ne = __reduce_add_sync(0xffffffffu, ne);
        int wa, we, ta, te;  // before this warp in the CTA, and in all of it
        if constexpr (kPacked) {
            wa = block_exclusive_scan(lane == 0 ? na | ne << 16 : 0, s_tmp, &ta);
            we = wa >> 16, wa &= 0xffff;
            te = ta >> 16, ta &= 0xffff;
        } else {
            wa = block_exclusive_scan(lane == 0 ? na : 0, s_tmp, &ta);
            we = block_exclusive_scan(lane == 0 ? ne : 0, s_tmp, &te);
        }
        int out = 0, ties = 0;  // kept, and equal to the edge, before this CTA's positions
        if (P > 1) {
            if (tid == 0) s_cta[0] = ta, s_cta[1] = te;
            cluster.sync();
            if (lane < rank) {
                const int2 h = *reinterpret_cast<const int2*>(cluster.map_shared_rank(s_cta, lane));
                out = h.x, ties = h.y;
            }
            out = __reduce_add_sync(0xffffffffu, out);
            ties = __reduce_add_sync(0xffffffffu, ties);
            out += min(ties, want);  // the first `want` keys equal to the edge are kept
        }
        int tie = ties + __shfl_sync(0xffffffffu, we, 0);
        int at = out + __shfl_sync(0xffffffffu, wa, 0) + min(tie, want) - min(ties, want);
        each([&](int c, const uint32_t (&v)[4]) {
            const int t = lo + c * kChunk + lane * 4;
            int both = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) both += (v[i] > edge) + ((v[i] == edge) << 16);
            const int scan = warp_inclusive_scan(both);
            int e = tie + ((scan - both) >> 16);
            int w = at + ((scan - both) & 0xffff) + min(e, want) - min(tie, want);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const bool eq = v[i] == edge;
                if (v[i] > edge || (eq && e < want)) {
                    keep[w] = t + i;
                    if (kept_acc) kept_acc[w] = weight_of(v[i]);
                    ++w;
                }
                e += eq;
            }
            const int last = __shfl_sync(0xffffffffu, scan, 31);
            const int after = tie + (last >> 16);
            at += (last & 0xffff) + min(after, want) - min(tie, want);
            tie = after;
        });
    }
    for (int j = gid; j < a.recent; j += all) {
        keep[k + j] = m + j;
        if (kept_acc) kept_acc[k + j] = acc[m + j];
    }
    if (k > 0) cluster.sync();  // no CTA leaves while another reads its counts
}

// A cluster of up to 4 CTAs per request (additions to scattered words leave an SM one at a time, so
// they are spread as long as all CTAs are resident); the steps follow one another, a cluster barrier
// between them ordering the additions, so that a token selected in several steps is added to in step
// order.  Up to kHeldSteps steps of kHeldEntries entries a thread are fetched before the first
// addition, the positions even before hs_attend's kernel has ended.  Four steps of 2048 entries with
// clusters of 1, 2, 4 and 8: 8.5, 6.4, 5.0 and 5.0 us for 8 requests, 9.1, 6.7, 6.8 and 11.7 for 64;
// of 512 entries for 256 requests 6.6, 10.3, 16.1 and 27.4.  Entries fetched step by step instead:
// 5.4 us for the 8 requests, 7.6 for the 64.
constexpr int kAccumulateThreads = 512;
constexpr int kHeldSteps = 4, kHeldEntries = 4;

template <int P>
__global__ void __launch_bounds__(kAccumulateThreads)
    accumulate_kernel(const float* weights, const int32_t* topk, const int32_t* req,
                      const int32_t* counts, int32_t S, int32_t K, float* acc, int32_t R,
                      int32_t L, bool after_attend) {
    cg::cluster_group cluster = cg::this_cluster();
    constexpr int all = kAccumulateThreads * P;
    const int b = blockIdx.x / P;
    const int first = (int)cluster.block_rank() * kAccumulateThreads + threadIdx.x;
    // Behind hs_attend's own kernel the positions, which that one has read, may be read before its
    // end; any other kernel before this one may still be writing them.
    if (!after_attend) wait_for_previous();
    const int q = ld(req + b);
    const int steps = q < 0 || q >= R ? 0 : counts ? min(ld(counts + b), S) : S;
    float* dst = acc + (long long)(steps > 0 ? q : 0) * L;
    const long long row = (long long)b * S * K;
    if (K <= kHeldEntries * all && steps <= kHeldSteps) {
        int t[kHeldSteps][kHeldEntries];
        float w[kHeldSteps][kHeldEntries];
#pragma unroll
        for (int s = 0; s < kHeldSteps; ++s)
#pragma unroll
            for (int i = 0; i < kHeldEntries; ++i)
                t[s][i] = s < steps && first + i * all < K
                              ? ld(topk + row + s * K + first + i * all)
                              : -1;
        if (after_attend) wait_for_previous();  // for the weights
#pragma unroll
        for (int s = 0; s < kHeldSteps; ++s)
#pragma unroll
            for (int i = 0; i < kHeldEntries; ++i) {
                if (t[s][i] >= L) t[s][i] = -1;
                w[s][i] = t[s][i] >= 0 ? ld(weights + row + s * K + first + i * all) : 0.f;
            }
#pragma unroll
        for (int s = 0; s < kHeldSteps; ++s) {
            if (s >= steps) break;
            if (s > 0) cluster.sync();
#pragma unroll
            for (int i = 0; i < kHeldEntries; ++i)
                if (t[s][i] >= 0) atomicAdd(dst + t[s][i], w[s][i]);
        }
        return;
    }
    if (after_attend) wait_for_previous();
    for (int s = 0; s < steps; ++s) {
        if (s > 0) cluster.sync();
#pragma unroll 4
        for (int j = first; j < K; j += all) {
            const int t = ld(topk + row + (long long)s * K + j);
            if (t >= 0 && t < L) atomicAdd(dst + t, ld(weights + row + (long long)s * K + j));
        }
    }
}

}  // namespace

cudaError_t launch_accumulate(const float* weights, const int32_t* topk, const int32_t* req,
                              const int32_t* counts, int32_t B, int32_t S, int32_t K, float* acc,
                              int32_t R, int32_t L, bool after_attend, cudaStream_t s) {
    constexpr int kRound = 2 * 152;  // two CTAs an SM
    const int P = B <= kRound / 4 ? 4 : (B <= kRound / 2 ? 2 : 1);
    return launch_chained(P == 4   ? accumulate_kernel<4>
                          : P == 2 ? accumulate_kernel<2>
                                   : accumulate_kernel<1>,
                          B * P, kAccumulateThreads, 0, P, s, weights, topk, req, counts, S, K, acc, R,
                          L, after_attend);
}

cudaError_t launch_evict(const float* acc, const int32_t* req, const int32_t* seq_lens, int32_t B,
                         int32_t recent, int32_t budget, int32_t R, int32_t L, int32_t* keep,
                         int32_t* kept, float* kept_acc, cudaStream_t s) {
    EvictArgs a;
    a.acc = acc;
    a.req = req;
    a.seq_lens = seq_lens;
    a.recent = recent;
    a.budget = budget;
    a.R = R;
    a.L = L;
    a.keep = keep;
    a.kept = kept;
    a.kept_acc = kept_acc;
    // Cluster size of the least estimate, in us: what a CTA of a cluster of 1, 2, 4 or 8 takes for few
    // keys, 0.37 for every 1024 of its keys (0.70, and 1.4 to start, if they are read anew in every
    // pass), times the rounds of a GB300's SMs.  Measured with 1, 2, 4 and 8: one request of 8192, 9.3,
    // 8.6, 9.8 and 12.8 us; 8 of 16384, 13.2, 10.6, 10.1 and 13.2; 64 of 16384, 13.3, 10.8, 20.3 and
    // 64; 64 of 131072, keys held by 8, 55 with 2, 70 with 4 and 94 with 8.
    constexpr int kHeld = kMaxChunks * kChunk * kEvictWarps;  // keys a CTA holds in registers
    constexpr struct { int size, resident; double start; } kClusters[] = {
        {1, 152, 7.0}, {2, 152, 8.0}, {4, 144, 9.2}, {8, 120, 12.4}};
    int P = 1;
    double least = 0;
    for (const auto& c : kClusters) {
        const double keys = (double)L / c.size, rounds = (B * (long long)c.size - 1) / c.resident + 1;
        const double t = rounds * (keys <= kHeld ? c.start + 0.37 / 1024 * keys
                                                 : c.start + 1.4 + 0.70 / 1024 * keys);
        if (c.size == 1 || t < least) least = t, P = c.size;
    }
    const long long chunks = ((long long)L + kChunk - 1) / kChunk;
    const int per_warp = (int)((chunks + P * kEvictWarps - 1) / (P * kEvictWarps));
    auto* kernel = per_warp <= 1            ? evict_kernel<1>
                   : per_warp <= 2          ? evict_kernel<2>
                   : per_warp <= kMaxChunks ? evict_kernel<kMaxChunks>
                                            : evict_kernel<0>;
    return launch_chained(kernel, B * P, kEvictThreads, 0, P, s, a);
}

}  // namespace hs
