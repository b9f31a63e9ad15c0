// Eviction by accumulated attention weight (sm_103a): adding a call's weights
// to the sums of each request, and choosing the tokens that a request keeps.
//
// Choosing is a selection of the k largest of n weights, not a sort: weights
// map to unsigned keys that order like them, three passes over the keys (11,
// 11 and 10 bits, most significant first) find the k-th largest key by
// counting, and one ordered pass writes the positions above it plus the first
// ties.  One thread-block cluster serves a request: each CTA counts its
// segment into its own shared memory, the counts are added over distributed
// shared memory, and the passes re-read the weights from L2 (4 bytes a token).
// The kernel is bound by the latency of its passes and barriers, not by the
// 4 * n bytes it reads.
#include <cooperative_groups.h>

#include "hs_kv.cuh"

namespace hs {
namespace {

namespace cg = cooperative_groups;

constexpr int kEvictThreads = 512;
constexpr int kMaxEvictCluster = 8;
constexpr int kBins = 2048;
constexpr int kPer = 4;  // consecutive positions of a thread in the ordered pass

// Key of a weight: larger weights have larger keys, NaN the smallest, the two
// zeros the same.
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);
    if (!(x == x)) return 0u;
    return u & 0x80000000u ? ~u : u | 0x80000000u;
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

__global__ void __launch_bounds__(kEvictThreads) evict_kernel(const EvictArgs a) {
    __shared__ int s_hist[kBins];   // this CTA's counts
    __shared__ int s_sum[kBins];    // the cluster's counts of this CTA's share of the bins
    __shared__ int s_tmp[33];
    __shared__ int s_pick[2];       // the chosen bin, and how many are wanted from it
    __shared__ int s_above, s_equal;
    cg::cluster_group cluster = cg::this_cluster();
    const int P = (int)cluster.num_blocks();
    const int rank = (int)cluster.block_rank();
    const int b = blockIdx.x / P;
    const int tid = threadIdx.x;
    const int q = __ldg(a.req + b);
    int n = __ldg(a.seq_lens + b);
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
    for (int j = gid; j < a.recent; j += all) {
        keep[k + j] = m + j;
        if (kept_acc) kept_acc[k + j] = acc[m + j];
    }
    if (k == 0) return;

    // This CTA's segment, and the k-th largest key digit by digit.
    const int seg = (m + P - 1) / P;
    const int lo = min(m, rank * seg), hi = min(m, lo + seg);
    uint32_t prefix = 0;  // the digits found so far
    int want = k;         // how many of the keys with that prefix are kept
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
        const int bins = pass == 2 ? 1024 : 2048;
        for (int i = tid; i < kBins; i += kEvictThreads) s_hist[i] = 0;
        __syncthreads();
        for (int i = lo + tid; i < hi; i += kEvictThreads) {
            const uint32_t key = key_of(__ldg(acc + i));
            const bool in = pass == 0 || key >> (pass == 1 ? 21 : 10) == prefix;
            if (in) atomicAdd(&s_hist[key >> shift & (bins - 1)], 1);
        }
        cluster.sync();
        if (P > 1) {
            const int share = kBins / P;
            for (int i = tid; i < share; i += kEvictThreads) {
                int sum = 0;
                for (int r = 0; r < P; ++r)
                    sum += cluster.map_shared_rank(s_hist, r)[rank * share + i];
                s_sum[i] = sum;
            }
            cluster.sync();
        }
        // Suffix counts: thread t owns the bins 4 t .. 4 t + 3 counted from the top.
        int mine[kBins / kEvictThreads], total = 0;
#pragma unroll
        for (int i = 0; i < kBins / kEvictThreads; ++i) {
            const int bin = kBins - 1 - (tid * (kBins / kEvictThreads) + i);
            mine[i] = P > 1 ? cluster.map_shared_rank(s_sum, bin / (kBins / P))[bin % (kBins / P)]
                            : s_hist[bin];
            total += mine[i];
        }
        int sum_all;
        int before = block_exclusive_scan(total, s_tmp, &sum_all);
#pragma unroll
        for (int i = 0; i < kBins / kEvictThreads; ++i) {
            if (before < want && want <= before + mine[i]) {
                s_pick[0] = kBins - 1 - (tid * (kBins / kEvictThreads) + i);
                s_pick[1] = want - before;
            }
            before += mine[i];
        }
        __syncthreads();
        prefix = (prefix << (pass == 2 ? 10 : 11)) | (uint32_t)s_pick[0];
        want = s_pick[1];
        cluster.sync();  // every CTA has read the counts before they are cleared again
    }
    // prefix is the k-th largest key; `want` of the keys equal to it are kept, lowest first.
    const uint32_t edge = prefix;
    int above = 0, equal = 0;
    for (int i = lo + tid; i < hi; i += kEvictThreads) {
        const uint32_t key = key_of(__ldg(acc + i));
        above += key > edge;
        equal += key == edge;
    }
    above = block_sum(above, s_tmp);
    equal = block_sum(equal, s_tmp);
    if (tid == 0) {
        s_above = above;
        s_equal = equal;
    }
    cluster.sync();
    int out = 0, ties = 0;  // written and ties seen before this CTA's segment
    for (int r = 0; r < rank; ++r) {
        const int e = *cluster.map_shared_rank(&s_equal, r);
        out += *cluster.map_shared_rank(&s_above, r) + max(0, min(e, want - ties));
        ties += e;
    }
    cluster.sync();  // the other CTAs' shared memory is not read after this
    for (int base = lo; base < hi; base += kEvictThreads * kPer) {
        float x[kPer];
        uint32_t key[kPer];
        int na = 0, ne = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int t = base + tid * kPer + i;
            x[i] = t < hi ? __ldg(acc + t) : 0.f;
            key[i] = key_of(x[i]);
            na += t < hi && key[i] > edge;
            ne += t < hi && key[i] == edge;
        }
        int both;
        const int scan = block_exclusive_scan(na | ne << 16, s_tmp, &both);
        int tie = ties + (scan >> 16);
        // entries of this chunk before this thread: those above, and the ties still wanted
        int at = out + (scan & 0xffff) + max(0, min(tie, want) - min(ties, want));
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int t = base + tid * kPer + i;
            if (t >= hi) break;
            const bool eq = key[i] == edge;
            if (key[i] > edge || (eq && tie < want)) {
                keep[at] = t;
                if (kept_acc) kept_acc[at] = x[i];
                ++at;
            }
            tie += eq;
        }
        const int t1 = ties + (both >> 16);
        out += (both & 0xffff) + max(0, min(t1, want) - min(ties, want));
        ties = t1;
    }
}

// One CTA per request; the steps follow one another, so that a token selected
// in several steps is added to in step order.
constexpr int kAccumulateThreads = 1024;

__global__ void __launch_bounds__(kAccumulateThreads)
    accumulate_kernel(const float* weights, const int32_t* topk, const int32_t* req,
                      const int32_t* counts, int32_t S, int32_t K, float* acc, int32_t R,
                      int32_t L) {
    const int b = blockIdx.x;
    const int q = __ldg(req + b);
    if (q < 0 || q >= R) return;
    const int steps = counts ? min(__ldg(counts + b), S) : S;
    float* dst = acc + (long long)q * L;
    for (int s = 0; s < steps; ++s) {
        const long long row = ((long long)b * S + s) * K;
        for (int j = threadIdx.x; j < K; j += kAccumulateThreads) {
            const int t = __ldg(topk + row + j);
            if (t >= 0 && t < L) atomicAdd(dst + t, __ldg(weights + row + j));
        }
        __syncthreads();
    }
}

}  // namespace

cudaError_t launch_accumulate(const float* weights, const int32_t* topk, const int32_t* req,
                              const int32_t* counts, int32_t B, int32_t S, int32_t K, float* acc,
                              int32_t R, int32_t L, cudaStream_t s) {
    accumulate_kernel<<<B, kAccumulateThreads, 0, s>>>(weights, topk, req, counts, S, K, acc, R,
                                                       L);
    return cudaGetLastError();
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
    int P = 1;
    while (P < kMaxEvictCluster && L / P > 8192) P *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(B * P);
    cfg.blockDim = dim3(kEvictThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = P;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, evict_kernel, a);
}

}  // namespace hs
