// Selection of key blocks for decode queries by bounds on their scores (sm_103a).
//
// score(n) = sum over query heads and channels of max(q lo_n, q hi_n).  lo <= hi, so a positive
// q takes hi and a negative one lo, and the query heads of a K/V head add up first:
//   score(n) = sum over K/V heads and channels of Q+ hi_n + Q- lo_n,
//   Q+ = sum of max(q, 0), Q- = sum of min(q, 0),
// two multiply-adds for each pair of bounds, whatever the number of query heads: the bounds
// are read once and nothing else counts (4 bytes for 2 * steps operations: memory).
//
// The first kernel scores: a warp takes 256 elements (512 bytes) of up to 32 / steps blocks, each lane
// 8 of them, holds the sums of all in registers and adds them up over its lanes by halving exchanges (31
// shuffles for 32 sums).
//
// The second selects, one CTA a query.  Sums in 32 bits depend on their order and would swap blocks whose
// scores are close.  So the first kernel also bounds the error of its sums (a few 2^-24 of
// sum |Q| max_n |bound|, the maximum taken channel by channel), and where blocks that could
// belong on either side of the border are more than there is room for, these are scored again in
// twice 32 bits (error-free products and sums) and selected by that, ties to the lowest index.  The
// selection is then that of the scores themselves, for every launch shape.
#include "hs_step.cuh"

namespace hs {
namespace {

constexpr int kScoreWarps = 8;
constexpr int kSlice = 256;            // elements of a block that a warp takes at a time
constexpr int kMostSums = 1024;        // scores of a CTA: its blocks times the steps
constexpr int kSelectThreads = 512;
constexpr int kBins = 1024;

// Blocks of a warp's registers: 32 sums.
constexpr int batch_blocks(int S) { return S == 1 ? 32 : S == 2 ? 16 : S == 3 ? 10 : 8; }

struct ScoreArgs {
    const uint16_t* q;
    const uint16_t* bounds;
    const int32_t* req;
    const int32_t* seq_lens;
    float* scores;  // [B][S][NB]
    float* error;   // [B][chunks][S]
    int64_t q_stride[3];
    int32_t B, S, Hkv, G, D, R, L, T, NB, row;  // row: elements of a block's bounds
    int32_t chunks, blocks;  // CTAs of a batch entry, blocks of each
    int32_t wpr;             // warps that share a block
    int32_t vec_bounds;
    float gamma;
    // the selection's
    int32_t select, first, last;
    int32_t* out_blocks;
    int32_t* topk;
    Divisor by_T;
};

template <bool FP16>
__device__ __forceinline__ float value(uint16_t x) {
    if constexpr (FP16) return __half2float(__ushort_as_half(x));
    return __uint_as_float((uint32_t)x << 16);
}

template <bool FP16>
__device__ __forceinline__ float2 values(uint32_t w) {
    if constexpr (FP16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// Larger of the magnitudes, two elements at a time (a NaN does not count).
template <bool FP16>
__device__ __forceinline__ uint32_t greater_magnitude(uint32_t m, uint32_t w) {
    w &= 0x7fff7fffu;
    if constexpr (FP16) {
        const __half2 x = __hmax2(*reinterpret_cast<__half2*>(&m), *reinterpret_cast<__half2*>(&w));
        return *reinterpret_cast<const uint32_t*>(&x);
    } else {
        const __nv_bfloat162 x = __hmax2(*reinterpret_cast<__nv_bfloat162*>(&m),
                                         *reinterpret_cast<__nv_bfloat162*>(&w));
        return *reinterpret_cast<const uint32_t*>(&x);
    }
}

// A number of about 48 bits, the sum of two floats.
struct Two {
    float hi, lo;
    // Adds x: the rounding error of the sum goes to lo (exact sum of two floats by Knuth).
    __device__ __forceinline__ void add(float x) {
        const float s = __fadd_rn(hi, x), y = __fsub_rn(s, hi);
        lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(s, y)), __fsub_rn(x, y)));
        hi = s;
    }
    __device__ __forceinline__ void normalise() {
        const float s = __fadd_rn(hi, lo);
        lo = __fsub_rn(lo, __fsub_rn(s, hi));
        hi = s;
    }
};

// Q+ and Q- of column `col` (K/V head, channel) of one query, in twice 32 bits.
template <bool FP16>
__device__ __forceinline__ void query_sums(const ScoreArgs& a, const uint16_t* q, int col, Two& up,
                                           Two& down) {
    const int h = col / a.D, d = col - h * a.D;
    const uint16_t* p = q + (long long)h * a.G * a.q_stride[2] + d;
    up = down = Two{0.f, 0.f};
#pragma unroll 4
    for (int g = 0; g < a.G; ++g) {
        const float x = value<FP16>(ld(p + g * a.q_stride[2]));
        if (x < 0.f)
            down.add(x);
        else
            up.add(x);  // a NaN spoils the query's scores
    }
    up.normalise();
    down.normalise();
}

// The 256 elements of a block that a warp takes: 8 a lane.
__device__ __forceinline__ uint4 load_bounds(const uint16_t* p, bool vec, bool on) {
    if (!on) return make_uint4(0, 0, 0, 0);
    if (vec) return ld_once_v4(p);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = (uint32_t)ld(p + 2 * i) | (uint32_t)ld(p + 2 * i + 1) << 16;
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <bool FP16, int S>
__global__ void __launch_bounds__(32 * kScoreWarps) score_kernel(const ScoreArgs a) {
    constexpr int NB = batch_blocks(S);
    constexpr int kGroup = NB % 8 == 0 ? 8 : 5;  // blocks under way together
    extern __shared__ __align__(16) float s_q[];  // [S][row], then the warps' sums
    __shared__ float s_error[kScoreWarps][S];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int chunk = blockIdx.x % a.chunks, b = blockIdx.x / a.chunks;
    float* const s_sum = s_q + S * a.row;  // [wpr][blocks * S]
    wait_for_previous();
    const int r = ld(a.req + b);
    int n = ld(a.seq_lens + b);
    n = r < 0 || r >= a.R || n < 0 ? 0 : min(n, a.L);
    const int nb = (n + a.T - 1) / a.T;
    const int n0 = chunk * a.blocks, n1 = min(n0 + a.blocks, a.NB);
    const int live = max(0, min(n1, nb) - n0);  // blocks to score
    if (live > 0) {
        // Q- and Q+ of all columns, in the order of the bounds.
        const int columns = a.Hkv * a.D;
        for (int i = tid; i < S * columns; i += 32 * kScoreWarps) {
            const int s = i / columns, col = i - s * columns;
            const uint16_t* q = a.q + b * a.q_stride[0] + s * a.q_stride[1];
            Two up, down;
            query_sums<FP16>(a, q, col, up, down);
            const int h = col / a.D;
            float* to = s_q + s * a.row + col + h * a.D;
            to[0] = down.hi;
            to[a.D] = up.hi;
        }
    }
    __syncthreads();
    float worst[S] = {};
    if (live > 0) {
        const uint16_t* base = a.bounds + ((long long)r * a.NB + n0) * a.row;
        const int part = warp % a.wpr, turns = kScoreWarps / a.wpr;
        for (int j0 = warp / a.wpr * NB; j0 < live; j0 += turns * NB) {
            float acc[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) acc[i] = 0.f;
            float error[S] = {};
            for (int e0 = part * kSlice; e0 < a.row; e0 += a.wpr * kSlice) {
                const int e = e0 + lane * 8;
                const bool on = e < a.row;
                float q[S][8];
#pragma unroll
                for (int s = 0; s < S; ++s) {
                    float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
                    if (on) {
                        x = *reinterpret_cast<const float4*>(s_q + s * a.row + e);
                        y = *reinterpret_cast<const float4*>(s_q + s * a.row + e + 4);
                    }
                    q[s][0] = x.x, q[s][1] = x.y, q[s][2] = x.z, q[s][3] = x.w;
                    q[s][4] = y.x, q[s][5] = y.y, q[s][6] = y.z, q[s][7] = y.w;
                }
                uint32_t most[4] = {};
#pragma unroll
                for (int g0 = 0; g0 < NB; g0 += kGroup) {
                    if (j0 + g0 >= live) break;
                    uint4 x[kGroup];
#pragma unroll
                    for (int g = 0; g < kGroup; ++g)
                        x[g] = load_bounds(base + (long long)(j0 + g0 + g) * a.row + e, a.vec_bounds,
                                           on && j0 + g0 + g < live);
#pragma unroll
                    for (int g = 0; g < kGroup; ++g) {
                        const uint32_t w[4] = {x[g].x, x[g].y, x[g].z, x[g].w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            most[i] = greater_magnitude<FP16>(most[i], w[i]);
                            const float2 v = values<FP16>(w[i]);
#pragma unroll
                            for (int s = 0; s < S; ++s) {
                                float& z = acc[s * NB + g0 + g];
                                z = fmaf(q[s][2 * i], v.x, z);
                                z = fmaf(q[s][2 * i + 1], v.y, z);
                            }
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 m = values<FP16>(most[i]);
#pragma unroll
                    for (int s = 0; s < S; ++s)
                        error[s] += fabsf(q[s][2 * i]) * m.x + fabsf(q[s][2 * i + 1]) * m.y;
                }
            }
#pragma unroll
            for (int s = 0; s < S; ++s)  // no bound where there is an infinity
                worst[s] = fmaxf(worst[s], error[s] == error[s] ? error[s] : INFINITY);
            // Lane l gets the sum over the lanes of number l.
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                const bool up = lane & o;
#pragma unroll
                for (int i = 0; i < o; ++i) {
                    const float give = up ? acc[i] : acc[i + o];
                    const float keep = up ? acc[i + o] : acc[i];
                    acc[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
                }
            }
            const int s = lane / NB, j = j0 + lane - s * NB;
            if (s < S && j < live) s_sum[part * a.blocks * S + s * a.blocks + j] = acc[0];
        }
    }
#pragma unroll
    for (int s = 0; s < S; ++s) {
        float x = worst[s];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        if (lane == 0) s_error[warp][s] = x;
    }
    __syncthreads();
    release_next();
    for (int i = tid; i < S * (n1 - n0); i += 32 * kScoreWarps) {
        const int s = i / (n1 - n0), j = i - s * (n1 - n0);
        float x = -INFINITY;
        if (j < live) {
            x = s_sum[s * a.blocks + j];
            for (int p = 1; p < a.wpr; ++p) x += s_sum[(p * S + s) * a.blocks + j];
        }
        a.scores[((long long)b * S + s) * a.NB + n0 + j] = x;
    }
    if (tid < S) {
        float most = 0.f;
        for (int t = 0; t < kScoreWarps; t += a.wpr) {
            float x = 0.f;
            for (int p = 0; p < a.wpr; ++p) x += s_error[t + p][tid];
            most = fmaxf(most, x);
        }
        a.error[((long long)b * a.chunks + chunk) * S + tid] = most * a.gamma;
    }
}

// Key of a score: larger scores have larger keys, NaN the smallest, the two zeros the same.
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);
    if (!(x == x)) return 0u;
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float score_of(uint32_t key) {
    return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}

struct Edge {
    uint32_t key;  // the k-th largest key
    int want;      // keys equal to it that are among the k
};

// The k-th largest of keys[lo, hi), 1 <= k <= hi - lo.  All threads call it.
__device__ __forceinline__ Edge kth_largest(const uint32_t* keys, int lo, int hi, int k,
                                            uint32_t* hist, int* tmp, uint32_t* range, int* pick) {
    const int tid = threadIdx.x;
    // The keys' range first: scores share their top bits, and counting by these would bring all into
    // a few bins.
    uint32_t least = 0xffffffffu, most = 0u;
    for (int i = lo + tid; i < hi; i += kSelectThreads) {
        least = min(least, keys[i]);
        most = max(most, keys[i]);
    }
    if (tid == 0) range[0] = 0xffffffffu, range[1] = 0u;
    for (int i = tid; i < kBins; i += kSelectThreads) hist[i] = 0;
    __syncthreads();
    least = __reduce_min_sync(0xffffffffu, least);
    most = __reduce_max_sync(0xffffffffu, most);
    if ((tid & 31) == 0) {
        atomicMin(&range[0], least);
        atomicMax(&range[1], most);
    }
    __syncthreads();
    uint32_t base = range[0];
    const uint32_t span = range[1] - base;
    int shift = span < kBins ? 0 : 22 - __clz(span);  // span >> shift < kBins
    uint32_t width = span;  // keys base .. base + width are counted
    int want = k;
    while (true) {
        for (int i = lo + tid; i < hi; i += kSelectThreads) {
            const uint32_t x = keys[i] - base;
            if (keys[i] >= base && x <= width) atomicAdd(&hist[x >> shift], 1u);
        }
        __syncthreads();
        constexpr int kOwn = kBins / kSelectThreads;
        const int top = kBins - (tid + 1) * kOwn;
        int mine[kOwn], sum = 0, all;
#pragma unroll
        for (int i = 0; i < kOwn; ++i) sum += mine[i] = hist[top + kOwn - 1 - i];
        int above = block_exclusive_scan(sum, tmp, &all);
#pragma unroll
        for (int i = 0; i < kOwn; ++i) {
            if (above < want && want <= above + mine[i]) {
                pick[0] = top + kOwn - 1 - i;
                pick[1] = want - above;
            }
            above += mine[i];
        }
        for (int i = 0; i < kOwn; ++i) hist[top + i] = 0;
        __syncthreads();
        base += (uint32_t)pick[0] << shift;
        want = pick[1];
        if (shift == 0) break;
        width = (1u << shift) - 1;
        shift = max(0, shift - 10);
        __syncthreads();  // the picks have been read
    }
    __syncthreads();
    return Edge{base, want};
}

// Score of block n in twice 32 bits; the whole warp calls it and every lane gets the result.
template <bool FP16>
__device__ __forceinline__ Two score_again(const ScoreArgs& a, const float4* table, int r, int n) {
    const int lane = threadIdx.x & 31, columns = a.Hkv * a.D;
    const uint16_t* base = a.bounds + ((long long)r * a.NB + n) * a.row;
    Two z = {0.f, 0.f};
    for (int col = lane; col < columns; col += 32) {
        const int h = col / a.D;
        const uint16_t* p = base + col + h * a.D;
        const float low = value<FP16>(ld(p)), high = value<FP16>(ld(p + a.D));
        const float4 t = table[col];  // Q+, Q-
        const float x = __fmul_rn(t.x, high), y = __fmul_rn(t.z, low);
        z.add(x);
        z.add(y);
        const float ex = __fmaf_rn(t.x, high, -x), ey = __fmaf_rn(t.z, low, -y);
        z.lo = __fadd_rn(z.lo, __fadd_rn(__fmaf_rn(t.y, high, ex), __fmaf_rn(t.w, low, ey)));
    }
    // Both lanes of a pair compute the same sum: the larger lane's number comes second in both.
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const float hi = __shfl_xor_sync(0xffffffffu, z.hi, o);
        const float lo = __shfl_xor_sync(0xffffffffu, z.lo, o);
        const bool up = lane & o;
        Two sum = {up ? hi : z.hi, up ? lo : z.lo};
        sum.add(up ? z.hi : hi);
        sum.lo = __fadd_rn(sum.lo, up ? z.lo : lo);
        z = sum;
    }
    z.normalise();
    return z;
}

template <bool FP16>
__global__ void __launch_bounds__(kSelectThreads) select_kernel(const ScoreArgs a) {
    extern __shared__ __align__(16) uint32_t s_keys[];  // [NB], then the table or the blocks
    __shared__ uint32_t s_hist[kBins];
    __shared__ int s_tmp[33], s_pick[2];
    __shared__ uint32_t s_range[2];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int bs = blockIdx.x, b = bs / a.S, s = bs - b * a.S;
    float4* const table = reinterpret_cast<float4*>(s_keys + ((a.NB + 3) & ~3));
    int* const chosen = reinterpret_cast<int*>(table);
    wait_for_previous();
    const int r = ld(a.req + b);
    int n = ld(a.seq_lens + b);
    n = r < 0 || r >= a.R || n < 0 ? 0 : min(n, a.L);
    const int nb = (n + a.T - 1) / a.T;
    const int lo = min(a.first, nb), hi = max(lo, nb - a.last);  // the candidates
    const int k = a.select - a.first - a.last;                    // wanted of them
    const bool all = nb <= a.select;
    Edge edge = {0u, 0};
    if (!all && k > 0) {
        const float* scores = a.scores + (long long)bs * a.NB;
        for (int i = tid; i < nb; i += kSelectThreads) s_keys[i] = key_of(ld(scores + i));
        float error = 0.f;
        for (int c = lane; c < a.chunks; c += 32)
            error = fmaxf(error, ld(a.error + ((long long)b * a.chunks + c) * a.S + s));
        // bit patterns of floats >= 0 order like the floats
        error = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(error)));
        __syncthreads();
        edge = kth_largest(s_keys, lo, hi, k, s_hist, s_tmp, s_range, s_pick);
        // The true scores of the k-th largest and of every block lie within `error` of the sums.
        const float at = score_of(edge.key);
        const float below = __fadd_rd(at, -2.f * error), above = __fadd_ru(at, 2.f * error);
        if (below > -INFINITY && above < INFINITY) {
            uint32_t low = key_of(below), high = key_of(above);
            int sure = 0, near = 0;
            for (int i = lo + tid; i < hi; i += kSelectThreads) {
                sure += s_keys[i] > high;
                near += s_keys[i] >= low && s_keys[i] <= high;
            }
            sure = block_sum(sure, s_tmp);
            near = block_sum(near, s_tmp);
            if (near == k - sure) {
                edge = Edge{low, near};  // all of them
                for (int i = lo + tid; i < hi; i += kSelectThreads)
                    if (s_keys[i] >= low && s_keys[i] <= high) s_keys[i] = low;
                __syncthreads();
            } else {
                const uint16_t* q = a.q + b * a.q_stride[0] + s * a.q_stride[1];
                for (int col = tid; col < a.Hkv * a.D; col += kSelectThreads) {
                    Two up, down;
                    query_sums<FP16>(a, q, col, up, down);
                    table[col] = make_float4(up.hi, up.lo, down.hi, down.lo);
                }
                __syncthreads();
                // Twice: by the upper half of the new scores, then the blocks equal in it by the lower.
#pragma unroll 1
                for (int half = 0; half < 2; ++half) {
                    for (int i0 = lo + warp * 32; i0 < hi; i0 += kSelectThreads) {
                        const int i = i0 + lane;
                        const uint32_t key = i < hi ? s_keys[i] : 0u;
                        const bool open = i < hi && key >= low && key <= high;
                        if (i < hi && !open) s_keys[i] = key > high ? 0xffffffffu : 0u;
                        unsigned todo = __ballot_sync(0xffffffffu, open);
                        while (todo) {
                            const int j = __ffs(todo) - 1;
                            todo &= todo - 1;
                            const Two z = score_again<FP16>(a, table, r, i0 + j);
                            const uint32_t x = key_of(half == 0 ? z.hi : z.lo);
                            if (lane == 0) s_keys[i0 + j] = min(max(x, 1u), 0xfffffffeu);
                        }
                    }
                    __syncthreads();
                    edge = kth_largest(s_keys, lo, hi, k, s_hist, s_tmp, s_range, s_pick);
                    int equal = 0;
                    for (int i = lo + tid; i < hi; i += kSelectThreads)
                        equal += s_keys[i] == edge.key;
                    equal = block_sum(equal, s_tmp);
                    if (equal == edge.want) break;
                    low = high = edge.key;
                }
            }
        }
    }
    release_next();
    // The chosen blocks in order; a thread takes consecutive ones.
    const int per = (nb + kSelectThreads - 1) / kSelectThreads;
    const int i0 = min(tid * per, nb), i1 = min(i0 + per, nb);
    int both = 0;  // blocks above the edge or always taken, and (upper half) equal to it
    if (!all) {
        for (int i = i0; i < i1; ++i) {
            const bool open = i >= lo && i < hi;
            both += !open || (k > 0 && s_keys[i] > edge.key);
            both += open && k > 0 && s_keys[i] == edge.key ? 1 << 16 : 0;
        }
    }
    int total;
    const int before = block_exclusive_scan(both, s_tmp, &total);
    int ties = before >> 16, to = (before & 0xffff) + min(ties, edge.want);
    if (all) to = i0;
    for (int i = i0; i < i1; ++i) {
        bool in = all || i < lo || i >= hi;
        if (!in && k > 0) {
            in = s_keys[i] > edge.key;
            if (s_keys[i] == edge.key) in = ties++ < edge.want;
        }
        if (in) chosen[to++] = i;
    }
    const int kept = min(nb, a.select);
    for (int i = kept + tid; i < a.select; i += kSelectThreads) chosen[i] = -1;
    __syncthreads();
    if (a.out_blocks) {
        int32_t* out = a.out_blocks + (long long)bs * a.select;
        for (int i = tid; i < a.select; i += kSelectThreads) out[i] = chosen[i];
    }
    int32_t* topk = a.topk + (long long)bs * a.select * a.T;
    for (int i = tid; i < a.select * a.T; i += kSelectThreads) {
        const int j = a.by_T.of(i), block = chosen[j];
        const int t = block * a.T + (i - j * a.T);
        topk[i] = block >= 0 && t < n ? t : -1;
    }
}

template <bool FP16, int S>
cudaError_t score(const ScoreArgs& a, size_t smem, cudaStream_t s) {
    static SmemOptIn opt;
    const cudaError_t e = ensure_smem(score_kernel<FP16, S>, smem, &opt);
    if (e != cudaSuccess) return e;
    return launch_chained(score_kernel<FP16, S>, a.B * a.chunks, 32 * kScoreWarps, smem, 0, s, a);
}

template <bool FP16>
cudaError_t run(const ScoreArgs& a, cudaStream_t s) {
    const size_t smem = 4 * ((size_t)a.S * a.row + (size_t)a.wpr * a.blocks * a.S);
    cudaError_t e;
    switch (a.S) {
        case 1: e = score<FP16, 1>(a, smem, s); break;
        case 2: e = score<FP16, 2>(a, smem, s); break;
        case 3: e = score<FP16, 3>(a, smem, s); break;
        case 4: e = score<FP16, 4>(a, smem, s); break;
        default: return cudaErrorInvalidValue;
    }
    if (e != cudaSuccess) return e;
    static SmemOptIn opt;
    const size_t table = 16 * (size_t)a.Hkv * a.D, chosen = 4 * (size_t)a.select;
    const size_t need = 4 * (size_t)((a.NB + 3) & ~3) + (table > chosen ? table : chosen);
    e = ensure_smem(select_kernel<FP16>, need, &opt);
    if (e != cudaSuccess) return e;
    return launch_chained(select_kernel<FP16>, a.B * a.S, kSelectThreads, need, 0, s, a);
}

}  // namespace

SelectShape select_shape(int32_t batch, int32_t steps, int32_t row, int32_t NB) {
    // Chunks of whole turns of a CTA's warps, about three CTAs an SM in all.
    const int wpr = row > 4 * kSlice ? 8 : row > 2 * kSlice ? 4 : row > kSlice ? 2 : 1;
    const int turn = batch_blocks(steps) * (kScoreWarps / wpr);
    const int most = kMostSums / steps / turn * turn;
    const long long want = 3 * 152 / batch > 0 ? 3 * 152 / batch : 1;
    long long blocks = (NB + want - 1) / want;
    blocks = (blocks + turn - 1) / turn * turn;
    if (blocks > most) blocks = most;
    SelectShape sh;
    sh.blocks = (int)blocks;
    sh.chunks = (int)((NB + blocks - 1) / blocks);
    return sh;
}

cudaError_t launch_select(const hs_select_args& x, cudaStream_t s) {
    ScoreArgs a = {};
    a.q = static_cast<const uint16_t*>(x.q_dev);
    a.bounds = static_cast<const uint16_t*>(x.bounds_dev);
    a.req = x.req_dev;
    a.seq_lens = x.seq_lens_dev;
    a.scores = x.scores_dev;
    a.error = static_cast<float*>(x.workspace_dev);
    a.B = x.batch;
    a.S = x.steps;
    a.Hkv = x.num_kv_heads;
    a.G = x.num_heads / x.num_kv_heads;
    a.D = x.head_dim;
    a.R = x.num_requests;
    a.L = x.max_seq_len;
    a.T = x.block_tokens;
    a.NB = (x.max_seq_len - 1) / x.block_tokens + 1;
    a.row = 2 * a.Hkv * a.D;
    a.wpr = a.row > 4 * kSlice ? 8 : a.row > 2 * kSlice ? 4 : a.row > kSlice ? 2 : 1;
    const SelectShape sh = select_shape(a.B, a.S, a.row, a.NB);
    a.chunks = sh.chunks;
    a.blocks = sh.blocks;
    a.vec_bounds = (uintptr_t)x.bounds_dev % 16 == 0;
    for (int i = 0; i < 3; ++i) a.q_stride[i] = x.q_stride[i];
    // A sum's terms go through one rounding of Q, one of each fused product and sum of a lane's 8
    // elements a slice, 5 additions over the lanes and one for each warp: half a step of 2^-23 of the
    // sum of magnitudes each; the bound itself is a sum of as many, rounded likewise.
    const int slices = (a.row + kSlice * a.wpr - 1) / (kSlice * a.wpr);
    a.gamma = (float)(1 + 8 * slices + 5 + a.wpr) * 0x1p-24f * 1.01f;
    a.select = x.select;
    a.first = x.first;
    a.last = x.last;
    a.out_blocks = x.blocks_dev;
    a.topk = x.topk_dev;
    a.by_T = Divisor::by(a.T);
    return x.dtype == HS_DTYPE_FP16 ? run<true>(a, s) : run<false>(a, s);
}

}  // namespace hs
