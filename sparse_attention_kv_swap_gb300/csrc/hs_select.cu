// Selection of key blocks for decode queries by bounds on their scores (sm_103a).
//
// score(n) = sum over query heads and channels of max(q lo_n, q hi_n).  lo <= hi, so a positive
// q takes hi and a negative one lo, and the query heads of a K/V head add up first:
//   score(n) = sum over K/V heads and channels of Q+ hi_n + Q- lo_n,
//   Q+ = sum of max(q, 0), Q- = sum of min(q, 0),
// two multiply-adds for each pair of bounds, whatever the number of query heads: the bounds
// are read once and nothing else counts (4 bytes for 2 * steps operations: memory).
//
// The first kernel scores: a warp takes 256 elements (512 bytes) of 4 or 8 blocks, each lane 8 of
// them, and holds the sums of all in registers, of even and odd channels apart (one instruction
// multiplies and adds both); over its lanes they add up by halving exchanges.  A lane copies its own 16
// bytes of the next blocks to shared memory ahead of itself (cp.async; no other lane reads
// them, so nothing is synchronised), and begins that before it computes Q.
//
// The second selects, one CTA a query.  Sums in 32 bits depend on their order and would swap blocks whose
// scores are close.  So the first kernel also bounds the error of its sums (a few 2^-24 of
// sum |Q| max_n |bound|, the maximum taken channel by channel), and where blocks that could
// belong on either side of the border are more than there is room for, these are scored again in
// twice 32 bits (error-free products and sums) and selected by that, ties to the lowest index.  The
// selection is then that of the scores themselves, for every launch shape.
//
// 64 requests of 512 blocks, 8 heads of 128, 64 query heads, take 38 us: the scores 28 (4.8 TB/s; 61
// instructions for each 512 bytes, half of them on the ALU, where 16-bit pairs become
// 32-bit numbers and their largest magnitudes are kept), the selection 7, launches the rest.
// 12 requests of up to 4096 blocks with 4 steps take 40: their lengths differ and a step's
// products are latencies of few warps (the sums of 4 steps leave registers for 16 warps an SM).
// More than kList blocks at the border are scored again a warp a block, by the query's one CTA: 390 us
// where all blocks of the first call are alike, 9.5 ms for one query of 16384 such blocks (36 us
// otherwise).
#include "hs_step.cuh"

namespace hs {
namespace {

constexpr int kScoreWarps = 8;
constexpr int kSlice = 256;            // elements of a block that a warp takes at a time
constexpr int kMostSums = 1024;        // scores of a CTA: its blocks times the steps
constexpr int kList = 64;              // close blocks that are ranked pair by pair
constexpr int kSelectThreads = 512, kSelectWarps = kSelectThreads / 32;
constexpr int kBins = 1024;

// Blocks of a warp's registers (8 to 16 sums), those it copies together, and copies of these: a ring of
// 64 KB a CTA.
constexpr int batch_blocks(int S) { return S == 1 ? 8 : 4; }
constexpr int kGroup = 4;
constexpr int kStages = 4;
constexpr size_t kRingBytes = (size_t)kScoreWarps * kStages * kGroup * kSlice * 2;
// CTAs of an SM, by registers and shared memory.
constexpr int score_ctas(int S) { return S <= 2 ? 3 : 2; }
// Warps that share a block: as many as leave each two slices of it or more (it adds up over its
// lanes once for them).
constexpr int warps_per_row(int row) {
    const int slices = (row + kSlice - 1) / kSlice;
    int w = 1;
    while (w < kScoreWarps && slices >= 4 * w) w *= 2;
    return w;
}

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
    int32_t vec_bounds, vec_q;
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

// Larger of the magnitudes, two elements at a time (a NaN does not count).  The sign bits of the result
// mean nothing.
template <bool FP16>
__device__ __forceinline__ uint32_t greater_magnitude(uint32_t m, uint32_t w) {
    uint32_t x;
    if constexpr (FP16)
        asm("max.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(x) : "r"(m), "r"(w));
    else
        asm("max.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(x) : "r"(m), "r"(w));
    return x;
}

// z += q v, both halves.
__device__ __forceinline__ void fma_pair(float2& z, float2 q, float2 v) {
    asm("{\n\t.reg .b64 x, y, z;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%0, %1};\n\t"
        "fma.rn.f32x2 z, x, y, z;\n\tmov.b64 {%0, %1}, z;\n\t}"
        : "+f"(z.x), "+f"(z.y)
        : "f"(q.x), "f"(q.y), "f"(v.x), "f"(v.y));
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

// Four consecutive 16-bit elements.
__device__ __forceinline__ uint2 load4(const uint16_t* p, bool vec) {
    if (vec) return ld(reinterpret_cast<const uint2*>(p));
    return make_uint2((uint32_t)ld(p) | (uint32_t)ld(p + 1) << 16,
                      (uint32_t)ld(p + 2) | (uint32_t)ld(p + 3) << 16);
}

// Q+ and Q- of channels d .. d + 3 of K/V head h of one query, in twice 32 bits.
template <bool FP16>
__device__ __forceinline__ void query_sums(const ScoreArgs& a, const uint16_t* q, int h, int d,
                                           Two (&up)[4], Two (&down)[4]) {
    const uint16_t* p = q + (long long)h * a.G * a.q_stride[2] + d;
#pragma unroll
    for (int k = 0; k < 4; ++k) up[k] = down[k] = Two{0.f, 0.f};
#pragma unroll 4
    for (int g = 0; g < a.G; ++g) {
        const uint2 w = load4(p + g * a.q_stride[2], a.vec_q);
        const float2 y[2] = {values<FP16>(w.x), values<FP16>(w.y)};
        const float x[4] = {y[0].x, y[0].y, y[1].x, y[1].y};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            down[k].add(x[k] < 0.f ? x[k] : 0.f);
            up[k].add(x[k] < 0.f ? 0.f : x[k]);  // a NaN spoils the query's scores
        }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        up[k].normalise();
        down[k].normalise();
    }
}

// Copies this lane's 8 elements of a block to shared memory, or zeros.
__device__ __forceinline__ void copy_bounds(uint32_t to, const uint16_t* p, bool vec, bool on) {
    if (vec) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(p),
                     "r"(on ? 16 : 0)
                     : "memory");
    } else {
        uint2 x = make_uint2(0, 0), y = x;
        if (on) x = load4(p, false), y = load4(p + 4, false);
        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(to), "r"(x.x), "r"(x.y),
                     "r"(y.x), "r"(y.y)
                     : "memory");
    }
}

template <bool FP16, int S>
__global__ void __launch_bounds__(32 * kScoreWarps, score_ctas(S)) score_kernel(const ScoreArgs a) {
    constexpr int NB = batch_blocks(S), kSums = S * NB > 8 ? 16 : 8;
    extern __shared__ __align__(16) uint8_t s_ring[];  // [warp][stage][block][256], then Q and sums
    __shared__ float s_error[kScoreWarps][S];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int chunk = blockIdx.x % a.chunks, b = blockIdx.x / a.chunks;
    float* const s_q = reinterpret_cast<float*>(s_ring + kRingBytes);  // [S][row]
    float* const s_sum = s_q + S * a.row;                                 // [wpr][blocks * S]
    wait_for_previous();
    const int r = ld(a.req + b);
    int n = ld(a.seq_lens + b);
    n = r < 0 || r >= a.R || n < 0 ? 0 : min(n, a.L);
    const int nb = (n + a.T - 1) / a.T;
    const int n0 = chunk * a.blocks, n1 = min(n0 + a.blocks, a.NB);
    const int live = max(0, min(n1, nb) - n0);  // blocks to score
    const uint16_t* const base = a.bounds + ((long long)max(r, 0) * a.NB + n0) * a.row;
    const int part = warp % a.wpr, turns = kScoreWarps / a.wpr;
    const int e_first = part * kSlice, e_step = a.wpr * kSlice;
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(s_ring) +
                          warp * (kStages * kGroup * kSlice * 2) + lane * 16;
    // The copies run ahead of the sums in the same order: blocks, slices, groups of the slice's blocks.
    int c_j = warp / a.wpr * NB, c_e = e_first, c_g = 0, c_stage = 0;
    const auto copy_next = [&] {
        if (c_j < live && c_e < a.row) {
            // blocks past the last are that one again: their sums are not kept
            const bool on = c_e + lane * 8 < a.row;
            const uint16_t* from = base + (on ? c_e + lane * 8 : 0);
            const uint32_t to = ring + c_stage * (kGroup * kSlice * 2);
#pragma unroll
            for (int g = 0; g < kGroup; ++g)
                copy_bounds(to + g * (kSlice * 2), from + min(c_j + c_g + g, live - 1) * a.row,
                            a.vec_bounds, on);
            c_g += kGroup;
            if (c_g >= NB || c_j + c_g >= live) {
                c_g = 0;
                c_e += e_step;
                if (c_e >= a.row) {
                    c_e = e_first;
                    c_j += turns * NB;
                }
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        c_stage = (c_stage + 1) % kStages;
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) copy_next();
    if (live > 0) {
        // Q- and Q+ of all columns, in the order of the bounds.
        const int quads = a.D / 4, all = a.Hkv * quads;
        for (int i = tid; i < S * all; i += 32 * kScoreWarps) {
            const int s = i / all, u = i - s * all, h = u / quads, d = 4 * (u - h * quads);
            Two up[4], down[4];
            query_sums<FP16>(a, a.q + b * a.q_stride[0] + s * a.q_stride[1], h, d, up, down);
            float* to = s_q + s * a.row + 2 * h * a.D + d;
            *reinterpret_cast<float4*>(to) =
                make_float4(down[0].hi, down[1].hi, down[2].hi, down[3].hi);
            *reinterpret_cast<float4*>(to + a.D) =
                make_float4(up[0].hi, up[1].hi, up[2].hi, up[3].hi);
        }
    }
    __syncthreads();
    float worst[S] = {};
    int stage = 0;
    for (int j0 = warp / a.wpr * NB; j0 < live; j0 += turns * NB) {
        float2 both[kSums];
#pragma unroll
        for (int i = 0; i < kSums; ++i) both[i] = make_float2(0.f, 0.f);
        float error[S] = {};
        for (int e0 = e_first; e0 < a.row; e0 += e_step) {
            const int e = e0 + lane * 8;
            float2 q[S][4];
#pragma unroll
            for (int s = 0; s < S; ++s) {
                float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
                if (e < a.row) {
                    x = *reinterpret_cast<const float4*>(s_q + s * a.row + e);
                    y = *reinterpret_cast<const float4*>(s_q + s * a.row + e + 4);
                }
                q[s][0] = make_float2(x.x, x.y), q[s][1] = make_float2(x.z, x.w);
                q[s][2] = make_float2(y.x, y.y), q[s][3] = make_float2(y.z, y.w);
            }
            uint32_t most[4] = {};
#pragma unroll
            for (int g0 = 0; g0 < NB; g0 += kGroup) {
                if (j0 + g0 >= live) break;
                asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
                copy_next();  // to the stage of the group before this one, whose sums are taken
                const uint32_t at = ring + stage * (kGroup * kSlice * 2);
#pragma unroll
                for (int g = 0; g < kGroup; ++g) {
                    uint32_t w[4];
                    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                                 : "r"(at + g * (kSlice * 2))
                                 : "memory");
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        most[i] = greater_magnitude<FP16>(most[i], w[i]);
                        const float2 v = values<FP16>(w[i]);
#pragma unroll
                        for (int s = 0; s < S; ++s) fma_pair(both[s * NB + g0 + g], q[s][i], v);
                    }
                }
                stage = (stage + 1) % kStages;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 m = values<FP16>(most[i]);
#pragma unroll
                for (int s = 0; s < S; ++s)
                    error[s] += fabsf(q[s][i].x) * fabsf(m.x) + fabsf(q[s][i].y) * fabsf(m.y);
            }
        }
#pragma unroll
        for (int s = 0; s < S; ++s)  // no bound where there is an infinity
            worst[s] = fmaxf(worst[s], error[s] == error[s] ? error[s] : INFINITY);
        // Lane l gets the sum over the lanes of number l modulo their count.
        float acc[kSums];
#pragma unroll
        for (int i = 0; i < kSums; ++i) acc[i] = both[i].x + both[i].y;
#pragma unroll
        for (int o = kSums / 2; o > 0; o >>= 1) {
            const bool up = lane & o;
#pragma unroll
            for (int i = 0; i < o; ++i) {
                const float give = up ? acc[i] : acc[i + o];
                const float keep = up ? acc[i + o] : acc[i];
                acc[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
            }
        }
#pragma unroll
        for (int o = kSums; o < 32; o <<= 1) acc[0] += __shfl_xor_sync(0xffffffffu, acc[0], o);
        const int s = lane / NB, j = j0 + lane - s * NB;
        if (s < S && j < live) s_sum[part * a.blocks * S + s * a.blocks + j] = acc[0];
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
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

// The k-th largest of keys[lo, hi), 1 <= k <= hi - lo.  All threads call it, each with the least and the
// greatest of its keys: scores share their top bits, and counting by these would bring all into a few
// bins.  Counts the keys of each of 1024 ranges and goes on within the one that holds the k-th, until
// that is a few keys, which are compared one by one.
__device__ __forceinline__ Edge kth_largest(const uint32_t* keys, int lo, int hi, int k,
                                            uint32_t least, uint32_t most, uint32_t* hist, int* tmp,
                                            uint32_t* range, int* pick, uint32_t* list) {
    const int tid = threadIdx.x;
    if (tid == 0) range[0] = 0xffffffffu, range[1] = 0u;
#pragma unroll
    for (int i = 0; i < kBins; i += kSelectThreads) hist[i + tid] = 0;
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
#pragma unroll 1
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
                pick[2] = mine[i];
                pick[3] = 0;
            }
            above += mine[i];
        }
#pragma unroll
        for (int i = 0; i < kOwn; ++i) hist[top + i] = 0;
        __syncthreads();
        base += (uint32_t)pick[0] << shift;
        want = pick[1];
        if (shift == 0) break;
        width = (1u << shift) - 1;
        const int count = pick[2];
        if (count <= kList) {
#pragma unroll 1
            for (int i = lo + tid; i < hi; i += kSelectThreads)
                if (keys[i] >= base && keys[i] - base <= width) list[atomicAdd(&pick[3], 1)] = keys[i];
            __syncthreads();
            if (tid < count) {
                int above = 0, equal = 0;
#pragma unroll 1
                for (int i = 0; i < count; ++i) {
                    above += list[i] > list[tid];
                    equal += list[i] == list[tid];
                }
                if (above < want && want <= above + equal) {  // equal keys write the same
                    range[0] = list[tid];
                    pick[1] = want - above;
                }
            }
            __syncthreads();
            base = range[0];
            want = pick[1];
            break;
        }
        shift = max(0, shift - 10);
        __syncthreads();  // the picks have been read
    }
    __syncthreads();
    return Edge{base, want};
}

// Sum in twice 32 bits over the quads of channels [u0, u1) of block n's score; the whole warp calls it
// and every lane gets the result.  The table holds, for each quad, Q+ (upper and lower halves), Q-.
template <bool FP16>
__device__ __forceinline__ Two score_again(const ScoreArgs& a, const float4* table, int r, int n,
                                           int u0, int u1) {
    const int lane = threadIdx.x & 31, quads = a.D / 4;
    const uint16_t* base = a.bounds + ((long long)r * a.NB + n) * a.row;
    Two z = {0.f, 0.f};
    for (int u = u0 + lane; u < u1; u += 32) {
        const int h = u / quads, d = 4 * (u - h * quads);
        const uint16_t* p = base + 2 * h * a.D + d;
        const uint2 wl = load4(p, a.vec_bounds), wh = load4(p + a.D, a.vec_bounds);
        const float2 l[2] = {values<FP16>(wl.x), values<FP16>(wl.y)};
        const float2 g[2] = {values<FP16>(wh.x), values<FP16>(wh.y)};
        const float low[4] = {l[0].x, l[0].y, l[1].x, l[1].y};
        const float high[4] = {g[0].x, g[0].y, g[1].x, g[1].y};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float4 t = table[4 * u + k];
            const float x = __fmul_rn(t.x, high[k]), y = __fmul_rn(t.z, low[k]);
            z.add(x);
            z.add(y);
            const float ex = __fmaf_rn(t.x, high[k], -x), ey = __fmaf_rn(t.z, low[k], -y);
            z.lo = __fadd_rn(z.lo,
                             __fadd_rn(__fmaf_rn(t.y, high[k], ex), __fmaf_rn(t.w, low[k], ey)));
        }
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
    __shared__ int s_tmp[33], s_pick[4];
    __shared__ uint32_t s_range[2], s_some[kList];
    __shared__ int s_list[kList], s_found, s_both, s_taken[kSelectWarps];
    __shared__ float2 s_part[kList];
    __shared__ uint64_t s_rank[kList];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int bs = blockIdx.x, b = bs / a.S, s = bs - b * a.S;
    float4* const table = reinterpret_cast<float4*>(s_keys + ((a.NB + 3) & ~3));
    int* const chosen = reinterpret_cast<int*>(table);
    wait_for_previous();
    // All loads under way at once; scores past the sequence are -inf.
    const int r = ld(a.req + b);
    int n = ld(a.seq_lens + b);
    float error = 0.f;
#pragma unroll 1
    for (int c = lane; c < a.chunks; c += 32)
        error = fmaxf(error, ld(a.error + ((long long)b * a.chunks + c) * a.S + s));
    // bit patterns of floats >= 0 order like the floats
    error = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(error)));
    constexpr int kLoads = 8;
    const float* const scores = a.scores + (long long)bs * a.NB;
    uint32_t least = 0xffffffffu, most = 0u;
    int nb = 0, lo = 0, hi = 0;
#pragma unroll 1
    for (int i0 = tid; i0 < a.NB + tid; i0 += kLoads * kSelectThreads) {
        float x[kLoads];
#pragma unroll
        for (int u = 0; u < kLoads; ++u) {
            const int i = i0 + u * kSelectThreads;
            x[u] = i < a.NB ? ld(scores + i) : 0.f;
        }
        if (i0 == tid) {
            n = r < 0 || r >= a.R || n < 0 ? 0 : min(n, a.L);
            nb = (n + a.T - 1) / a.T;
            lo = min(a.first, nb), hi = max(lo, nb - a.last);  // the candidates
        }
#pragma unroll
        for (int u = 0; u < kLoads; ++u) {
            const int i = i0 + u * kSelectThreads;
            const uint32_t key = key_of(x[u]);
            if (i < a.NB) s_keys[i] = key;
            if (i >= lo && i < hi) {
                least = min(least, key);
                most = max(most, key);
            }
        }
    }
    const int k = a.select - a.first - a.last;  // wanted of the candidates
    const bool all = nb <= a.select;
    Edge edge = {0xffffffffu, 0};
    if (!all && k > 0) {
        if (tid == 0) s_found = s_both = 0;
        edge = kth_largest(s_keys, lo, hi, k, least, most, s_hist, s_tmp, s_range, s_pick, s_some);
        // The true scores of the k-th largest and of every block lie within `error` of the sums.
        const float at = score_of(edge.key);
        const float below = __fadd_rd(at, -2.f * error), above = __fadd_ru(at, 2.f * error);
        if (below > -INFINITY && above < INFINITY) {
            uint32_t low = key_of(below), high = key_of(above);
            int both = 0;  // blocks above the band, and (upper half) within it
#pragma unroll 1
            for (int i = lo + tid; i < hi; i += kSelectThreads) {
                const uint32_t key = s_keys[i];
                both += key > high ? 1 : key >= low ? 1 << 16 : 0;
                if (key <= high && key >= low) {
                    const int at = atomicAdd(&s_found, 1);
                    if (at < kList) s_list[at] = i;  // in any order: ranked below
                }
            }
            both = __reduce_add_sync(0xffffffffu, both);
            if (lane == 0 && both) atomicAdd(&s_both, both);
            __syncthreads();
            both = s_both;
            const int near = both >> 16, open = k - (both & 0xffff);
            if (near == open) {
                edge = Edge{low - 1, 0};  // all of them
            } else {
                const uint16_t* q = a.q + b * a.q_stride[0] + s * a.q_stride[1];
                const int quads = a.D / 4, units = a.Hkv * quads;
                for (int u = tid; u < units; u += kSelectThreads) {
                    const int h = u / quads, d = 4 * (u - h * quads);
                    Two up[4], down[4];
                    query_sums<FP16>(a, q, h, d, up, down);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        table[4 * u + i] =
                            make_float4(up[i].hi, up[i].lo, down[i].hi, down[i].lo);
                }
                __syncthreads();
                if (near <= kList) {
                    // A few: a block's sum in equal parts over the warps, then a rank for each.
                    const int parts = near >= kSelectWarps ? 1 : kSelectWarps / near;
                    const int each = (units + parts - 1) / parts;
                    for (int w = warp; w < near * parts; w += kSelectWarps) {
                        const int i = w / parts, u0 = (w - i * parts) * each;
                        const Two z = score_again<FP16>(a, table, r, s_list[i], u0,
                                                        min(u0 + each, units));
                        if (lane == 0) s_part[w] = make_float2(z.hi, z.lo);
                    }
                    __syncthreads();
                    if (tid < near) {
                        Two z = {0.f, 0.f};
                        for (int i = 0; i < parts; ++i) {
                            const float2 x = s_part[tid * parts + i];
                            z.add(x.x);
                            z.lo = __fadd_rn(z.lo, x.y);
                        }
                        z.normalise();
                        s_rank[tid] = (uint64_t)key_of(z.hi) << 32 | key_of(z.lo);
                    }
                    __syncthreads();
                    if (tid < near) {
                        const uint64_t mine = s_rank[tid];
                        const int me = s_list[tid];
                        int before = 0;
                        for (int i = 0; i < near; ++i)
                            before += s_rank[i] > mine || (s_rank[i] == mine && s_list[i] < me);
                        s_keys[me] = before < open ? 0xffffffffu : 0u;
                    }
                    edge = Edge{high, 0};
                    __syncthreads();
                } else {
                    // Many (mostly equal ones): by the upper half of the new scores, then the blocks
                    // equal in it by the lower.
#pragma unroll 1
                    for (int half = 0; half < 2; ++half) {
                        for (int i0 = lo + warp * 32; i0 < hi; i0 += kSelectThreads) {
                            const int i = i0 + lane;
                            const uint32_t key = i < hi ? s_keys[i] : 0u;
                            const bool in = i < hi && key >= low && key <= high;
                            if (i < hi && !in) s_keys[i] = key > high ? 0xffffffffu : 0u;
                            unsigned todo = __ballot_sync(0xffffffffu, in);
                            while (todo) {
                                const int j = __ffs(todo) - 1;
                                todo &= todo - 1;
                                const Two z = score_again<FP16>(a, table, r, i0 + j, 0, units);
                                const uint32_t x = key_of(half == 0 ? z.hi : z.lo);
                                if (lane == 0) s_keys[i0 + j] = min(max(x, 1u), 0xfffffffeu);
                            }
                        }
                        __syncthreads();
                        least = 0xffffffffu, most = 0u;
                        for (int i = lo + tid; i < hi; i += kSelectThreads) {
                            least = min(least, s_keys[i]);
                            most = max(most, s_keys[i]);
                        }
                        edge = kth_largest(s_keys, lo, hi, k, least, most, s_hist, s_tmp, s_range,
                                           s_pick, s_some);
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
    }
    release_next();
    // The chosen blocks in order.  A warp has consecutive ones: it counts those above the edge (or
    // always taken) and, in the upper half of the number, those equal to it.
    const int per = (nb + kSelectThreads - 1) / kSelectThreads * 32;
    const int i0 = warp * per, i1 = min(i0 + per, nb);
    const auto kind = [&](int i) {
        if (i >= i1) return 0;
        if (all || i < lo || i >= hi) return 1;
        const uint32_t key = s_keys[i];
        return key > edge.key ? 1 : key == edge.key ? 1 << 16 : 0;
    };
    int taken = 0;
#pragma unroll 1
    for (int i = i0; i < i1; i += 32) taken += kind(i + lane);
    taken = __reduce_add_sync(0xffffffffu, taken);
    if (lane == 0) s_taken[warp] = taken;
    __syncthreads();
    taken = __reduce_add_sync(0xffffffffu, lane < warp ? s_taken[lane] : 0);
    int above = taken & 0xffff, equal = taken >> 16;
    const unsigned below_lane = (1u << lane) - 1;
#pragma unroll 1
    for (int i = i0; i < i1; i += 32) {
        const int x = kind(i + lane);
        const unsigned ups = __ballot_sync(0xffffffffu, x == 1);
        const unsigned ties = __ballot_sync(0xffffffffu, x > 1);
        const int at = equal + __popc(ties & below_lane);
        if (x == 1 || (x > 1 && at < edge.want))
            chosen[above + __popc(ups & below_lane) + min(at, edge.want)] = i + lane;
        above += __popc(ups);
        equal += __popc(ties);
    }
    const int kept = min(nb, a.select);
#pragma unroll 1
    for (int i = kept + tid; i < a.select; i += kSelectThreads) chosen[i] = -1;
    __syncthreads();
    if (a.out_blocks) {
        int32_t* out = a.out_blocks + (long long)bs * a.select;
#pragma unroll 1
        for (int i = tid; i < a.select; i += kSelectThreads) out[i] = chosen[i];
    }
    int32_t* topk = a.topk + (long long)bs * a.select * a.T;
#pragma unroll 1
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
    const size_t smem =
        kRingBytes + 4 * ((size_t)a.S * a.row + (size_t)a.wpr * a.blocks * a.S);
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
    // Chunks of whole turns of a CTA's warps, as many CTAs as the SMs hold: all read from the start on,
    // and a second wave of a few would take as long as the first.
    const int wpr = warps_per_row(row);
    int turn = batch_blocks(steps) * (kScoreWarps / wpr);
    if (turn < kSelectChunk) turn = kSelectChunk;  // a multiple of either
    const int most = kMostSums / steps / turn * turn;
    const long long held = score_ctas(steps) * 152;
    const long long want = batch < held ? held / batch : 1;
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
    a.wpr = warps_per_row(a.row);
    const SelectShape sh = select_shape(a.B, a.S, a.row, a.NB);
    a.chunks = sh.chunks;
    a.blocks = sh.blocks;
    a.vec_bounds = (uintptr_t)x.bounds_dev % 16 == 0;
    a.vec_q = (uintptr_t)x.q_dev % 8 == 0;
    for (int i = 0; i < 3; ++i) {
        a.q_stride[i] = x.q_stride[i];
        a.vec_q = a.vec_q && x.q_stride[i] % 4 == 0;
    }
    // A sum's terms go through one rounding of Q, one of each fused product and sum of a lane's 4
    // channels of either parity a slice, one of the parities' sum, 5 additions over the lanes and one for
    // each warp: half a step of 2^-23 of the sum of magnitudes each; the bound itself is a sum of as many
    // positive terms (up to 8 a slice), rounded likewise.
    const int slices = (a.row + kSlice * a.wpr - 1) / (kSlice * a.wpr);
    a.gamma = (float)(1 + 4 * slices + 1 + 5 + a.wpr) * 0x1p-24f * 1.01f;
    a.select = x.select;
    a.first = x.first;
    a.last = x.last;
    a.out_blocks = x.blocks_dev;
    a.topk = x.topk_dev;
    a.by_T = Divisor::by(a.T);
    return x.dtype == HS_DTYPE_FP16 ? run<true>(a, s) : run<false>(a, s);
}

}  // namespace hs
