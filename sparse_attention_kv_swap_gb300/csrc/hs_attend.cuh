// Attention of decode queries over 8-bit rows at device locations (sm_103a);
// the contract is hs_attend's in include/hisparse_swap.h.
//
// A thread-block cluster of P CTAs serves one query position (b, s); the CTAs
// take its selected rows in turns of 16, for all heads, and drop the masked
// ones.  A warp's task is one K/V head (and up to 16 of the query heads that
// share it) over tiles of 16 tokens:
//   1. scores: S^T[token, head] = K[token, d] Q^T[d, head] with f16
//      m16n8k16 products summed in 32 bits.  A selected row is read by exactly
//      one warp per K/V head and group of query heads, so the warps share nothing: each copies the
//      pieces of its head (cp.async, whole 128-byte lines where D allows:
//      gathering in 64-byte pieces costs a fifth of the bandwidth) into a queue
//      of its own in shared memory, several tiles ahead, and reads them back
//      as operands (ldmatrix).  A product may visit d in any order, so the
//      four bytes of a word are four d of one step.  Codes are exact in f16;
//      the query is scaled by a power of two per head into f16's range, which
//      keeps bf16's and f16's significands whole down to 2^-28 of the head's
//      largest element (smaller ones are off by 2^-39 of it at most).  Scores stay in 32 bits, in
//      the fragment's own layout, in tensor memory: 512 columns of an SM that
//      nothing else here needs, where shared memory would hold a quarter as
//      many tokens beside the queues.
//   2. softmax over the task's own tokens: all scores are known, so there is
//      no running rescale.
//   3. O^T[d, head] = V^T[d, token] P^T[token, head]: the byte form of
//      ldmatrix transposes V, so that a word holds four tokens of one d.  The
//      rows of a K tile are taken in the order 0, 1, 4, 5, .. | 2, 3, 6, 7, ..
//      so that the transposed P (movmatrix) pairs the same tokens.  P is
//      exp(s - max) times the token's V scale, multiplied by what brings the largest
//      one of a head in the task to 2^15, and rounded to f16: by 2^-11 of each at
//      most, or 2^-40 of the largest one where that is more; the largest itself
//      stays whole.  That is an eighth of a bf16 output's own rounding, and as much
//      as an f16 output's (against 64 bits, f16 outputs of the timed cases are
//      off by 2.1 to 2.3e-4 of their norm; 2.1e-4 with P in 32 bits).  The factor
//      belongs to the largest product of P and V scale, not to the largest V scale:
//      that one may belong to a token of no weight.
// With 4 query heads to a K/V head or fewer, one fragment takes two tiles: the
// 8 columns are the heads of the first tile and again those of the second, the
// queries lying in both halves, and each lane keeping its tile's product.  Scores,
// exponentials and tensor memory then halve (NT = 0 below).
// Then the CTAs of the cluster exchange maxima and sums over distributed
// shared memory, each adds up a share of the output over the CTAs in rank
// order, and each turns its own scores into weights with the query's final
// sums.  Nothing goes through global memory but inputs and outputs, and no
// result depends on timing, but for sums that get several additions in one launch: of a
// request that the batch holds twice, or of a token that a query holds in two rows.
//
// What bounds it: every row is read once per step, 2 * Hkv * D bytes, for
// 4 * Hq * D operations, i.e. 2 * (Hq / Hkv) operations a byte: memory, with
// the products far below the tensor rate even on mma.sync.  64 queries of 2048
// rows, 8 heads of 128 (268 MB), take 62-63 us, 4.3 TB/s.  Gathering the same rows and
// nothing else, launches back to back, takes 44 us in whole rows and 48 through queues
// like these; the rest is the start and the end of a cluster (positions, scales,
// exchange), in which nothing is gathered and which all CTAs go through together.  Where steps share rows
// or heads are many, the work on the codes bounds it: converting 16 x D codes
// to f16 is most of the 460 instructions that a tile takes for 8 query heads,
// and 64 x 4 queries of 2048 rows, 4 heads of 128, 70% of them shared by
// neighbouring steps, take 92 us (5.8 TB/s out of L2 and memory).  tcgen05.mma would
// want 128 rows of one operand in shared memory as f16, which here would mean
// writing every code back after its conversion; its e4m3 form takes codes
// as they are, but queries and weights then in three e4m3 parts each, int8
// not at all.  The mma.sync e4m3 form in three parts took 27 us for the scores
// that take 16 by conversion.
#pragma once

#include <cooperative_groups.h>

#include "hs_kv.cuh"

namespace hs {

struct AttendKernelArgs {
    const void* q;
    void* out;
    int32_t fp16, B, S, K, Hq, Hkv, G, R, L, NB, W;
    Divisor block;  // by block_tokens
    float scale_log2;  // sm_scale * log2(e)
    int64_t q_stride[3], out_stride[3];
    const uint8_t* rows;
    long long num_rows;
    const int32_t* locs;
    const int32_t* topk;
    const int32_t* req;
    const float* scales;
    float* lse;
    float* weights;
    float* acc;
    uint8_t* spill;  // scores and per-token arrays of every CTA if the SM cannot hold them
    // launch shape
    int32_t vec_q, vec_out, vec_scale;  // vector loads and stores are aligned
    int32_t TS, TC;          // tokens of a CTA at most; stride of a scale row
    int32_t ngroups, nsub;   // query-head groups of a K/V head; parts of a CTA's tokens
    int32_t alias;           // 1: the output partials reuse the queues' memory
    int32_t task_cols;       // tensor-memory columns of a task's scores
    int32_t cols;            // of the CTA (0: scores in the workspace)
    int32_t token_bytes;     // workspace bytes of a CTA
};

struct AttendShape {
    int P, threads, nt;  // cluster, threads, 8-head tiles of a task
    bool spill;
    size_t smem;
    AttendKernelArgs a;  // TS .. token_bytes filled in
};

// Defined once per code in hs_attend_e4m3.cu and hs_attend_int8.cu.
cudaError_t attend_run_e4m3(const AttendShape& sh, int D, cudaStream_t s);
cudaError_t attend_run_int8(const AttendShape& sh, int D, cudaStream_t s);
// CTAs in clusters of P that the current device runs at once, with so much shared memory and 8
// warps a CTA (0 if the query fails).
int attend_resident(int P, size_t smem);

constexpr int kMaxCluster = 16;
// Warps of a CTA at most: 128 registers a thread, twice that for the widest tasks with 64-bit
// addresses throughout.
constexpr int attend_warps(int D, bool spill) { return D > 192 && spill ? 8 : 16; }

// Tiles in a warp's queue (16 * D bytes each): all but one are on their way
// while one is used.  With D = 128 and 3, 4 or 6 tiles, 64 x 4 queries of 2048 rows took 103, 99
// and 111 us with their sums (deeper queues leave room for fewer tokens), 64 x 1 queries 61.7,
// 62.5 and 63.6; with D = 64 and 4, 6 or 8, 16 queries of 8192 rows 42.8, 41.6 and 48.0.
constexpr int attend_stages(int D) {
    return D <= 32 ? 8 : (D <= 64 ? 6 : (D <= 96 ? 5 : (D <= 128 ? 4 : 3)));
}

#ifdef __CUDACC__

namespace attend {

namespace cg = cooperative_groups;

__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The codes in the low and the high half of a word, as two f16 pairs.
template <int CODE>
__device__ __forceinline__ void halves(uint32_t w, uint32_t& lo, uint32_t& hi) {
    if constexpr (CODE == HS_KV_E4M3) {
        asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n"
            " cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}"
            : "=r"(lo), "=r"(hi)
            : "r"(w));
    } else {
        // 0x6400 | x is the f16 1024 + x for a byte x: with the code's sign bit
        // flipped, x = code + 128, and 1152 is taken off exactly.
        const uint32_t x = w ^ 0x80808080u;
        const __half2 off = __half2half2(__ushort_as_half(0x6480));
        uint32_t p = __byte_perm(x, 0x64646464u, 0x4140), q = __byte_perm(x, 0x64646464u, 0x4342);
        const __half2 a = __hsub2(*reinterpret_cast<__half2*>(&p), off);
        const __half2 b = __hsub2(*reinterpret_cast<__half2*>(&q), off);
        lo = *reinterpret_cast<const uint32_t*>(&a);
        hi = *reinterpret_cast<const uint32_t*>(&b);
    }
}

__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ float log2_fast(float x) {
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float reciprocal_fast(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Transposes an 8 x 8 matrix of 16-bit elements that the warp holds as pairs.
__device__ __forceinline__ uint32_t transpose(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ uint32_t shared_address(const void* p) {
    return (uint32_t)__cvta_generic_to_shared(p);
}

// A tile in the queue is 16 rows of D bytes, their 16-byte chunks permuted by
// row so that the 8 chunks of one ldmatrix matrix fall into different banks:
// of rows 0-7 or 8-15 (V), of rows 0, 1, 4, 5, 8, 9, 12, 13 or those two
// further (K).
template <int D>
__device__ __forceinline__ uint32_t chunk_at(int row, int chunk) {
    int x = 0;
    if constexpr (D % 128 == 0)
        x = (row & 1) | (row >> 1 & 2) | ((row >> 1 ^ row >> 3) & 1) << 2;
    else if constexpr (D % 64 == 0)  // two rows to 128 bytes
        x = (row >> 2 & 1) | ((row >> 1 ^ row >> 3) & 1) << 1;
    else if constexpr (D == 32)
        x = (row >> 2 ^ row >> 3) & 1;
    return (uint32_t)(row * D + (chunk ^ x) * 16);
}

__device__ __forceinline__ void commit_copies() {
    asm volatile("cp.async.commit_group;" ::: "memory");
}
// Waits for all but the last N committed groups of copies of this thread.
template <int N>
__device__ __forceinline__ void wait_copies() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Four 8 x 8 matrices of 16-bit elements, lane l giving the address of row l % 8 of matrix l / 8.
__device__ __forceinline__ void read_matrices(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}
// Two 16 x 16 matrices of bytes, transposed, lane l giving the address of row l % 16 of matrix
// l / 16: word i of lane (g, c) holds rows 4 c .. 4 c + 3 of column g + 8 * (i % 2) of matrix i / 2.
__device__ __forceinline__ void read_transposed(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}

// The 16-bit elements 16 w + 4 c .. + 3 of a query row, as pairs.
template <int STEPS>
__device__ __forceinline__ void load_query(uint32_t (&r)[2 * STEPS], const uint16_t* p, int c,
                                           bool on, bool vec) {
#pragma unroll
    for (int w = 0; w < STEPS; ++w) {
        const uint16_t* at = p + 16 * w + 4 * c;
        if (vec) {
            r[2 * w] = r[2 * w + 1] = 0;
            if (on)
                asm volatile("ld.global.v2.u32 {%0, %1}, [%2];"
                             : "=r"(r[2 * w]), "=r"(r[2 * w + 1])
                             : "l"(at));
        } else {
            r[2 * w] = on ? (uint32_t)ld(at) | ((uint32_t)ld(at + 1) << 16) : 0u;
            r[2 * w + 1] = on ? (uint32_t)ld(at + 2) | ((uint32_t)ld(at + 3) << 16) : 0u;
        }
    }
}

// A pair of bf16 or f16 elements as 32-bit values.
__device__ __forceinline__ float2 pair(uint32_t w, int fp16) {
    if (fp16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// Loads from the shared memory of another CTA of the cluster: `p` is this CTA's own address of
// the array.
__device__ __forceinline__ uint32_t remote(const float* p, int rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(shared_address(p)), "r"(rank));
    return r;
}
__device__ __forceinline__ float load_remote(const float* p, int rank) {
    float x;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(remote(p, rank)));
    return x;
}
__device__ __forceinline__ float4 load_remote4(const float* p, int rank) {
    float4 x;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w)
                 : "r"(remote(p, rank)));
    return x;
}

// Place of a token's scale in its row: the two tokens of a lane's score fragment, t and t + 2,
// lie side by side.
__device__ __forceinline__ int scale_slot(int t) {
    return (t & ~3) | (t & 1) << 1 | (t >> 1 & 1);
}

// Query head, within its group, of column 2 c of a score fragment.
template <int NT>
__device__ __forceinline__ int column_head(int c) {
    return NT == 0 ? (2 * c) & 3 : 2 * c;
}

// Reductions over the 8 lanes that share c (lanes differ in g).
__device__ __forceinline__ float max_over_g(float x) {
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}
__device__ __forceinline__ float sum_over_g(float x) {
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// The scores of a warp's tasks, one score fragment a lane per tile and 8-head
// tile: in tensor memory (a warp reaches the 32 lanes of its quarter, and the
// columns divide among the warps of a quarter), or in the workspace.
template <int NT, bool SPILL>
struct Scores {
    uint32_t col;  // first column of the task, with the warp's lanes in the high half
    float4* mem;

    // `turn`: which of the warp's tasks.
    __device__ __forceinline__ Scores(const AttendKernelArgs& a, uint32_t base, float* ws, int warp,
                                      int nwarps, int turn) {
        if constexpr (SPILL) {
            mem = reinterpret_cast<float4*>(ws) +
                  (long long)(turn * nwarps + warp) * (a.task_cols / 4) * 32 + (threadIdx.x & 31);
        } else {
            const int rows = (nwarps + 3) >> 2;  // warps of a quarter at most
            col = base + ((uint32_t)(warp & 3) << 21) +
                  (uint32_t)((turn * rows + (warp >> 2)) * a.task_cols);
        }
    }
    // All lanes of the warp store and load together.
    __device__ __forceinline__ void store(int tile, const float (&s)[NT][4]) const {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            if constexpr (SPILL)
                mem[(tile * NT + nt) * 32] =
                    make_float4(s[nt][0], s[nt][1], s[nt][2], s[nt][3]);
            else
                asm volatile(
                    "tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                        col + (tile * NT + nt) * 4),
                    "f"(s[nt][0]), "f"(s[nt][1]), "f"(s[nt][2]), "f"(s[nt][3])
                    : "memory");
        }
    }
    __device__ __forceinline__ void stored() const {
        if constexpr (!SPILL) asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
    }
    __device__ __forceinline__ void load(int tile, float (&s)[NT][4]) const {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            if constexpr (SPILL) {
                const float4 x = mem[(tile * NT + nt) * 32];
                s[nt][0] = x.x, s[nt][1] = x.y, s[nt][2] = x.z, s[nt][3] = x.w;
            } else {
                asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
                             : "=f"(s[nt][0]), "=f"(s[nt][1]), "=f"(s[nt][2]), "=f"(s[nt][3])
                             : "r"(col + (tile * NT + nt) * 4)
                             : "memory");
            }
        }
    }
    // The loaded scores may be used after this (without a wait: one was waited for already).
    __device__ __forceinline__ void loaded(float (&s)[NT][4], bool wait = true) const {
        if constexpr (!SPILL) {
            if (wait) asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int k = 0; k < 4; ++k) asm volatile("" : "+f"(s[nt][k]));
        }
    }
};

// Memory of a CTA: maxima and sums [nsub][HP], the query's log2-sum-exp [HP],
// factors [P][Hq]; the arrays by token; the warps' queues, whose memory the
// output partials [Hq][D + 4] take over where every warp has one task.  With SPILL
// the arrays by token lie in the workspace, and the scores behind them.
template <bool SPILL>
struct Layout {
    float *max, *sum, *lse, *factor;
    int* loc;      // [TS] row
    int* pos;      // [TS] position in the sequence
    int* src;      // [TS] entry of the selection
    float* scale;  // [2 Hkv][TC], then the heads' weights [groups][TS]
    float* score;  // SPILL
    float* out;
    uint8_t* queue;

    __device__ __forceinline__ Layout(const AttendKernelArgs& a, uint8_t* smem, int P, int HP,
                                      int D, int nwarps, int block) {
        max = reinterpret_cast<float*>(smem);
        sum = max + a.nsub * HP;
        lse = sum + a.nsub * HP;
        factor = lse + HP;
        uint8_t* next = reinterpret_cast<uint8_t*>(factor + ((P * a.Hq + 3) & ~3));
        uint8_t* token = SPILL ? a.spill + (size_t)block * a.token_bytes : next;
        loc = reinterpret_cast<int*>(token);
        pos = loc + a.TS;
        src = pos + a.TS;
        scale = reinterpret_cast<float*>(src + a.TS);
        score = scale + ::max(2 * a.Hkv * a.TC, a.Hkv * a.ngroups * a.TS);
        queue = SPILL ? next : reinterpret_cast<uint8_t*>(score);
        out = reinterpret_cast<float*>(
            a.alias ? queue : queue + (size_t)nwarps * attend_stages(D) * 16 * D);
    }
};

// The cluster's output and weights, from every CTA's maxima, sums and partial
// outputs.  What it needs of the launch is read anew rather than kept in
// registers through the kernel.
template <int D, int NT, bool SPILL>
__device__ __forceinline__ void finish(const AttendKernelArgs& a, uint8_t* smem, int HP, int GP,
                                       int live, uint32_t tmem) {
    int P, rank, block;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(P));
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    asm volatile("mov.u32 %0, %%ctaid.x;" : "=r"(block));
    release_next();
    const int tid = threadIdx.x, nthreads = blockDim.x;
    const Layout<SPILL> at(a, smem, P, HP, D, nthreads >> 5, block);
    const int bs = block / P, b = bs / a.S, st = bs - b * a.S;
    // All ranks' values are on their way before the first is used: a remote load takes long.
    for (int j = tid; j < HP; j += nthreads) {
        const int h = j / GP, i = h * a.G + (j - h * GP);
        if (j - h * GP >= a.G) {
            at.lse[j] = INFINITY;  // a padded head has no weight
            continue;
        }
        float x[kMaxCluster], y[kMaxCluster];
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r) {
            x[r] = r < P ? load_remote(at.max + j, r) : -INFINITY;
            y[r] = r < P ? load_remote(at.sum + j, r) : 0.f;
        }
        float m = -INFINITY, l = 0.f;
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r) m = fmaxf(m, x[r]);
        const float safe = m == -INFINITY ? 0.f : m;
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r) {
            x[r] = exp2_fast(x[r] - safe);
            l += y[r] * x[r];
        }
        const float norm = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r)
            if (r < P) at.factor[r * a.Hq + i] = x[r] * norm;
        const float lse2 = m + log2f(l);
        at.lse[j] = l == 0.f ? INFINITY : lse2;  // weights of an empty query: 0
        if (rank == 0 && a.lse)
            a.lse[(long long)bs * a.Hq + i] = l == 0.f ? -INFINITY : lse2 * 0.69314718056f;
    }
    __syncthreads();
    // A share of the output's quads.  The first one's partial outputs come from the other CTAs
    // while the weights are computed.
    const int quads = a.Hq * (D / 4);
    const int lo = quads * rank / P, hi = quads * (rank + 1) / P;
    float4 y[kMaxCluster / 2];
    auto fetch_quad = [&](int i, int r0) {
#pragma unroll
        for (int r = 0; r < kMaxCluster / 2; ++r)
            if (r0 + r < P) y[r] = load_remote4(at.out + 4 * (i + i / (D / 4)), r0 + r);
    };
    if (lo + tid < hi) fetch_quad(lo + tid, 0);
    if (a.weights || a.acc) {
        // Each task's heads first, then the sum over the tasks in their order.
        const int groups = a.Hkv * a.ngroups, ntasks = groups * a.nsub;
        const int tiles = (live + 15) >> 4, nwarps = nthreads >> 5, warp = tid >> 5;
        const int g = (tid & 31) >> 2, c = tid & 3, t_lo = 4 * (g >> 1) + (g & 1);
        constexpr int F = NT == 0 ? 2 : 1, N = NT == 0 ? 1 : NT;
        for (int task = warp, turn = 0; task < ntasks; task += nwarps, ++turn) {
            const int sub = task / groups, hg = task - sub * groups;
            const int h = hg / a.ngroups, j0 = (hg - h * a.ngroups) * 8 * NT;
            const int tile0 = tiles * sub / a.nsub, n = tiles * (sub + 1) / a.nsub - tile0;
            const Scores<N, SPILL> scores(a, tmem, at.score, warp, nwarps, turn);
            const float* lse = at.lse + h * GP + j0 + column_head<NT>(c);
            float l[N][2];
#pragma unroll
            for (int nt = 0; nt < N; ++nt) l[nt][0] = lse[nt * 8], l[nt][1] = lse[nt * 8 + 1];
            float* dst = at.scale + hg * a.TS + tile0 * 16;
            constexpr int AHEAD = N == 1 ? 4 : 2;  // fragments on their way together
            for (int i0 = 0; i0 < n; i0 += AHEAD * F) {
                float z[AHEAD][N][4], w0[AHEAD], w1[AHEAD];  // tokens t_lo and t_lo + 2
#pragma unroll
                for (int u = 0; u < AHEAD; ++u) scores.load(min(i0 + u * F, n - 1) / F, z[u]);
                scores.loaded(z[0]);
#pragma unroll
                for (int u = 0; u < AHEAD; ++u) {
                    if (u > 0) scores.loaded(z[u], false);
                    w0[u] = w1[u] = 0.f;
#pragma unroll
                    for (int nt = 0; nt < N; ++nt) {
                        w0[u] +=
                            exp2_fast(z[u][nt][0] - l[nt][0]) + exp2_fast(z[u][nt][1] - l[nt][1]);
                        w1[u] +=
                            exp2_fast(z[u][nt][2] - l[nt][0]) + exp2_fast(z[u][nt][3] - l[nt][1]);
                    }
                }
#pragma unroll
                for (int o = 1; o <= (F == 1 ? 2 : 1); o <<= 1) {
#pragma unroll
                    for (int u = 0; u < AHEAD; ++u) {
                        w0[u] += __shfl_xor_sync(0xffffffffu, w0[u], o);
                        w1[u] += __shfl_xor_sync(0xffffffffu, w1[u], o);
                    }
                }
#pragma unroll
                for (int u = 0; u < AHEAD; ++u) {
                    const int tile = i0 + u * F + (F == 1 ? 0 : c >> 1);
                    if (c % (4 / F) == 0 && tile < n) {
                        dst[tile * 16 + t_lo] = w0[u];
                        dst[tile * 16 + t_lo + 2] = w1[u];
                    }
                }
            }
        }
        __syncthreads();
        const long long entry0 = (long long)bs * a.K;
        float* acc = a.acc ? a.acc + (long long)ld(a.req + b) * a.L : nullptr;
        for (int i = tid; i < live; i += nthreads) {
            float w = 0.f;
#pragma unroll 8
            for (int j = 0; j < groups; ++j) w += at.scale[j * a.TS + i];
            if (acc) atomicAdd(acc + at.pos[i], w);
            if (a.weights) a.weights[entry0 + at.src[i]] = w;
        }
    }
    for (int i = lo + tid; i < hi; i += nthreads) {
        const int head = i / (D / 4), d = (i - head * (D / 4)) * 4;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int r0 = 0; r0 < P; r0 += kMaxCluster / 2) {
            if (i != lo + tid || r0 > 0) fetch_quad(i, r0);
#pragma unroll
            for (int r = 0; r < kMaxCluster / 2; ++r) {
                if (r0 + r < P) {
                    const float f = at.factor[(r0 + r) * a.Hq + head];
                    x = make_float4(x.x + y[r].x * f, x.y + y[r].y * f, x.z + y[r].z * f,
                                    x.w + y[r].w * f);
                }
            }
        }
        const long long to = b * a.out_stride[0] + st * a.out_stride[1] + head * a.out_stride[2] + d;
        uint32_t w0, w1;
        if (a.fp16) {
            w0 = pack_half2(x.x, x.y);
            w1 = pack_half2(x.z, x.w);
        } else {
            const __nv_bfloat162 p = __floats2bfloat162_rn(x.x, x.y);
            const __nv_bfloat162 q = __floats2bfloat162_rn(x.z, x.w);
            w0 = *reinterpret_cast<const uint32_t*>(&p);
            w1 = *reinterpret_cast<const uint32_t*>(&q);
        }
        uint16_t* dst = static_cast<uint16_t*>(a.out) + to;
        if (a.vec_out) {
            *reinterpret_cast<uint2*>(dst) = make_uint2(w0, w1);
        } else {
            dst[0] = (uint16_t)w0;
            dst[1] = (uint16_t)(w0 >> 16);
            dst[2] = (uint16_t)w1;
            dst[3] = (uint16_t)(w1 >> 16);
        }
    }
}

template <int CODE, int D, int NT, bool SPILL>
__global__ void __launch_bounds__(32 * attend_warps(D, SPILL), 1)
    attend_kernel(const AttendKernelArgs a) {
    constexpr int F = NT == 0 ? 2 : 1;    // tiles of a fragment
    constexpr int N = NT == 0 ? 1 : NT;   // fragments of a tile
    constexpr int STEPS = D / 16;         // of a score: 16 d each
    constexpr int COPIES = D / 32;    // 16-byte chunks of a tile per lane
    // Entries a thread takes at a time, and their scales held in registers (those of 8 heads);
    // fewer beside wide queries
    constexpr int kTurns = D * N > 128 ? 1 : 2, kHeldScales = D * N > 128 ? 4 : 16;
    constexpr int STAGES = attend_stages(D);
    constexpr uint32_t kTile = 16 * D;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ int s_scan[33];
    __shared__ uint32_t s_tmem;
    cg::cluster_group cluster = cg::this_cluster();
    const int P = (int)cluster.num_blocks();
    const int rank = (int)cluster.block_rank();
    const int bs = blockIdx.x / P;
    const int b = bs / a.S, st = bs - b * a.S;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int nthreads = blockDim.x, nwarps = nthreads >> 5;
    const int g = lane >> 2, c = lane & 3;
    const int GP = a.ngroups * (NT == 0 ? 4 : 8 * NT);  // padded query heads of a K/V head
    const int HP = a.Hkv * GP;
    const Layout<SPILL> at(a, smem, P, HP, D, nwarps, blockIdx.x);
    int *const t_loc = at.loc, *const t_pos = at.pos, *const t_src = at.src;
    float* const t_scale = at.scale;

    if (!SPILL && warp == 0) {
        // Never waits for another CTA of these kernels: a CTA's shared memory is at least its share of
        // the columns, so that those that an SM holds have columns for all.  It does wait for what
        // holds columns otherwise, be it the kernel before this one or one on another stream.
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         shared_address(&s_tmem)),
                     "r"(a.cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    }

    wait_for_previous();
    const int groups = a.Hkv * a.ngroups;
    const int ntasks = groups * a.nsub;
    // Queries as the B operand: lane (g, c) holds elements 16 w + 4 c .. + 3 of head g (g % 4).
    uint32_t qf[N][STEPS][2];
    float factor[N][2];  // of the scores of heads 2 c and 2 c + 1
    auto load_q = [&](int task) {
        const int hg = task % groups, h = hg / a.ngroups, j0 = (hg - h * a.ngroups) * 8 * NT;
#pragma unroll
        for (int nt = 0; nt < N; ++nt) {
            const int j = j0 + nt * 8 + (NT == 0 ? g & 3 : g);
            const long long from = b * a.q_stride[0] + st * a.q_stride[1] +
                                   (long long)(h * a.G + j) * a.q_stride[2];
            uint32_t raw[2 * STEPS];
            load_query<STEPS>(raw, static_cast<const uint16_t*>(a.q) + from, c, j < a.G, a.vec_q);
            float peak = 0.f;
#pragma unroll
            for (int i = 0; i < 2 * STEPS; ++i) {
                const float2 x = pair(raw[i], a.fp16);
                peak = fmaxf(peak, fmaxf(fabsf(x.x), fabsf(x.y)));
            }
            peak = fmaxf(peak, __shfl_xor_sync(0xffffffffu, peak, 1));
            peak = fmaxf(peak, __shfl_xor_sync(0xffffffffu, peak, 2));
            // the head's largest element goes to [2^14, 2^15), f16's top
            int e = (int)(__float_as_uint(peak) >> 23) - 127;
            e = e < -100 ? -100 : e;
            const float up = __uint_as_float((uint32_t)(14 - e + 127) << 23);
#pragma unroll
            for (int i = 0; i < 2 * STEPS; ++i) {
                const float2 x = pair(raw[i], a.fp16);
                qf[nt][i >> 1][i & 1] = pack_half2(x.x * up, x.y * up);
            }
            const float down = __uint_as_float((uint32_t)(e - 14 + 127) << 23) * a.scale_log2;
            factor[nt][0] = __shfl_sync(0xffffffffu, down, 4 * column_head<NT>(c));
            factor[nt][1] = __shfl_sync(0xffffffffu, down, 4 * column_head<NT>(c) + 4);
        }
    };

    // The CTA's entries, kTurns * nthreads at a time (all of them, mostly).  The first are under
    // way while the queries come.
    const long long entry0 = (long long)bs * a.K;
    const int chunks = (a.K + 15) >> 4, own = (chunks - rank + P - 1) / P;
    const int entries = own * 16 - (own > 0 && (chunks - 1) % P == rank ? chunks * 16 - a.K : 0);
    auto entry_of = [&](int i) { return ((i >> 4) * P + rank) * 16 + (i & 15); };
    int loc[kTurns], pos[kTurns];
    auto load_entries = [&](int i0) {
#pragma unroll
        for (int u = 0; u < kTurns; ++u) {
            const int i = i0 + u * nthreads + tid;
            loc[u] = -1, pos[u] = 0;
            if (i < entries) {
                loc[u] = ld(a.locs + entry0 + entry_of(i));
                pos[u] = ld(a.topk + entry0 + entry_of(i));
            }
        }
    };
    load_entries(0);
    const int req = ld(a.req + b);
    if (warp < ntasks) load_q(warp);
    const bool known = req >= 0 && req < a.R;
    // Masked entries are dropped.  A thread fetches the scales of its entries as soon as it has
    // the positions, kHeldScales of each into registers.
    const int per = 2 * a.Hkv;
    const float* scales = a.scales + (long long)(known ? req : 0) * a.NB * per;
    float held[kTurns][kHeldScales];
    int live = 0, at_last[kTurns];
    auto fetch_scales = [&](float (&x)[kHeldScales], int t, int ch) {
        const float* src = scales + (long long)a.block.of(t) * per + ch;
#pragma unroll
        for (int k = 0; k < kHeldScales; k += 4) {
            if (ch + k >= per) break;
            if (a.vec_scale) {
                const float4 v = ld(reinterpret_cast<const float4*>(src + k));
                x[k] = v.x, x[k + 1] = v.y, x[k + 2] = v.z, x[k + 3] = v.w;
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    x[k + i] = ch + k + i < per ? ld(src + k + i) : 0.f;
            }
        }
    };
    auto put_scales = [&](const float (&x)[kHeldScales], int to, int ch) {
#pragma unroll
        for (int k = 0; k < kHeldScales; ++k)
            if (ch + k < per) t_scale[(ch + k) * a.TC + scale_slot(to)] = x[k];
    };
#pragma unroll
    for (int u = 0; u < kTurns; ++u) at_last[u] = -1;
    for (int i0 = 0; i0 < entries; i0 += kTurns * nthreads) {
        int row[kTurns], t[kTurns];
#pragma unroll
        for (int u = 0; u < kTurns; ++u) {
            if (at_last[u] >= 0) put_scales(held[u], at_last[u], 0);  // of the turns before
            const int i = i0 + u * nthreads + tid;
            row[u] = known && loc[u] < a.num_rows && pos[u] >= 0 && pos[u] < a.L ? loc[u] : -1;
            t[u] = pos[u];
            if (row[u] >= 0)
                fetch_scales(held[u], t[u], 0);
            else if (i < entries && a.weights)
                a.weights[entry0 + entry_of(i)] = 0.f;
        }
        load_entries(i0 + kTurns * nthreads);  // the next, if any
#pragma unroll
        for (int u = 0; u < kTurns; ++u) {
            const int left = entries - (i0 + u * nthreads);
            if (left <= 0) break;
            int n = __syncthreads_count(row[u] >= 0);
            int to = live + tid;  // in place while no entry is masked
            if (n != min(nthreads, left))
                to = live + block_exclusive_scan(row[u] >= 0, s_scan, &n);
            at_last[u] = -1;
            if (row[u] >= 0) {
                t_loc[to] = row[u];
                t_pos[to] = t[u];
                t_src[to] = entry_of(i0 + u * nthreads + tid);
                at_last[u] = to;
            }
            live += n;
        }
    }
    const int tiles = (live + 15) >> 4;
    __syncthreads();
    // The places up to a whole tile repeat a live row: their scores are masked and their
    // weights zero.
    for (int i = live + tid; i < tiles * 16; i += nthreads) {
        t_loc[i] = t_loc[live - 1];
        t_pos[i] = t_pos[live - 1];
        for (int ch = 0; ch < per; ++ch) t_scale[ch * a.TC + scale_slot(i)] = 0.f;
    }
    if (!SPILL) asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    __syncthreads();
    const uint32_t tmem = SPILL ? 0u : s_tmem;

    // The warp's queue: item i of a task is the K rows of its tile i, then the V rows of its
    // tile i - n.
    const uint32_t queue = shared_address(at.queue) + warp * STAGES * kTile;
    auto copy_item = [&](int i, int stage, int h, int tile0, int n) {
        if (i < 2 * n) {
            const bool v = i >= n;
            const uint8_t* p = a.rows + (v ? a.Hkv + h : h) * D;
            const int* l = t_loc + (tile0 + (v ? i - n : i)) * 16;
            const uint32_t tile = queue + stage * kTile;
            int from = lane;
            if (D * N > 128) asm volatile("" : "+r"(from));  // offsets computed here, not kept
            // A lane's chunks lie in COPIES consecutive rows, or are dealt out in order where a row's
            // chunks do not divide the lanes.
            constexpr bool kRows = 32 % (D / 16) == 0;
            constexpr int kGroup = kRows && COPIES % 4 == 0 ? 4 : 1;
#pragma unroll
            for (int k0 = 0; k0 < COPIES; k0 += kGroup) {
                int loc[kGroup];
                const int row0 = kRows ? from / (D / 16) * COPIES + k0 : (k0 * 32 + from) / (D / 16);
                const int chunk = (kRows ? from : k0 * 32 + from) % (D / 16);
                if constexpr (kGroup == 4) {
                    const int4 x = *reinterpret_cast<const int4*>(l + row0);
                    loc[0] = x.x, loc[1] = x.y, loc[2] = x.z, loc[3] = x.w;
                } else {
                    loc[0] = l[row0];
                }
#pragma unroll
                for (int k = 0; k < kGroup; ++k)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                                     tile + chunk_at<D>(row0 + k, chunk)),
                                 "l"(p + (long long)loc[k] * a.W + chunk * 16)
                                 : "memory");
            }
        }
        commit_copies();  // of nothing past the last item, so that the count stays even
    };
    auto first_items = [&](int task) {
        const int sub = task / groups, h = (task - sub * groups) / a.ngroups;
        const int tile0 = tiles * sub / a.nsub, n = tiles * (sub + 1) / a.nsub - tile0;
#pragma unroll
        for (int i = 0; i < STAGES - 1; ++i) copy_item(i, i, h, tile0, n);
    };
    if (warp < ntasks) first_items(warp);  // under way while the scales come

#pragma unroll
    for (int u = 0; u < kTurns; ++u)
        if (at_last[u] >= 0) put_scales(held[u], at_last[u], 0);
    if (per > kHeldScales) {  // the others of many heads
        for (int i = tid; i < live; i += nthreads) {
            for (int ch = kHeldScales; ch < per; ch += kHeldScales) {
                fetch_scales(held[0], t_pos[i], ch);
                put_scales(held[0], i, ch);
            }
        }
    }
    __syncthreads();

    for (int task = warp, turn = 0; task < ntasks; task += nwarps, ++turn) {
        const int sub = task / groups, hg = task - sub * groups;
        const int h = hg / a.ngroups, j0 = (hg - h * a.ngroups) * 8 * NT;
        const int tile0 = tiles * sub / a.nsub, n = tiles * (sub + 1) / a.nsub - tile0;
        const float* sk = t_scale + h * a.TC + tile0 * 16;
        const float* sv = t_scale + (a.Hkv + h) * a.TC + tile0 * 16;
        const Scores<N, SPILL> scores(a, tmem, at.score, warp, nwarps, turn);
        if (turn > 0) {
            load_q(task);
            first_items(task);
        }
        int stage = 0;  // of the item in use
        // Item i is in shared memory for the whole warp, and the item before used up: its stage
        // takes the next copy.
        auto next_item = [&](int i) {
            wait_copies<STAGES - 2>();
            __syncwarp();
            copy_item(i + STAGES - 1, stage == 0 ? STAGES - 1 : stage - 1, h, tile0, n);
            const uint32_t tile = queue + stage * kTile;
            stage = stage + 1 == STAGES ? 0 : stage + 1;
            return tile;
        };
        // Tokens of a tile in this lane's score fragments: t_lo and t_lo + 2.
        const int t_lo = 4 * (g >> 1) + (g & 1);
        // This lane's row in the matrices of a K tile (its chunk is lane / 16) and of a V tile.
        const int k_row = 4 * ((lane & 7) >> 1) + (lane & 1) + 2 * (lane >> 3 & 1);
        const int v_row = lane & 15;

        // ---- scores --------------------------------------------------------------
        float top[N][2];   // of heads 2 c and 2 c + 1
        float most[N][2];  // largest of score + log2(V scale)
#pragma unroll
        for (int nt = 0; nt < N; ++nt)
            top[nt][0] = top[nt][1] = most[nt][0] = most[nt][1] = -INFINITY;
        // Columns 0-3 and 4-7 belong to the two tiles of a fragment.
        const uint32_t own[2] = {F == 1 || g < 4 ? ~0u : 0u, g >= 4 ? ~0u : 0u};
        for (int i = 0; i < n; i += F) {
            float z[N][4];  // the products, then the scores
#pragma unroll
            for (int f = 0; f < F; ++f) {
                if (f > 0 && i + f >= n) break;
                const uint32_t tile = next_item(i + f);
                float s[N][2][4] = {};
#pragma unroll
                for (int w = 0; w < STEPS; w += 2) {
                    uint32_t r[4];  // rows t_lo, t_lo + 2 of chunk w, then of chunk w + 1
                    read_matrices(r, tile + chunk_at<D>(k_row, w + (lane >> 4)));
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        uint32_t a0, a1, a2, a3;
                        halves<CODE>(r[2 * k], a0, a2);
                        halves<CODE>(r[2 * k + 1], a1, a3);
#pragma unroll
                        for (int nt = 0; nt < N; ++nt)
                            mma(s[nt][k], a0, a1, a2, a3, qf[nt][w + k][0], qf[nt][w + k][1]);
                    }
                }
#pragma unroll
                for (int nt = 0; nt < N; ++nt)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (f == 0 || c >> 1 == f) z[nt][k] = s[nt][0][k] + s[nt][1][k];
            }
            const int mine = F == 1 ? i : i + (c >> 1);  // the tile of this lane's columns
            const int t0 = (mine < n ? mine : 0) * 16 + t_lo;
            const bool on0 = mine < n && tile0 * 16 + t0 < live;
            const bool on1 = mine < n && tile0 * 16 + t0 + 2 < live;
            const float2 kk = *reinterpret_cast<const float2*>(sk + (mine < n ? mine : 0) * 16 + 2 * g);
            const float k0 = kk.x, k1 = kk.y;
            const float2 vv = *reinterpret_cast<const float2*>(sv + (mine < n ? mine : 0) * 16 + 2 * g);
            const float v0 = log2_fast(vv.x), v1 = log2_fast(vv.y);
#pragma unroll
            for (int nt = 0; nt < N; ++nt) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float f = factor[nt][k];
                    z[nt][k] = on0 ? z[nt][k] * (k0 * f) : -INFINITY;
                    z[nt][k + 2] = on1 ? z[nt][k + 2] * (k1 * f) : -INFINITY;
                    top[nt][k] = fmaxf(top[nt][k], fmaxf(z[nt][k], z[nt][k + 2]));
                    most[nt][k] = fmaxf(most[nt][k], fmaxf(z[nt][k] + v0, z[nt][k + 2] + v1));
                }
            }
            scores.store(i / F, z);
        }

        // The queries are used up; without this the compiler keeps them for the next turn, which
        // loads its own.
#pragma unroll
        for (int nt = 0; nt < N; ++nt)
#pragma unroll
            for (int w = 0; w < STEPS; ++w) asm("" : "=r"(qf[nt][w][0]), "=r"(qf[nt][w][1]));

        // ---- softmax over the task's tokens ----------------------------------------
        scores.stored();
        float safe[N][2], sum[N][2];
        // What brings the head's largest product of P and V scale to 2^15; where registers are
        // short, in the place of the head's sum, which comes after.
        constexpr bool kUpShared = D * N > 192 && N > 1;
        float up[N][2];
        float* const up_at = at.sum + sub * HP + h * GP + j0 + column_head<NT>(c);
#pragma unroll
        for (int nt = 0; nt < N; ++nt) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                top[nt][k] = max_over_g(top[nt][k]);
                most[nt][k] = max_over_g(most[nt][k]);
                if (F == 2) {  // the head's other tiles
                    top[nt][k] = fmaxf(top[nt][k], __shfl_xor_sync(0xffffffffu, top[nt][k], 2));
                    most[nt][k] = fmaxf(most[nt][k], __shfl_xor_sync(0xffffffffu, most[nt][k], 2));
                }
                if (g == 0)
                    at.max[sub * HP + h * GP + j0 + nt * 8 + column_head<NT>(c) + k] = top[nt][k];
                safe[nt][k] = top[nt][k] == -INFINITY ? 0.f : top[nt][k];
                up[nt][k] = exp2_fast(fminf(fmaxf(15.f - (most[nt][k] - safe[nt][k]), -126.f), 126.f));
                if (kUpShared && g == 0) up_at[nt * 8 + k] = up[nt][k];
                sum[nt][k] = 0.f;
            }
        }

        // ---- values --------------------------------------------------------------
        float o[STEPS][N][4] = {};
        for (int i = 0; i < n; i += F) {
            float z[N][4];
            scores.load(i / F, z);
            const int mine = F == 1 ? i : i + (c >> 1) < n ? i + (c >> 1) : i;
            uint32_t tile = next_item(n + i);
            scores.loaded(z);
            // the scales last, for the registers
            const float2 vv = *reinterpret_cast<const float2*>(sv + mine * 16 + 2 * g);
            const float v0 = vv.x, v1 = vv.y;
            uint32_t pf[N][2];
#pragma unroll
            for (int nt = 0; nt < N; ++nt) {
                const float p0 = exp2_fast(z[nt][0] - safe[nt][0]);
                const float p1 = exp2_fast(z[nt][1] - safe[nt][1]);
                const float p2 = exp2_fast(z[nt][2] - safe[nt][0]);
                const float p3 = exp2_fast(z[nt][3] - safe[nt][1]);
                sum[nt][0] += p0 + p2;
                sum[nt][1] += p1 + p3;
                // P first: the V scale may be any of 32 bits' where P is 0
                float2 u;
                if constexpr (kUpShared)
                    u = *reinterpret_cast<const float2*>(up_at + nt * 8);
                else
                    u = make_float2(up[nt][0], up[nt][1]);
                pf[nt][0] = transpose(pack_half2(p0 * u.x * v0, p1 * u.y * v0));
                pf[nt][1] = transpose(pack_half2(p2 * u.x * v1, p3 * u.y * v1));
            }
#pragma unroll
            for (int f = 0; f < F; ++f) {
                if (f > 0 && i + f >= n) break;
                if (f > 0) tile = next_item(n + i + f);
#pragma unroll
                for (int w = 0; w < STEPS; w += 2) {
                    // d = g, g + 8 of chunk w, then of chunk w + 1; four tokens each
                    uint32_t r[4];
                    read_transposed(r, tile + chunk_at<D>(v_row, w + (lane >> 4)));
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        uint32_t a0, a1, a2, a3;
                        halves<CODE>(r[2 * k], a0, a2);
                        halves<CODE>(r[2 * k + 1], a1, a3);
#pragma unroll
                        for (int nt = 0; nt < N; ++nt) {
                            uint32_t b0 = pf[nt][0], b1 = pf[nt][1];
                            if (F == 2) b0 &= own[f], b1 &= own[f];
                            mma(o[w + k][nt], a0, a1, a2, a3, b0, b1);
                        }
                    }
                }
            }
        }
        if constexpr (F == 2) {  // both tiles' columns of a head
#pragma unroll
            for (int w = 0; w < STEPS; ++w)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    o[w][0][k] += __shfl_xor_sync(0xffffffffu, o[w][0][k], 2);
        }
        int ranks = P;  // the layout anew, so that it takes no registers through the loops
        asm("" : "+r"(ranks));
        const Layout<SPILL> done(a, smem, ranks, HP, D, nwarps, blockIdx.x);
        float fold[N][2];
        if (kUpShared) __syncwarp();  // with no tile, nothing came between
#pragma unroll
        for (int nt = 0; nt < N; ++nt) {
#pragma unroll
            for (int k = 0; k < 2; ++k)
                fold[nt][k] = reciprocal_fast(
                    kUpShared ? done.sum[sub * HP + h * GP + j0 + nt * 8 + column_head<NT>(c) + k]
                              : up[nt][k]);
        }
        if (kUpShared) __syncwarp();
#pragma unroll
        for (int nt = 0; nt < N; ++nt) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                sum[nt][k] = sum_over_g(sum[nt][k]);
                if (F == 2) sum[nt][k] += __shfl_xor_sync(0xffffffffu, sum[nt][k], 2);
                if (g == 0)
                    done.sum[sub * HP + h * GP + j0 + nt * 8 + column_head<NT>(c) + k] =
                        sum[nt][k];
            }
        }
        // The outputs may take the queues' place: then every warp has one task, and all are done
        // with their queues here.  Several parts of a slice have one task a warp too; their
        // outputs are added in order, relative to their common maximum.
        if (a.alias || a.nsub > 1) __syncthreads();
#pragma unroll
        for (int nt = 0; nt < N; ++nt) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                if (a.nsub > 1) {
                    const int to = h * GP + j0 + nt * 8 + column_head<NT>(c) + k;
                    float m = -INFINITY;
                    for (int u = 0; u < a.nsub; ++u) m = fmaxf(m, done.max[u * HP + to]);
                    fold[nt][k] *=
                        exp2_fast(done.max[sub * HP + to] - (m == -INFINITY ? 0.f : m));
                }
            }
        }
        for (int u = 0; u < a.nsub; ++u) {
            if (u == sub) {
#pragma unroll
                for (int nt = 0; nt < N; ++nt) {
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int j = j0 + nt * 8 + 2 * c + k;
                        if (j >= a.G || (F == 2 && c > 1)) continue;
                        const float f = fold[nt][k];
                        float* row = done.out + (h * a.G + j) * (D + 4) + g;
#pragma unroll
                        for (int w = 0; w < STEPS; ++w) {
                            const float y0 = o[w][nt][k] * f, y1 = o[w][nt][k + 2] * f;
                            row[16 * w] = u > 0 ? row[16 * w] + y0 : y0;
                            row[16 * w + 8] = u > 0 ? row[16 * w + 8] + y1 : y1;
                        }
                    }
                }
            }
            if (a.nsub > 1) __syncthreads();
        }
    }
    if (a.nsub > 1) {  // one maximum and sum per head of the slice
        for (int i = tid; i < HP; i += nthreads) {
            float m = -INFINITY, l = 0.f;
            for (int u = 0; u < a.nsub; ++u) m = fmaxf(m, at.max[u * HP + i]);
            const float safe = m == -INFINITY ? 0.f : m;
            for (int u = 0; u < a.nsub; ++u)
                l += at.sum[u * HP + i] * exp2_fast(at.max[u * HP + i] - safe);
            at.max[i] = m;
            at.sum[i] = l;
        }
    }

    // ---- the cluster's result ----------------------------------------------------
    cluster.sync();
    finish<D, NT, SPILL>(a, smem, HP, GP, live, tmem);
    if (!SPILL) asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    cluster.sync();  // no CTA leaves while another reads its shared memory
    if (!SPILL && warp == 0) {
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                     "r"(a.cols));
    }
}

// Opens the kernel to shared memory of this size and to clusters of P.
template <int CODE, int D, int NT, bool SPILL>
cudaError_t open_kernel(int P, size_t smem) {
    static SmemOptIn opt;
    auto* kernel = attend_kernel<CODE, D, NT, SPILL>;
    const cudaError_t e = ensure_smem(kernel, smem, &opt);
    if (e != cudaSuccess || P <= 8) return e;
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
}

template <int CODE, int D, int NT, bool SPILL>
cudaError_t run_one(const AttendShape& sh, cudaStream_t s) {
    const cudaError_t e = open_kernel<CODE, D, NT, SPILL>(sh.P, sh.smem);
    if (e != cudaSuccess) return e;
    return launch_chained(attend_kernel<CODE, D, NT, SPILL>, sh.a.B * sh.a.S * sh.P, sh.threads,
                          sh.smem, sh.P, s, sh.a);
}

template <int CODE, int D>
cudaError_t run_dim(const AttendShape& sh, cudaStream_t s) {
    if (sh.spill) return run_one<CODE, D, 1, true>(sh, s);
    if constexpr (D <= 192)
        if (sh.nt == 0) return run_one<CODE, D, 0, false>(sh, s);
    if constexpr (D <= 128)
        if (sh.nt == 2) return run_one<CODE, D, 2, false>(sh, s);
    return run_one<CODE, D, 1, false>(sh, s);
}

template <int CODE>
cudaError_t run(const AttendShape& sh, int D, cudaStream_t s) {
    switch (D) {
        case 32: return run_dim<CODE, 32>(sh, s);
        case 64: return run_dim<CODE, 64>(sh, s);
        case 96: return run_dim<CODE, 96>(sh, s);
        case 128: return run_dim<CODE, 128>(sh, s);
        case 192: return run_dim<CODE, 192>(sh, s);
        case 256: return run_dim<CODE, 256>(sh, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace attend

#endif  // __CUDACC__

}  // namespace hs
