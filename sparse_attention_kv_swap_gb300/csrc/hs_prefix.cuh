// Attention over prefixes that requests of a batch share (sm_103a); the contract is
// hs_attend_prefix's in include/hisparse_swap.h.
//
// The queries of all requests of a prefix that read one K/V head are the rows of two matrix products
// with that head's keys and values, and each tile of these is read once for up to 256 rows.  One
// CTA an SM; the work is a list of units, one unit being a tile of tokens for a tile of rows of a
// K/V head, and every CTA takes an equal run of consecutive ones, so that few rows over a long
// prefix and many rows over a short one fill the SMs alike.  Rows whose units fell to several
// CTAs are put together by a second kernel (combine_kernel, hs_prefix.cu).
//
// Warps of a CTA, which hand tiles of 64 tokens to one another by barriers in shared memory:
//   copies (1)      the codes of a K/V head, to rings in shared memory (TMA)
//   scales (1)      the tokens' scales
//   converters (4 for keys, 4 for values)   write codes as f16 in the layout of the matrix instructions
//                   (128-byte swizzle).  Codes are exact in f16.
//   matrix (1 for each of the NPIPE pipelines)   S = Q K^T (128 rows x 64 tokens) and O += P V by
//                   tcgen05.mma, accumulators and P in tensor memory
//   softmax (8 for each pipeline)   a thread has half a row (32 tokens): it reads S, writes P over it
// Two pipelines (D <= 128) hold rows 0-127 and 128-255 of a row tile, or, where it has 128 rows or fewer,
// the even and the odd tiles of tokens of the same rows.  Each has two places for S: the scores of
// the next tile are there when the softmax of one is done, and its product with V runs beside
// the softmax of the next.
//
// Numbers: a query is scaled by a power of two into f16's range, as in hs_attend.  With z = s log2(e)
// and v_t the V scale, the row keeps one reference r:
//   p_t = 2^(z_t - r),  l = sum p_t,  P_t = f16(p_t v_t),  O = sum P_t code_t,  out = O / l
// r is chosen so that the largest p_t v_t so far lies between 2^9 and 2^16 (r grows only when that
// is passed, and O and l are scaled then): f16 keeps its 11 bits down to 2^-23 of the largest term and
// is off by 2^-34 of it below.  Where V scales differ by 2^88 and more, r stays within 100
// of the largest z, so that l stays in range.
//
// What bounds it (e4m3, D = 128, 8 K/V heads, both kernels): 64 requests of 8 query heads a K/V head
// over 32768 shared tokens take 83 us, 0.83 PFLOP/s, 1.0 us a tile of an SM; 2 requests of 4 over 131072
// take 86 us, 3.1 TB/s, 0.6 us a tile.  That is mostly what it takes to hand a tile on from role to
// role: with the work of all roles left out (a version of 86 and 89 us) 59 and 58 stayed, and without the
// conversions, the softmax, the copies or nearly all matrix instructions alone 2 to 5 were saved.  (A
// warp for all 64 tokens of its rows, with half as many softmax warps, made the second call 4% slower, the
// first 1.5% faster.)  27 and 22 us of these calls do not grow with their length: launches, the first tile's
// way through the roles, partial outputs of every SM and their joining.  The smallest call, a tile an SM
// at most and few parts, takes 12.
#pragma once

#include <cuda.h>

#include "hs_step.cuh"

namespace hs {

constexpr int kPrefixCtas = 256;  // at most

struct PrefixArgs {
    const uint16_t* q;
    uint16_t* out;
    int32_t fp16, B, S, G, Hq, Hkv, R, L, NB, W, P;
    Divisor block;     // by block_tokens
    int32_t even;      // block_tokens is a multiple of 16 and sm_scale >= 0
    float scale_log2;  // |sm_scale| * log2(e)
    float k_sign;      // its sign
    int64_t q_stride[3], out_stride[3], join_stride[3];
    int32_t vec_q, vec_out, vec_join;
    const uint8_t* rows;
    const float* scales;
    const int32_t* prefix;
    const int32_t* lens;
    const int32_t* starts;
    float* lse;
    const uint16_t* join;
    const float* join_lse;
    int32_t ctas;
    float* part;       // [ctas][2][D / 4][rows of a tile][4] outputs
    float2* part_sum;  // [ctas][2][rows of a tile] (r, l)
    float* part_join;  // [ctas][2][rows of a tile] the row's given lse, where lse is that itself
};

constexpr int prefix_pipes(int D) { return D <= 128 ? 2 : 1; }
constexpr int prefix_panels(int D) { return (D + 63) / 64; }

// The store as the copies see it: [R][L][W] bytes, in boxes of so many tokens and bytes of a head.
constexpr int prefix_box(int D) { return D % 128 == 0 ? 128 : D % 64 == 0 ? 64 : 32; }

cudaError_t prefix_run_e4m3(const PrefixArgs& a, const CUtensorMap& map, int D, cudaStream_t s);
cudaError_t prefix_run_int8(const PrefixArgs& a, const CUtensorMap& map, int D, cudaStream_t s);

#ifdef __CUDACC__

namespace prefix {

// Tiles of `each` tokens for n: n may be 2^31 - 1.
__device__ __forceinline__ int tiles_of(int n, int each) {
    return (int)(((uint32_t)n + each - 1) / each);
}

// The prefixes of a call and their units.
struct Plan {
    int32_t lo[HS_MAX_PREFIXES], hi[HS_MAX_PREFIXES];  // batch rows
    int32_t len[HS_MAX_PREFIXES], req[HS_MAX_PREFIXES];  // tokens, and the store's request
    int32_t unit[HS_MAX_PREFIXES + 1];  // first unit; units of a prefix: [K/V head][row tile][tile]
};

// Filled by one warp; everyone else waits at the caller's barrier.  From L2: combine_kernel comes here
// before it waits.
__device__ __forceinline__ void fill_plan(Plan& plan, const PrefixArgs& a, int rows, int tokens) {
    const int lane = threadIdx.x & 31;
    int taken = 0;          // batch rows of the prefixes before
    int units = 0;
    for (int p0 = 0; p0 < a.P; p0 += 32) {
        const int p = p0 + lane;
        int first = 0, end = 0, len = 0, r = 0;
        if (p < a.P) {
            first = min(max(__ldcg(a.starts + p), 0), a.B);
            end = max(min(max(__ldcg(a.starts + p + 1), 0), a.B), first);
            r = __ldcg(a.prefix + p);
            len = r < 0 || r >= a.R ? 0 : min(max(__ldcg(a.lens + p), 0), a.L);
        }
        int most = max(end, taken);  // the largest end up to this prefix
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, most, o);
            if (lane >= o) most = max(most, x);
        }
        int before = __shfl_up_sync(0xffffffffu, most, 1);
        if (lane == 0) before = taken;
        const int lo = max(first, before), hi = max(end, lo);
        int mine = 0;  // the launcher has made sure that all fit 31 bits
        if (p < a.P && len > 0)
            mine = a.Hkv * (((hi - lo) * a.S * a.G + rows - 1) / rows) * tiles_of(len, tokens);
        int sum = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += x;
        }
        if (p < a.P) {
            plan.lo[p] = lo;
            plan.hi[p] = hi;
            plan.len[p] = len;
            plan.req[p] = r;
            plan.unit[p] = units + sum - mine;
        }
        units += __shfl_sync(0xffffffffu, sum, 31);
        taken = __shfl_sync(0xffffffffu, most, 31);
    }
    if (lane == 0) plan.unit[a.P] = units;
}

// CTAs with work: each has a unit or more.
__device__ __forceinline__ int working(int units, int ctas) { return min(units, ctas); }
// First unit of CTA `cta` of `n` that work.
__device__ __forceinline__ int first_unit(int units, int cta, int n) {
    return units / n * cta + min(cta, units % n);
}

// Consecutive units of one tile of rows.
struct Segment {
    int p, h, row0, rows;  // prefix, K/V head, first row of the tile, rows of the prefix
    int tile0, n, tiles;   // tiles of tokens: the first, how many, all of the prefix
    __device__ __forceinline__ Segment(const Plan& plan, const PrefixArgs& a, int from, int to,
                                       int tile_rows, int tile_tokens) {
        p = a.P - 1;
        while (plan.unit[p] > from) --p;  // the last one that begins here or before: not empty
        rows = (plan.hi[p] - plan.lo[p]) * a.S * a.G;
        tiles = tiles_of(plan.len[p], tile_tokens);
        const int at = from - plan.unit[p];
        const int turn = at / tiles, row_tiles = (rows + tile_rows - 1) / tile_rows;
        tile0 = at - turn * tiles;
        h = turn / row_tiles;
        row0 = (turn - h * row_tiles) * tile_rows;
        n = min(tiles - tile0, to - from);
    }
};

__device__ __forceinline__ uint32_t shared_address(const void* p) {
    return (uint32_t)__cvta_generic_to_shared(p);
}

// ---- barriers in shared memory --------------------------------------------------

__device__ __forceinline__ void barrier_init(uint32_t bar, int count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// True once the phase of this parity is over; the thread sleeps for up to 20 us before it says no.
// (Without the time it comes back at once, and the waiting warps' loops take half of the others' issue
// slots.)
__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n"
        " selp.u32 %0, 1, 0, p;\n}"
        : "=r"(done)
        : "r"(bar), "r"(parity), "r"(20000)
        : "memory");
    return done != 0;
}

// Waits for the phase of this parity, with a limit that no wait comes near (about a second): then,
// or once another thread has given up, the CTA goes on without waiting and its outputs become
// NaN.
constexpr int kTries = 1 << 16;
__device__ __forceinline__ void wait_slow(uint32_t bar, uint32_t parity, volatile int* gave_up) {
#pragma unroll 1
    for (int i = 0; i < kTries; ++i)
        if (try_wait(bar, parity) || *gave_up) return;
    *gave_up = 1;
}
// The same where a thread must not go on, whoever has given up.
__device__ __forceinline__ void wait_still(uint32_t bar, uint32_t parity) {
#pragma unroll 1
    for (int i = 0; i < kTries && !try_wait(bar, parity); ++i) {
    }
}
__device__ __forceinline__ void wait(uint32_t bar, uint32_t parity, volatile int* gave_up) {
    if (!try_wait(bar, parity)) wait_slow(bar, parity, gave_up);
}

// ---- tensor memory and matrix instructions -----------------------------------------

__device__ __forceinline__ void load_columns(uint32_t (&x)[32], uint32_t at) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
        "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, "
        "%28, %29, %30, %31}, [%32];"
        : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]), "=r"(x[4]), "=r"(x[5]), "=r"(x[6]),
          "=r"(x[7]), "=r"(x[8]), "=r"(x[9]), "=r"(x[10]), "=r"(x[11]), "=r"(x[12]), "=r"(x[13]),
          "=r"(x[14]), "=r"(x[15]), "=r"(x[16]), "=r"(x[17]), "=r"(x[18]), "=r"(x[19]),
          "=r"(x[20]), "=r"(x[21]), "=r"(x[22]), "=r"(x[23]), "=r"(x[24]), "=r"(x[25]),
          "=r"(x[26]), "=r"(x[27]), "=r"(x[28]), "=r"(x[29]), "=r"(x[30]), "=r"(x[31])
        : "r"(at)
        : "memory");
}
__device__ __forceinline__ void load_columns(uint32_t (&x)[16], uint32_t at) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
        "%11, %12, %13, %14, %15}, [%16];"
        : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]), "=r"(x[4]), "=r"(x[5]), "=r"(x[6]),
          "=r"(x[7]), "=r"(x[8]), "=r"(x[9]), "=r"(x[10]), "=r"(x[11]), "=r"(x[12]), "=r"(x[13]),
          "=r"(x[14]), "=r"(x[15])
        : "r"(at)
        : "memory");
}
// The loaded values may be used after this.
template <int N>
__device__ __forceinline__ void loaded(uint32_t (&x)[N]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+r"(x[i]));
}
__device__ __forceinline__ void store_columns(uint32_t at, const uint32_t (&x)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
        "%11, %12, %13, %14, %15, %16};" ::"r"(at),
        "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7]),
        "r"(x[8]), "r"(x[9]), "r"(x[10]), "r"(x[11]), "r"(x[12]), "r"(x[13]), "r"(x[14]),
        "r"(x[15])
        : "memory");
}
__device__ __forceinline__ void stored() {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// What this thread has written to shared memory, or seen written by others, is seen by the matrix
// instructions that follow: this thread's, or those of threads that it lets go after.  It waits for
// this thread's loads: the converters, which always have some under way, leave it to the warp
// that issues (with theirs, a tile took 5000 cycles).
__device__ __forceinline__ void fence_shared() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// One lane of a whole warp.
__device__ __forceinline__ bool elected() {
    uint32_t x;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}"
                 : "=r"(x));
    return x != 0;
}

// Descriptor of a matrix in shared memory with the 128-byte swizzle: rows of 128 bytes, eight to a
// group of 1024; `lead` is the distance of panels of 64 elements where the rows run along the
// product's sum (V), and unused where they run along its result (Q, K).
__device__ __forceinline__ uint64_t matrix(uint32_t at, uint32_t lead) {
    return (uint64_t)((at & 0x3ffff) >> 4) | (uint64_t)(lead >> 4) << 16 |
           (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

// f16 by f16 into f32, 128 rows and n columns; B by columns of the sum if `rows_of_sum`.
constexpr uint32_t instruction(int n, bool rows_of_sum) {
    return 1u << 4 | (rows_of_sum ? 1u << 16 : 0u) | (uint32_t)(n >> 3) << 17 | (128u >> 4) << 24;
}

__device__ __forceinline__ void multiply(uint32_t d, uint64_t a, uint64_t b, uint32_t kind,
                                         bool add) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(kind), "r"((uint32_t)add)
        : "memory");
}
__device__ __forceinline__ void multiply_tensor(uint32_t d, uint32_t a, uint64_t b, uint32_t kind,
                                                bool add) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
        "r"(a), "l"(b), "r"(kind), "r"((uint32_t)add)
        : "memory");
}
// The barrier gets an arrival once the matrix instructions that this thread has issued are done.
__device__ __forceinline__ void commit(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
        : "memory");
}

// ---- arithmetic ------------------------------------------------------------------

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 pair(uint32_t w, int fp16) {
    if (fp16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ uint32_t unpair(float a, float b, int fp16) {
    if (fp16) return pack_half2(a, b);
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// Eight 16-bit elements.
__device__ __forceinline__ uint4 load8(const uint16_t* p, bool vec) {
    if (vec) return ld(reinterpret_cast<const uint4*>(p));
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = (uint32_t)ld(p + 2 * i) | (uint32_t)ld(p + 2 * i + 1) << 16;
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint2 load4(const uint16_t* p, bool vec) {
    if (vec) return ld(reinterpret_cast<const uint2*>(p));
    return make_uint2((uint32_t)ld(p) | (uint32_t)ld(p + 1) << 16,
                      (uint32_t)ld(p + 2) | (uint32_t)ld(p + 3) << 16);
}
__device__ __forceinline__ void store4(uint16_t* p, uint32_t a, uint32_t b, bool vec) {
    if (vec) {
        *reinterpret_cast<uint2*>(p) = make_uint2(a, b);
    } else {
        p[0] = (uint16_t)a, p[1] = (uint16_t)(a >> 16);
        p[2] = (uint16_t)b, p[3] = (uint16_t)(b >> 16);
    }
}

// The codes in the low and the high half of a word, as two f16 pairs.
template <int CODE>
__device__ __forceinline__ void halves(uint32_t w, uint32_t& lo, uint32_t& hi) {
    if constexpr (CODE == HS_KV_E4M3) {
        __half2 x, y;
        decode_halves(w, x, y);
        lo = *reinterpret_cast<const uint32_t*>(&x);
        hi = *reinterpret_cast<const uint32_t*>(&y);
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

// Place of 8 elements (16 bytes) in a matrix of rows of 128 bytes, 64 elements to a panel.
__device__ __forceinline__ uint32_t place(int row, int d, int panel_bytes) {
    return (uint32_t)(d / 64 * panel_bytes + row * 128 + (((d % 64) / 8 ^ (row & 7)) << 4));
}

// A query row: batch row, step, head.
struct Row {
    int b, s, head;
    __device__ __forceinline__ Row(const PrefixArgs& a, int first, int h, int r) {
        const int sg = a.S * a.G, m = r / sg, rest = r - m * sg;
        b = first + m;
        s = rest / a.G;
        head = h * a.G + rest - s * a.G;
    }
    __device__ __forceinline__ long long at(const int64_t (&stride)[3]) const {
        return b * stride[0] + s * stride[1] + head * stride[2];
    }
};

// How a row's own attention over the prefix, of log2-sum-exp `lse2` (-inf: none), is joined
// with the given one: the factors of both outputs and the lse.
struct Joined {
    float mine, other, lse;
    // `o`: the given lse, -inf without one.
    __device__ __forceinline__ Joined(float lse2, float o) {
        const float e = lse2 * 0.69314718056f;
        mine = lse2 == -INFINITY ? 0.f : 1.f;
        other = 0.f;
        lse = e;
        if (o == -INFINITY) return;
        const float top = fmaxf(e, o);
        const float x = expf(e - top), y = expf(o - top), sum = x + y;
        mine = x / sum;
        other = y / sum;
        lse = top + logf(sum);
    }
};

// The largest p_t v_t gets 2^kTop when the reference is set, and may grow by 2^kRoom from there.
constexpr float kTop = 9.5f, kRoom = 6.f;

// The product with V that a pipeline issued last; none in the first tile of a segment.
struct Product {
    uint32_t done, parity;
    bool none;
    volatile int* gave_up;
};

// The two warps that share rows, a half of a tile's tokens (and of O's columns) each.
struct Twins {
    int id;                // named barrier
    float* mine;           // this row's places in shared memory
    const float* other;
    __device__ __forceinline__ void sync() const {
        asm volatile("bar.sync %0, 64;" ::"r"(id) : "memory");
    }
    // Whether x holds for a row of either warp.
    __device__ __forceinline__ bool any(bool x) const {
        uint32_t y;
        asm volatile(
            "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.or.pred q, %2, 64, p;\n"
            " selp.u32 %0, 1, 0, q;\n}"
            : "=r"(y)
            : "r"((uint32_t)x), "r"(id)
            : "memory");
        return y != 0;
    }
    // The larger of both halves'.  A barrier must come before the next call.
    __device__ __forceinline__ float larger(float x) const {
        *mine = x;
        sync();
        return fmaxf(x, *other);
    }
};

// The reference moves to what the halves want, if one of them has outgrown it: O and l with it.  Both
// warps call it, once a tile, with their S in registers: P may be written over S after it.
template <int D>
__device__ __forceinline__ void move_reference(uint32_t o_col, float want, const Product& before,
                                               const Twins& twins, float& ref, float& l) {
    if (!twins.any(before.none || want > ref + kRoom)) return;
    want = twins.larger(want);
    if (before.none) {
        ref = want;
        return;
    }
    const bool grow = want > ref + kRoom;
    const float step = grow ? ref - want : 0.f;
    const float by = exp2_fast(step);  // 0 under 2^-126: so little of O does not show beside the new term
    // l, of terms up to 2^106, may still count then: by two factors that are not 0
    const float root = exp2_fast(0.5f * step);
    l = step < -125.f ? l * root * root : l * by;
    if (grow) ref = want;
    wait(before.done, before.parity, before.gave_up);
    fence_after();
#pragma unroll 1
    for (int c = 0; c < D / 2; c += 16) {
        uint32_t x[16];
        load_columns(x, o_col + c);
        loaded(x);
#pragma unroll
        for (int k = 0; k < 16; ++k) x[k] = __float_as_uint(__uint_as_float(x[k]) * by);
        store_columns(o_col + c, x);
    }
}

// Half a tile of a row: S is replaced by P.  Any scales and any number of live tokens.
template <int D>
__device__ __forceinline__ void softmax_any(uint32_t s_col, uint32_t p_col, uint32_t o_col, float f,
                                            const float* s_k, const float* s_v, const float* s_log,
                                            int live, const Product& before, const Twins& twins,
                                            float& ref, float& l) {
    uint32_t x[32];
    load_columns(x, s_col);
    loaded(x);
    // The largest score, and the largest of score + log2(V scale).
    float top = -INFINITY, most = -INFINITY;
#pragma unroll
    for (int k = 0; k < 32; k += 4) {
        const float4 ks = *reinterpret_cast<const float4*>(s_k + k);
        const float4 lg = *reinterpret_cast<const float4*>(s_log + k);
        const float kk[4] = {ks.x, ks.y, ks.z, ks.w}, ll[4] = {lg.x, lg.y, lg.z, lg.w};
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const float z = __uint_as_float(x[k + m]) * kk[m] * f;
            x[k + m] = __float_as_uint(z);
            if (k + m < live) {
                most = fmaxf(most, z + ll[m]);
                top = fmaxf(top, z);
            }
        }
    }
    move_reference<D>(o_col, fmaxf(most - kTop, top - 100.f), before, twins, ref, l);
    uint32_t y[16];
#pragma unroll
    for (int k = 0; k < 32; k += 4) {
        const float4 vs = *reinterpret_cast<const float4*>(s_v + k);
        const float vv[4] = {vs.x, vs.y, vs.z, vs.w};
        float e[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            e[m] = exp2_fast(__uint_as_float(x[k + m]) - ref);
            if (k + m >= live) e[m] = 0.f;
            l += e[m];
            e[m] *= vv[m];
        }
        y[k / 2] = pack_half2(e[0], e[1]);
        y[k / 2 + 1] = pack_half2(e[2], e[3]);
    }
    store_columns(p_col, y);
}

// a * b + c for two pairs at once.
__device__ __forceinline__ float2 fma_pair(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n .reg .b64 a, b, c, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n"
        " mov.b64 c, {%6, %7};\n fma.rn.f32x2 d, a, b, c;\n mov.b64 {%0, %1}, d;\n}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 add_pair(float2 a, float2 b) {
    float2 d;
    asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n"
        " add.rn.f32x2 d, a, b;\n mov.b64 {%0, %1}, d;\n}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// The same for whole tiles whose scales are equal in each 16 tokens, V scales of 2^-60 to 2^50,
// with none above in the segment so far, and K scales >= 0: the scales leave the loops.  p_t v_t comes
// out of the exponential at once, 2^(z_t + log2 v - r), and l takes the sum of 16 by 1 / v.  r is
// at most the largest z plus 50 - kTop then, so that a token whose weight counts in l, z_t no less than
// the largest by 25, has an exponent above -126: no weight is flushed to 0 before it is divided by v.
struct Even {  // of 16 tokens each: factor of the products, log2 of the V scale, its reciprocal
    float k[2], log[2], inverse[2];
    __device__ __forceinline__ Even(const float4* s_even, float f) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float4 x = s_even[i];
            k[i] = x.x * f, log[i] = x.y, inverse[i] = x.z;
        }
    }
};
template <int D>
__device__ __forceinline__ void softmax_even(uint32_t s_col, uint32_t p_col, uint32_t o_col,
                                             const Even& scale, const Product& before,
                                             const Twins& twins, float& ref, float& l) {
    uint32_t x[32];
    load_columns(x, s_col);
    loaded(x);
    float most = -INFINITY;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t* z = x + 16 * h;
        float m[4];  // four chains
#pragma unroll
        for (int k = 0; k < 4; ++k)
            m[k] = fmaxf(fmaxf(__uint_as_float(z[k]), __uint_as_float(z[k + 4])),
                         fmaxf(__uint_as_float(z[k + 8]), __uint_as_float(z[k + 12])));
        m[0] = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
        most = fmaxf(most, fmaf(m[0], scale.k[h], scale.log[h]));
    }
    move_reference<D>(o_col, most - kTop, before, twins, ref, l);
    uint32_t w[16];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const float k0 = scale.k[h], o0 = scale.log[h] - ref;
        const float2 kk = make_float2(k0, k0), off = make_float2(o0, o0);
        float2 sum[2] = {};
#pragma unroll
        for (int k = 0; k < 16; k += 2) {
            float2 e = make_float2(__uint_as_float(x[16 * h + k]),
                                   __uint_as_float(x[16 * h + k + 1]));
            e = fma_pair(e, kk, off);
            e.x = exp2_fast(e.x);
            e.y = exp2_fast(e.y);
            sum[k / 2 & 1] = add_pair(sum[k / 2 & 1], e);
            w[8 * h + k / 2] = pack_half2(e.x, e.y);
        }
        sum[0] = add_pair(sum[0], sum[1]);
        l = fmaf(sum[0].x + sum[0].y, scale.inverse[h], l);
    }
    store_columns(p_col, w);
}

// ---- the kernel -------------------------------------------------------------------

// Tiles of f16 in place, for keys and for values each: as many as leave room for rings of three.
constexpr int prefix_pool(int D) { return D == 256 ? 1 : D == 192 ? 2 : D > 64 ? 3 : 4; }

template <int D>
struct Shape {
    static constexpr int kPipes = prefix_pipes(D), kTok = kPrefixTokens;
    static constexpr int kPanels = prefix_panels(D);
    static constexpr int kRows = kPrefixRows * kPipes;          // of a tile
    static constexpr int kQ = kPanels * kPrefixRows * 128;      // bytes of a pipeline's queries
    static constexpr int kTile = kPanels * kTok * 128;          // of a tile's keys or values
    static constexpr int kScales = 4;                           // scales of tiles in place
    static constexpr int kSoftmax = 8 * kPipes, kConvert = 4;   // warps; kConvert of keys, and of values
    static constexpr int kControl = kSoftmax + 2 * kConvert;    // first of 4: matrix (2), copies, scales
    static constexpr int kThreads = 32 * (kControl + 4);
    static constexpr int kBox = prefix_box(D);
    static constexpr int kRaw = kTok * D;                       // bytes of a tile's codes, K or V
    static constexpr int kPool = prefix_pool(D);
    static constexpr int kF16 = kPipes * kQ + 2 * kPool * kTile;
    static constexpr int kFit = (209 * 1024 - kF16) / (2 * kRaw);
    static constexpr int kRing = kFit < 8 ? kFit : 8;           // tiles in the rings
    static_assert(kRing >= 2, "one is used, one on its way");
    static constexpr int kSmem = kF16 + 2 * kRing * kRaw + 1024;  // aligned by the kernel
    static constexpr int kChunks = kTok * D / 16 / (32 * kConvert);  // of 16 codes a converter
    // Registers of a thread: what the block is launched with, then each role's share.  A quarter of an SM
    // holds two warps of each pipeline, two converters and one of the others.
    static constexpr int kLaunchRegs = kPipes == 2 ? 72 : 96;
    static constexpr int kSoftmaxRegs = kPipes == 2 ? 88 : 104;
    static constexpr int kConvertRegs = kPipes == 2 ? 48 : 88, kControlRegs = kPipes == 2 ? 56 : 88;
    static_assert(2 * kPipes * kSoftmaxRegs + 2 * kConvertRegs + kControlRegs <=
                      (2 * kPipes + 3) * kLaunchRegs,
                  "a share beyond what was launched would wait for ever");
    static constexpr int kOut = 2 * kPipes * kTok;              // tensor-memory column of O
    static_assert(kOut + kPipes * D <= 512, "tensor memory");
};

// The outputs of a segment, and the partial ones of a segment that is not a whole tile: called by
// all softmax warps together.  `done`: the barrier of this pipeline's product (0: it had no tile).
template <int D>
__device__ __forceinline__ void finish(const PrefixArgs& a, const Plan& plan, uint8_t* smem,
                                       float2* s_sum, uint32_t o_col, int from, int u0, int u1,
                                       int row, int p, int half, const Twins& sums, float ref,
                                       float l, uint32_t done, uint32_t parity,
                                       volatile int* gave_up) {
    using X = Shape<D>;
    constexpr int NP = X::kPipes, kQuads = D / 4;
    const Segment g(plan, a, from, u1, X::kRows, X::kTok);
    const bool both = NP == 2 && g.rows - g.row0 > kPrefixRows;
    const bool whole = g.n == g.tiles;
    const int r = g.row0 + (both ? p * kPrefixRows : 0) + row;
    const bool on = r < g.rows;
    const Row at(a, plan.lo[g.p], g.h, on ? r : g.row0);
    if (done) {
        wait(done, parity, gave_up);
        fence_after();
    }
    if (*gave_up) l = NAN;
    // the halves' sums, added in the same order by both
    *sums.mine = l;
    sums.sync();
    l = half ? *sums.other + l : l + *sums.other;
    sums.sync();
    o_col += half * (D / 2);
    const int d0 = half * (D / 2);  // this half's columns
    const bool alive = r - (row & 31) < g.rows;  // the warp has rows
    // Two halves of the tokens: of a whole tile, the second pipeline's go through the queries' memory;
    // else each is a part of its own.
    float4* const second = reinterpret_cast<float4*>(smem) + row * kQuads;
    float mine_by = 1.f, second_by = 0.f;
    const bool join = NP == 2 && !both && whole;
    if (join) {
        asm volatile("bar.sync 9, 512;" ::: "memory");  // both are done with the queries
        if (p == 1) {
            if (half == 0) s_sum[row] = make_float2(ref, l);
            if (done && alive) {
#pragma unroll 1
                for (int c = 0; c < D / 2; c += 16) {
                    uint32_t x[16];
                    load_columns(x, o_col + c);
                    loaded(x);
#pragma unroll
                    for (int k = 0; k < 4; ++k)  // rotated by the row: different banks
                        second[((d0 + c) / 4 + k + row) % kQuads] = make_float4(
                            __uint_as_float(x[4 * k]), __uint_as_float(x[4 * k + 1]),
                            __uint_as_float(x[4 * k + 2]), __uint_as_float(x[4 * k + 3]));
                }
            }
        }
        asm volatile("bar.sync 9, 512;" ::: "memory");
        if (p == 0 && g.n > 1) {
            const float2 o = s_sum[row];
            const float top = fmaxf(ref + log2f(l), o.x + log2f(o.y));
            mine_by = exp2_fast(ref - top);
            second_by = exp2_fast(o.x - top);
            l = l * mine_by + o.y * second_by;
            ref = top;
        }
    }
    if (alive && (!join || p == 0)) {
        const long long out_row = ((long long)at.b * a.S + at.s) * a.Hq + at.head;
        float other = 0.f;
        if (whole) {
            const Joined j(ref + log2f(l), a.join ? ld(a.join_lse + out_row) : -INFINITY);
            const float by = j.mine / l;
            mine_by *= by;
            second_by *= by;
            other = j.other;
            // both halves have read the given one, which may lie in the same place
            sums.sync();
            if (on && a.lse && half == 0) a.lse[out_row] = j.lse;
        }
        const long long slot = 2 * (long long)blockIdx.x + (from == u0 ? 0 : 1);
        const int tile_row = p * kPrefixRows + row;
        float4* part = reinterpret_cast<float4*>(a.part) + slot * kQuads * X::kRows + tile_row;
        // without a tile: nothing, whatever the reference
        if (!whole && on && half == 0) {
            const long long place = slot * X::kRows + tile_row;
            a.part_sum[place] = make_float2(done ? ref : -INFINITY, l);
            if (a.join && a.lse == a.join_lse) a.part_join[place] = ld(a.join_lse + out_row);
        }
        if (!whole && !done) return;
        uint16_t* out = a.out + at.at(a.out_stride);
        const uint16_t* others = a.join + at.at(a.join_stride);
#pragma unroll 1
        for (int c = 0; c < D / 2; c += 16) {
            uint32_t x[16];
            load_columns(x, o_col + c);
            loaded(x);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float y[4];
#pragma unroll
                for (int m = 0; m < 4; ++m) y[m] = __uint_as_float(x[4 * k + m]) * mine_by;
                if (join && g.n > 1) {
                    const float4 z = second[((d0 + c) / 4 + k + row) % kQuads];
                    y[0] += z.x * second_by, y[1] += z.y * second_by;
                    y[2] += z.z * second_by, y[3] += z.w * second_by;
                }
                if (!on) continue;
                const int d = d0 + c + 4 * k;
                if (!whole) {
                    part[(long long)(d / 4) * X::kRows] = make_float4(y[0], y[1], y[2], y[3]);
                    continue;
                }
                if (other > 0.f) {
                    const uint2 z = load4(others + d, a.vec_join);
                    const float2 z0 = pair(z.x, a.fp16), z1 = pair(z.y, a.fp16);
                    y[0] += z0.x * other, y[1] += z0.y * other;
                    y[2] += z1.x * other, y[3] += z1.y * other;
                }
                store4(out + d, unpair(y[0], y[1], a.fp16), unpair(y[2], y[3], a.fp16), a.vec_out);
            }
        }
    }
    if (join) asm volatile("bar.sync 9, 512;" ::: "memory");
}

// Barriers in shared memory.
enum Bar : int {
    kQFull = 0,      // [pipe] the queries of a segment
    kSFull = 2,      // [pipe][place] scores, by the matrix instructions
    kPFull = 6,      // [pipe][place]
    kPvDone = 10,    // [pipe] a product with V
    kKFull = 12, kVFull = 16, kKEmpty = 20, kVEmpty = 24,   // [kPool] f16 tiles
    kRawFull = 28, kRawEmpty = 44,                          // [keys, values][8] codes
    kScFull = 60, kScEmpty = 68,                            // [pipe][kScales]
    kOFull = 76,     // [pipe] the products of a segment: kPvDone alone could not tell the last from the
                     // one before the last but one
    kDone = 78, kBars = 79
};

template <int CODE, int D>
__global__ void __launch_bounds__(Shape<D>::kThreads, 1)
    prefix_kernel(const PrefixArgs a, const __grid_constant__ CUtensorMap map) {
    using X = Shape<D>;
    constexpr int NP = X::kPipes, TOK = X::kTok;
    extern __shared__ uint8_t smem_raw[];
    __shared__ Plan plan;
    // Scales of the tiles of each pipeline.
    struct Scales {
        float k[TOK], v[TOK], log[TOK];  // log2 of the V scale
        float4 even[TOK / 16];           // of 16 tokens: K, log2 V, 1 / V
        int each;                        // the tokens' own are to be used
    };
    __shared__ __align__(16) Scales s_scales[NP][X::kScales];
    __shared__ __align__(8) unsigned long long s_bar[kBars];
    __shared__ float2 s_sum[kPrefixRows];  // of the second pipeline
    __shared__ float s_half[2][NP][2][kPrefixRows];  // what halves of rows tell one another; their sums
    __shared__ uint32_t s_tmem;
    __shared__ int s_gave_up;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint8_t* const smem = smem_raw + (-(int)shared_address(smem_raw) & 1023);
    const uint32_t q_at = shared_address(smem), k_at = q_at + NP * X::kQ;
    const uint32_t v_at = k_at + X::kPool * X::kTile, raw_at = v_at + X::kPool * X::kTile;
    const uint32_t bars = shared_address(s_bar);
    auto bar = [&](int i) { return (uint32_t)(bars + 8 * i); };

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            barrier_init(bar(kQFull + i), 8);
            barrier_init(bar(kPvDone + i), 1);
            barrier_init(bar(kOFull + i), 1);
        }
        for (int i = 0; i < 4; ++i) {
            barrier_init(bar(kSFull + i), 1);
            barrier_init(bar(kPFull + i), 8);
            barrier_init(bar(kKFull + i), X::kConvert);
            barrier_init(bar(kVFull + i), X::kConvert);
            barrier_init(bar(kKEmpty + i), NP);
            barrier_init(bar(kVEmpty + i), NP);
            for (int p = 0; p < 2; ++p) {
                barrier_init(bar(kScFull + 4 * p + i), 1);
                barrier_init(bar(kScEmpty + 4 * p + i), 8);
            }
        }
        for (int i = 0; i < 16; ++i) {
            barrier_init(bar(kRawFull + i), 1);
            barrier_init(bar(kRawEmpty + i), X::kConvert);
        }
        barrier_init(bar(kDone), NP);
        s_gave_up = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == X::kControl) {
        // One CTA an SM; waits for what else holds tensor memory, never the other way round.
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                         shared_address(&s_tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        fence_before();
    }
    wait_for_previous();
    if (warp == X::kControl + 1) fill_plan(plan, a, X::kRows, TOK);
    __syncthreads();
    fence_after();
    const uint32_t tmem = s_tmem;
    const int units = plan.unit[a.P];
    const int ctas = working(units, a.ctas);
    const bool works = (int)blockIdx.x < ctas;
    const int u0 = works ? first_unit(units, blockIdx.x, ctas) : 0;
    const int u1 = works ? first_unit(units, blockIdx.x + 1, ctas) : 0;
    const int count = u1 - u0;  // tiles of this CTA, numbered from 0
    volatile int* const gave_up = &s_gave_up;

    if (warp >= X::kControl) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(X::kControlRegs));
        const int role = warp - X::kControl;
        if (role < NP) {
            // ---- matrix instructions: the whole warp goes along, one lane issues ---------------
            constexpr uint32_t kScores = instruction(TOK, false), kValues = instruction(D, true);
            const int p = role;
            const bool leader = elected();
            const uint32_t base = __shfl_sync(0xffffffffu, tmem, 0);
            uint32_t done = 0, segments = 0;  // items and segments before
            // Each pipeline releases every tile, one of the other's as soon as it is there: the barriers'
            // phases then tell tiles apart, for nobody is two behind or ahead.
            int k_next = 0, v_next = 0;
            auto pass = [&](int full, int empty, int& next, int to) {
                for (; NP == 2 && next < to; ++next) {
                    const int place = next % X::kPool;
                    wait(bar(full) + 8 * place, next / X::kPool & 1, gave_up);
                    if (leader) arrive(bar(empty) + 8 * place);
                    __syncwarp();
                }
            };
            for (int from = u0; from < u1;) {
                const Segment g(plan, a, from, u1, X::kRows, TOK);
                const int n = __shfl_sync(0xffffffffu, g.n, 0);
                const bool both =
                    __shfl_sync(0xffffffffu, (int)(NP == 2 && g.rows - g.row0 > kPrefixRows), 0);
                const bool shared = NP == 2 && !both;  // the pipelines take turns
                const int items = shared ? (n + 1 - p) / 2 : n, first = from - u0 + (shared ? p : 0);
                if (items > 0) wait(bar(kQFull + p), segments++ & 1, gave_up);
                for (int k = 0; k < items + 2; ++k) {
                    if (k >= 2) {  // O += P V of two items before
                        const uint32_t it = done + k - 2;
                        const int t = first + (shared ? 2 : 1) * (k - 2);
                        const int place = t % X::kPool;
                        pass(kVFull, kVEmpty, v_next, t);
                        v_next = t + 1;
                        wait(bar(kVFull) + 8 * place, t / X::kPool & 1, gave_up);
                        wait(bar(kPFull + 2 * p) + 8 * (it & 1), it >> 1 & 1, gave_up);
                        fence_shared();
                        fence_after();
                        const uint64_t b = matrix(v_at + place * X::kTile, TOK * 128);
                        const uint32_t s = base + (2 * p + (it & 1)) * TOK;
                        if (leader) {
#pragma unroll
                            for (int i = 0; i < TOK / 16; ++i)  // 16 tokens are 16 rows of 128 bytes
                                multiply_tensor(base + X::kOut + p * D, s + 8 * i,
                                                b + i * (2048 >> 4), kValues, i > 0 || k > 2);
                            commit(bar(kVEmpty) + 8 * place);
                            commit(bar(kPvDone + p));
                            if (k == items + 1) commit(bar(kOFull + p));
                        }
                        __syncwarp();
                    }
                    if (k < items) {  // S = Q K^T, where P of two items before has been
                        const uint32_t it = done + k;
                        const int t = first + (shared ? 2 : 1) * k;
                        const int place = t % X::kPool;
                        pass(kKFull, kKEmpty, k_next, t);
                        k_next = t + 1;
                        wait(bar(kKFull) + 8 * place, t / X::kPool & 1, gave_up);
                        fence_shared();
                        fence_after();
                        const uint64_t q = matrix(q_at + p * X::kQ, 16);
                        const uint64_t key = matrix(k_at + place * X::kTile, 16);
                        const uint32_t s = base + (2 * p + (it & 1)) * TOK;
                        if (leader) {
#pragma unroll
                            for (int i = 0; i < D / 16; ++i) {
                                const int panel = i / 4, in = i % 4 * 32;
                                multiply(s, q + ((panel * kPrefixRows * 128 + in) >> 4),
                                         key + ((panel * TOK * 128 + in) >> 4), kScores, i > 0);
                            }
                            commit(bar(kSFull + 2 * p) + 8 * (it & 1));
                            commit(bar(kKEmpty) + 8 * place);
                        }
                        __syncwarp();
                    }
                }
                pass(kKFull, kKEmpty, k_next, from - u0 + n);
                pass(kVFull, kVEmpty, v_next, from - u0 + n);
                done += items;
                from += n;
            }
            if (leader) commit(bar(kDone));
            __syncwarp();
            wait_still(bar(kDone), 0);
        } else if (role == 2) {
            // ---- copies ------------------------------------------------------------------
            const bool leader = elected();
            int tile = 0, end = 0, x = 0, r = 0, slot = 0;
            uint32_t free = 1;  // phase of the ring's places
            for (int i = 0; i < count; ++i) {
                if (++tile >= end) {
                    const Segment g(plan, a, u0 + i, u1, X::kRows, TOK);
                    tile = g.tile0;
                    end = g.tile0 + g.n;
                    x = g.h * D;
                    r = plan.req[g.p];
                }
#pragma unroll
                for (int side = 0; side < 2; ++side) {  // keys, values
                    wait(bar(kRawEmpty + 8 * side) + 8 * slot, free, gave_up);
                    const uint32_t full = bar(kRawFull + 8 * side) + 8 * slot;
                    if (leader) {
                        asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(
                                         full),
                                     "n"(X::kRaw)
                                     : "memory");
#pragma unroll
                        for (int k = 0; k < D / X::kBox; ++k)
                            asm volatile(
                                "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::"
                                "complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
                                    raw_at + (side * X::kRing + slot) * X::kRaw +
                                    k * TOK * X::kBox),
                                "l"(&map), "r"(full), "r"(x + side * a.Hkv * D + k * X::kBox),
                                "r"(tile * TOK), "r"(r)
                                : "memory");
                    }
                    __syncwarp();
                }
                if (++slot == X::kRing) slot = 0, free ^= 1;
            }
            // No copy is under way when the CTA ends, even if a wait was given up.
            for (int i = max(0, count - X::kRing); i < count; ++i)
                for (int side = 0; side < 2; ++side)
                    wait_still(bar(kRawFull + 8 * side) + 8 * (i % X::kRing), i / X::kRing & 1);
        } else if (role == 3) {
            // ---- scales --------------------------------------------------------------------
            // The lanes take 8 tiles at once, 4 groups of 16 tokens each; the next 8 are on their way
            // meanwhile.  Letting a tile go waits for the loads that are under way: with a load
            // for each tile, and every token's scales written, this warp alone took 1500 cycles a tile.
            // Tiles whose scales differ within a group, or are not all there, get every token's.
            int items[2] = {0, 0};  // of each pipeline
            for (int from = u0; from < u1;) {
                bool even = a.even;  // no V scale of the segment has been beyond softmax_even so far
                const Segment g(plan, a, from, u1, X::kRows, TOK);
                const int len = plan.len[g.p], first = g.tile0, n = g.n;
                const bool both = NP == 1 || g.rows - g.row0 > kPrefixRows;
                const float* const scales =
                    a.scales + (long long)plan.req[g.p] * a.NB * 2 * a.Hkv + g.h;
                auto load = [&](uint32_t token, float& k, float& v) {  // those ahead pass 2^31
                    k = v = 0.f;
                    if (token < (uint32_t)len) {
                        const float* at = scales + (long long)a.block.of((int)token) * 2 * a.Hkv;
                        k = ld(at);
                        v = ld(at + a.Hkv);
                    }
                };
                float k, v, next_k, next_v;
                load((uint32_t)first * TOK + lane * 16, next_k, next_v);
                for (int c = 0; c < n; c += 8) {
                    k = next_k, v = next_v;
                    load((uint32_t)(first + c + 8) * TOK + lane * 16, next_k, next_v);
                    const unsigned small = __ballot_sync(0xffffffffu, v < 0x1p-60f);
                    even = even && !__any_sync(0xffffffffu, v > 0x1p50f);
                    const float4 group = make_float4(k * a.k_sign, log2f(v), __frcp_rn(v), 0.f);
                    const int stop = min(8, n - c);
#pragma unroll 1
                    for (int j = 0; j < stop; ++j) {
                        const int tile = first + c + j;
                        const bool each = !even || small >> (4 * j) & 15 || len - tile * TOK < TOK;
#pragma unroll
                        for (int p = 0; p < NP; ++p) {
                            if (!both && ((c + j) & 1) != p) continue;
                            const int sc = items[p] % X::kScales;
                            wait(bar(kScEmpty + 4 * p) + 8 * sc, (items[p] / X::kScales & 1) ^ 1,
                                 gave_up);
                            Scales& s = s_scales[p][sc];
                            if (lane >> 2 == j) s.even[lane & 3] = group;
                            if (lane == 0) s.each = each;
                            if (each) {
#pragma unroll
                                for (int h = 0; h < TOK; h += 32) {
                                    float one_k, one_v;
                                    load((uint32_t)tile * TOK + h + lane, one_k, one_v);
                                    s.k[h + lane] = one_k * a.k_sign;
                                    s.v[h + lane] = one_v;
                                    s.log[h + lane] = log2f(one_v);
                                }
                            }
                            __syncwarp();
                            if (lane == 0) arrive(bar(kScFull + 4 * p) + 8 * sc);
                            ++items[p];
                        }
                    }
                }
                from += n;
            }
        }
    } else if (warp >= X::kSoftmax) {
        // ---- converters ------------------------------------------------------------------
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(X::kConvertRegs));
        const int side = warp >= X::kSoftmax + X::kConvert;  // 0: keys, 1: values
        const int t = tid % (32 * X::kConvert);
        constexpr int kRowChunks = D / 16;  // 16-byte pieces of a token
        const uint32_t raws = raw_at + side * X::kRing * X::kRaw;
        const uint32_t tiles = side ? v_at : k_at;
        int tile = 0, end = 0, len = 0, slot = 0, place_of = 0;
        uint32_t full = 0, free = 1;  // phases of the ring's and of the f16 tiles' places
        for (int i = 0; i < count; ++i) {
            if (++tile >= end) {
                const Segment g(plan, a, u0 + i, u1, X::kRows, TOK);
                tile = g.tile0;
                end = g.tile0 + g.n;
                len = plan.len[g.p];
            }
            const int live = len - tile * TOK;  // codes of tokens from here on count as zeros
            const uint32_t raw = raws + slot * X::kRaw, to = tiles + place_of * X::kTile;
            const uint32_t raw_full = bar(kRawFull + 8 * side) + 8 * slot;
            const uint32_t empty = bar(side ? kVEmpty : kKEmpty) + 8 * place_of;
            // both are asked at once: an answer takes some 100 cycles
            const bool have = try_wait(raw_full, full), may = try_wait(empty, free);
            if (!have) wait_slow(raw_full, full, gave_up);
            if (!may) wait_slow(empty, free, gave_up);
            // Eight lanes take one piece of eight rows: what they read and store together lies in
            // different banks.
            constexpr int kGroup = X::kChunks % 4 == 0 ? 4 : X::kChunks % 2 == 0 ? 2 : 1;
#pragma unroll
            for (int c0 = 0; c0 < X::kChunks; c0 += kGroup) {
                uint4 x[kGroup];
#pragma unroll
                for (int c = 0; c < kGroup; ++c) {
                    const int j = (c0 + c) * 32 * X::kConvert + t;
                    const int row = j / (8 * kRowChunks) * 8 + j % 8, piece = j / 8 % kRowChunks;
                    constexpr int kIn = X::kBox / 16;  // pieces of a box's row
                    const int swizzle =
                        X::kBox == 128 ? row & 7 : X::kBox == 64 ? row >> 1 & 3 : row >> 2 & 1;
                    const uint32_t at = raw + piece / kIn * (TOK * X::kBox) + row * X::kBox +
                                        ((piece % kIn ^ swizzle) << 4);
                    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(x[c].x), "=r"(x[c].y), "=r"(x[c].z), "=r"(x[c].w)
                                 : "r"(at)
                                 : "memory");
                }
#pragma unroll
                for (int c = 0; c < kGroup; ++c) {
                    const int j = (c0 + c) * 32 * X::kConvert + t;
                    const int row = j / (8 * kRowChunks) * 8 + j % 8, piece = j / 8 % kRowChunks;
                    if (live < TOK && row >= live) x[c] = make_uint4(0, 0, 0, 0);
                    uint32_t y[8];
                    halves<CODE>(x[c].x, y[0], y[1]);
                    halves<CODE>(x[c].y, y[2], y[3]);
                    halves<CODE>(x[c].z, y[4], y[5]);
                    halves<CODE>(x[c].w, y[6], y[7]);
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                                     to + place(row, piece * 16, TOK * 128)),
                                 "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3])
                                 : "memory");
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                                     to + place(row, piece * 16 + 8, TOK * 128)),
                                 "r"(y[4]), "r"(y[5]), "r"(y[6]), "r"(y[7])
                                 : "memory");
                }
            }
            __syncwarp();
            if (lane == 0) {
                arrive(bar(side ? kVFull : kKFull) + 8 * place_of);
                arrive(bar(kRawEmpty + 8 * side) + 8 * slot);
            }
            if (++slot == X::kRing) slot = 0, full ^= 1;
            if (++place_of == X::kPool) place_of = 0, free ^= 1;
        }
    } else {
        // ---- softmax ---------------------------------------------------------------
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(X::kSoftmaxRegs));
        const int p = warp / 8, half = warp / 4 & 1, row = tid % kPrefixRows;
        const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);
        const uint32_t o_col = lanes + X::kOut + p * D;
        const Twins twins = {1 + 4 * p + (warp & 3), &s_half[0][p][half][row],
                           &s_half[0][p][half ^ 1][row]};
        uint32_t done = 0, segments = 0;  // items and segments (with items) before
        for (int from = u0; from < u1;) {
            const Segment g(plan, a, from, u1, X::kRows, TOK);
            const bool both = NP == 2 && g.rows - g.row0 > kPrefixRows;
            const bool shared = NP == 2 && !both;  // the pipelines take turns
            const int first = from - u0 + (shared ? p : 0), stop = from - u0 + g.n;
            const int step = shared ? 2 : 1;
            const int r = g.row0 + (both ? p * kPrefixRows : 0) + row;
            const bool on = r < g.rows;
            // Warps without rows leave theirs as they are: a row's products are its own.
            const bool alive = r - lane < g.rows;
            // less TOK a tile of the CTA; may pass 2^31
            const uint32_t rest = plan.len[g.p] + (uint32_t)(from - u0 - g.tile0) * TOK;
            float f = 0.f;  // of the products
            if (first < stop) {
                // The row's largest element goes to [2^14, 2^15), f16's top.
                const Row at(a, plan.lo[g.p], g.h, on ? r : g.row0);
                const uint16_t* q = a.q + at.at(a.q_stride) + half * (D / 2);
                uint4 x[D / 16];
#pragma unroll
                for (int i = 0; i < D / 16; ++i) x[i] = make_uint4(0, 0, 0, 0);
                if (on && a.vec_q) {  // all on their way together
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) x[i] = load8(q + 8 * i, true);
                } else if (on) {
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) x[i] = load8(q + 8 * i, false);
                }
                float peak = 0.f;
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float2 y = pair(w[k], a.fp16);
                        peak = fmaxf(peak, fmaxf(fabsf(y.x), fabsf(y.y)));
                    }
                }
                peak = twins.larger(peak);
                int e = (int)(__float_as_uint(peak) >> 23) - 127;
                e = e < -100 ? -100 : e;
                const float up = __uint_as_float((uint32_t)(14 - e + 127) << 23);
                f = __uint_as_float((uint32_t)(e - 14 + 127) << 23) * a.scale_log2;
                if (alive) {
                    const uint32_t to = q_at + p * X::kQ;
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) {
                        uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float2 y = pair(w[k], a.fp16);
                            w[k] = pack_half2(y.x * up, y.y * up);
                        }
                        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                                         to + place(row, half * (D / 2) + 8 * i, kPrefixRows * 128)),
                                     "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                                     : "memory");
                    }
                }
                fence_shared();
                __syncwarp();
                if (lane == 0) arrive(bar(kQFull + p));
            }
            float ref = 0.f, l = 0.f;
            for (int t = first; t < stop; t += step, ++done) {
                const int sc = done % X::kScales;
                const uint32_t sc_full = bar(kScFull + 4 * p) + 8 * sc;
                const uint32_t s_full = bar(kSFull + 2 * p) + 8 * (done & 1);
                // both are asked at once: an answer takes some 100 cycles
                const bool have = try_wait(sc_full, done / X::kScales & 1);
                const bool there = try_wait(s_full, done >> 1 & 1);
                if (!have) wait_slow(sc_full, done / X::kScales & 1, gave_up);
                if (!there) wait_slow(s_full, done >> 1 & 1, gave_up);
                const Scales& scales = s_scales[p][sc];
                fence_after();
                if (alive) {
                    const uint32_t s_col = lanes + (2 * p + (done & 1)) * TOK;
                    const uint32_t mine = s_col + half * 32, to = s_col + half * 16;
                    // The product before, which may still be adding to O; the one before that is done, for
                    // these scores were issued behind it.
                    const Product before = {bar(kPvDone + p), (done + 1) & 1, t == first, gave_up};
                    const int live = (int)(rest - (uint32_t)t * TOK);  // tokens of the tile, or more
                    if (!scales.each)
                        softmax_even<D>(mine, to, o_col + half * (D / 2),
                                        Even(scales.even + 2 * half, f), before, twins, ref, l);
                    else
                        softmax_any<D>(mine, to, o_col + half * (D / 2), f, scales.k + 32 * half,
                                       scales.v + 32 * half, scales.log + 32 * half,
                                       live - 32 * half, before, twins, ref, l);
                }
                stored();
                fence_before();
                __syncwarp();
                if (lane == 0) {
                    arrive(bar(kPFull + 2 * p) + 8 * (done & 1));
                    arrive(bar(kScEmpty + 4 * p) + 8 * sc);
                }
            }

            // ---- the segment's outputs ---------------------------------------------------
            // What they need of the segment is read anew, so that it takes no registers in the loop.
            int anew = from, row_anew = row;
            const Twins sums = {twins.id, &s_half[1][p][half][row], &s_half[1][p][half ^ 1][row]};
            asm volatile("" : "+r"(anew), "+r"(row_anew));
            if (from + g.n >= u1) release_next();
            finish<D>(a, plan, smem, s_sum, o_col, anew, u0, u1, row_anew, p, half,
                      sums, ref, l,
                      first < stop ? bar(kOFull + p) : 0u, segments & 1, gave_up);
            segments += first < stop;
            from += g.n;
        }
    }
    if (warp >= X::kSoftmax) release_next();
    __syncwarp();
    fence_before();
    __syncthreads();
    if (warp == X::kControl) {
        __syncwarp();
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
    }
}

template <int CODE, int D>
cudaError_t run_one(const PrefixArgs& a, const CUtensorMap& map, cudaStream_t s) {
    static SmemOptIn opt;
    cudaError_t e = ensure_smem(prefix_kernel<CODE, D>, Shape<D>::kSmem, &opt);
    if (e != cudaSuccess) return e;
    // The roles' shares are there only if the compiler has used the whole launch bound.
    static std::atomic<int> regs{0};
    int n = regs.load(std::memory_order_relaxed);
    if (n == 0) {
        cudaFuncAttributes attr;
        e = cudaFuncGetAttributes(&attr, prefix_kernel<CODE, D>);
        if (e != cudaSuccess) return e;
        n = attr.numRegs;
        regs.store(n, std::memory_order_relaxed);
    }
    if (n != Shape<D>::kLaunchRegs) return cudaErrorInvalidConfiguration;
    return launch_chained(prefix_kernel<CODE, D>, a.ctas, Shape<D>::kThreads, Shape<D>::kSmem, 0, s,
                          a, map);
}

template <int CODE>
cudaError_t run(const PrefixArgs& a, const CUtensorMap& map, int D, cudaStream_t s) {
    switch (D) {
        case 32: return run_one<CODE, 32>(a, map, s);
        case 64: return run_one<CODE, 64>(a, map, s);
        case 96: return run_one<CODE, 96>(a, map, s);
        case 128: return run_one<CODE, 128>(a, map, s);
        case 192: return run_one<CODE, 192>(a, map, s);
        case 256: return run_one<CODE, 256>(a, map, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace prefix

#endif  // __CUDACC__

}  // namespace hs
