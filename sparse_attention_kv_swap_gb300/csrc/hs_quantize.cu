// Quantisation of keys and values into 8-bit rows with a scale for each block
// of tokens and head, and the compaction of a sequence after an eviction
// (sm_103a).  Layouts and rounding rules: include/hisparse_swap.h.
//
// A scale group is the D values of T tokens of one (block, K or V, head).  One
// CTA owns one group: it holds the group's values in registers, takes their
// largest magnitude (one block reduction), turns it into the scale and stores
// the codes, so that the input is read once and the codes are written once.
// Both kernels are bound by memory traffic: 3 bytes per element to quantise
// 16-bit values, 2 to compact.  4 x 8192 tokens of 8 heads of 128 in blocks of
// 64 are quantised from bf16 in 32 us, 6.2 TB/s (66 us from addresses that
// do not allow 16-byte loads); 64 x 2048 such rows are compacted in 97 us,
// 5.5 TB/s, from 128-byte pieces anywhere in the source (int8: 109 us, bound by
// instructions).
#include <type_traits>

#include "hs_kv.cuh"

namespace hs {
namespace {

// Thread tid of a group works on part tid % parts of the tokens tid / parts, + step, + 2 * step, ..:
// a part is 16 elements (16 bytes of codes).  A thread keeps kHeld parts in registers (half as many of
// 32-bit input); groups too large for that at the most threads read the rest twice.
constexpr int kHeld = 4;
constexpr int kQuantizeThreads = 448;  // two such CTAs an SM leave 72 registers a thread
constexpr int kCompactThreads = 512;

// Threads of a group of so many tokens, whole warps: the fewest whose registers hold it.  More leave
// each too few loads on their way, fewer read twice.  4 x 8192 tokens, 8 heads of 128, bf16, with 32,
// 64, 128 and 256 threads: 53, 42, 32 and 49 us in blocks of 64 tokens, 32, 43, 70 and 143 of 16;
// 256 and 448 threads in blocks of 256: 49 and 44.  Compaction of 64 x 2048 tokens of that row
// with 64, 128 and 256: 131, 97 and 149 us in blocks of 64; 256 and 512 in blocks of 256: 137 and 112.
int group_threads(int tokens, int parts, int held, int most) {
    const int step = (tokens + held - 1) / held;
    const long long threads = ((long long)step * parts + 31) / 32 * 32;
    return threads < most ? (int)threads : most;
}

// 16 consecutive input elements, as loaded.
template <int DTYPE>
struct Raw {
    static constexpr int kVecs = DTYPE == HS_DTYPE_FP32 ? 4 : 2;
    uint4 v[kVecs];

    __device__ __forceinline__ void load(const void* base, long long at, bool vec) {
        if (vec) {
            const uint4* p = reinterpret_cast<const uint4*>(
                static_cast<const uint8_t*>(base) + at * (DTYPE == HS_DTYPE_FP32 ? 4 : 2));
#pragma unroll
            for (int i = 0; i < kVecs; ++i) v[i] = ld_once_v4(p + i);
        } else {
            uint32_t w[4 * kVecs];
#pragma unroll
            for (int i = 0; i < 4 * kVecs; ++i) {
                if constexpr (DTYPE == HS_DTYPE_FP32) {
                    w[i] = static_cast<const uint32_t*>(base)[at + i];
                } else {
                    const uint16_t* p = static_cast<const uint16_t*>(base) + at + 2 * i;
                    w[i] = (uint32_t)p[0] | ((uint32_t)p[1] << 16);
                }
            }
#pragma unroll
            for (int i = 0; i < kVecs; ++i)
                v[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        }
    }

    // Elements 4 * i .. 4 * i + 3.
    __device__ __forceinline__ void get(int i, float (&x)[4]) const {
        if constexpr (DTYPE == HS_DTYPE_FP32) {
            x[0] = __uint_as_float(v[i].x);
            x[1] = __uint_as_float(v[i].y);
            x[2] = __uint_as_float(v[i].z);
            x[3] = __uint_as_float(v[i].w);
        } else {
            const uint32_t lo = i & 1 ? v[i >> 1].z : v[i >> 1].x;
            const uint32_t hi = i & 1 ? v[i >> 1].w : v[i >> 1].y;
            if constexpr (DTYPE == HS_DTYPE_BF16) {
                x[0] = __uint_as_float(lo << 16);
                x[1] = __uint_as_float(lo & 0xffff0000u);
                x[2] = __uint_as_float(hi << 16);
                x[3] = __uint_as_float(hi & 0xffff0000u);
            } else {
                const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&lo));
                const float2 q = __half22float2(*reinterpret_cast<const __half2*>(&hi));
                x[0] = p.x;
                x[1] = p.y;
                x[2] = q.x;
                x[3] = q.y;
            }
        }
    }

    // Largest finite magnitude.
    __device__ __forceinline__ float magnitude() const {
        float a = 0.f;
        if constexpr (DTYPE == HS_DTYPE_FP32) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float x[4];
                get(i, x);
#pragma unroll
                for (int j = 0; j < 4; ++j) a = fmaxf(a, finite_magnitude(x[j]));
            }
        } else {
            using Pair = std::conditional_t<DTYPE == HS_DTYPE_BF16, __nv_bfloat162, __half2>;
            const uint32_t inf = DTYPE == HS_DTYPE_BF16 ? 0x7f807f80u : 0x7c007c00u;
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    // an infinity or a NaN is not below infinity, and becomes 0
                    uint32_t u = w[j] & 0x7fff7fffu;
                    u &= __hlt2_mask(*reinterpret_cast<const Pair*>(&u),
                                     *reinterpret_cast<const Pair*>(&inf));
                    const Pair p = __hmax2(*reinterpret_cast<const Pair*>(&m),
                                           *reinterpret_cast<const Pair*>(&u));
                    m = *reinterpret_cast<const uint32_t*>(&p);
                }
            }
            const Pair p = *reinterpret_cast<const Pair*>(&m);
            a = fmaxf(__low2float(p), __high2float(p));
        }
        return a;
    }

    template <int CODE>
    __device__ __forceinline__ uint4 encode(float r) const {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float x[4];
            get(i, x);
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = __fmul_rn(x[j], r);
            w[i] = encode4<CODE>(x);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// Two floats in a register pair.
__device__ __forceinline__ uint64_t pair(uint32_t lo, uint32_t hi) {
    uint64_t x;
    asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "r"(lo), "r"(hi));
    return x;
}
__device__ __forceinline__ uint64_t add_pair(uint64_t a, uint64_t b) {
    asm("add.rn.f32x2 %0, %0, %1;" : "+l"(a) : "l"(b));
    return a;
}
__device__ __forceinline__ uint64_t mul_pair(uint64_t a, uint64_t b) {
    asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(a) : "l"(b));
    return a;
}

// 16 codes under one scale, as values under another (r = 1 / the new scale).  INSIDE: the new
// scale covers the values.
template <int CODE, bool INSIDE>
__device__ __forceinline__ uint4 recode(const uint4& c, float scale, float r) {
    const uint32_t in[4] = {c.x, c.y, c.z, c.w};
    uint32_t w[4];
    if constexpr (CODE == HS_KV_E4M3) {
        // Powers of two, as the scales written here are: the two factors are one, and exact in
        // f16 too down to 2^-14 (below it, subnormal codes would lose bits before rounding).
        const float ratio = scale * r;
        const bool power = ((__float_as_uint(scale) | __float_as_uint(r)) & 0x7fffffu) == 0;
        if (power && ratio == 1.f) return c;
        if (power && ratio >= 6.103515625e-05f && ratio <= 32768.f) {
            const __half2 f = __float2half2_rn(ratio);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                __half2 lo, hi;
                decode_halves(in[i], lo, hi);
                lo = __hmul2(lo, f);
                hi = __hmul2(hi, f);
                asm("{\n .reg .b16 a, b;\n cvt.rn.satfinite.e4m3x2.f16x2 a, %1;\n"
                    " cvt.rn.satfinite.e4m3x2.f16x2 b, %2;\n mov.b32 %0, {a, b};\n}"
                    : "=r"(w[i])
                    : "r"(*reinterpret_cast<uint32_t*>(&lo)),
                      "r"(*reinterpret_cast<uint32_t*>(&hi)));
            }
            return make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
    if constexpr (CODE == HS_KV_INT8 && INSIDE) {
        // decode4 and encode4 on pairs, two operations an instruction (64 x 2048 tokens of 8 heads of
        // 128 compacted in 109 us; 119 one by one)
        const uint64_t s2 = pair(__float_as_uint(scale), __float_as_uint(scale));
        const uint64_t r2 = pair(__float_as_uint(r), __float_as_uint(r));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t u = in[i] ^ 0x80808080u;
            uint64_t x[2] = {pair(__byte_perm(u, 0x4b000000u, 0x7540),
                                  __byte_perm(u, 0x4b000000u, 0x7541)),
                             pair(__byte_perm(u, 0x4b000000u, 0x7542),
                                  __byte_perm(u, 0x4b000000u, 0x7543))};
            uint32_t y[4];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                x[j] = add_pair(x[j], pair(0xcb000080u, 0xcb000080u));  // -(2^23 + 128)
                x[j] = mul_pair(mul_pair(x[j], s2), r2);
                asm("mov.b64 {%0, %1}, %2;" : "=r"(y[2 * j]), "=r"(y[2 * j + 1]) : "l"(x[j]));
            }
            // One by one: as a pair, the addition is fused with the product before it.
#pragma unroll
            for (int j = 0; j < 4; ++j)
                y[j] = __float_as_uint(__fadd_rn(__uint_as_float(y[j]), 12582912.f));
            w[i] = __byte_perm(__byte_perm(y[0], y[1], 0x0040), __byte_perm(y[2], y[3], 0x0040),
                               0x5410);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float x[4];
            decode4<CODE>(in[i], x);
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = __fmul_rn(__fmul_rn(x[j], scale), r);
            w[i] = encode4<CODE, INSIDE>(x);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Largest magnitude of 16 codes under a scale.  Rounding is monotonic, so it is the product of
// the scale and the largest code; a NaN code does not count.  int8 codes are compared as pairs of 16-bit
// integers, each with a code in its high byte and whatever lies beside it in its low one (64 x 2048
// tokens of 8 heads of 128 compacted in 119 us; 127 with the codes as floats, which e4m3 is
// better off with: 97 us against 101).
template <int CODE>
__device__ __forceinline__ float magnitude(const uint4& c, float scale) {
    const uint32_t in[4] = {c.x, c.y, c.z, c.w};
    float a;
    if constexpr (CODE == HS_KV_E4M3) {
        __half2 m = __half2half2(__ushort_as_half(0));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            __half2 lo, hi;
            decode_halves(in[i], lo, hi);
            m = __hmax2(m, __hmax2(__habs2(lo), __habs2(hi)));
        }
        a = fmaxf(__low2float(m), __high2float(m));
    } else {
        uint32_t most = 0, least = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            most = __vimax3_s16x2(most, in[i], in[i] << 8);
            least = __vimin3_s16x2(least, in[i], in[i] << 8);
        }
        const int hi = max((int)most >> 24, (int)(most << 16) >> 24);
        const int lo = min((int)least >> 24, (int)(least << 16) >> 24);
        a = (float)max(hi, -lo);
    }
    return finite_magnitude(__fmul_rn(a, scale));
}

// Stores 16 bytes of row (q, t) at byte `off`: into the store, and with CACHE
// into the token's extra-page row (n: the request's length after the call)
// and its hot row as well.
template <bool CACHE>
__device__ __forceinline__ void store_row(const QuantizeArgs& a, int q, int t, int n, int off,
                                          const uint4& x) {
    const int W = a.f.item_size_bytes;
    st_v4(a.rows + ((long long)q * a.L + t) * W + off, x);
    if constexpr (CACHE) {
        const Dims& d = a.d;
        if (d.E > 0 && t >= (n - 1) / d.E * d.E)
            st_v4(a.lv.device_kv +
                      ((long long)d.R * (d.H + d.C) + (long long)q * d.E + t % d.E) * W + off,
                  x);
        const int slot = resident_slot(d, a.lv, q, t, a.status);
        if (slot >= 0) {
            const long long base = (long long)q * (d.H + d.C);
            st_v4(a.lv.device_kv + (base + a.lv.phys[base + slot]) * W + off, x);
        }
    }
}

// With CACHE the copies' addresses take registers that a second CTA an SM would need.
template <int CODE, int DTYPE, bool CACHE>
__global__ void __launch_bounds__(kQuantizeThreads, CACHE ? 1 : 2) quantize_kernel(const QuantizeArgs a) {
    __shared__ float s_tmp[32];
    const int heads = a.f.num_kv_heads, D = a.f.head_dim, T = a.f.block_tokens;
    // CTAs of one block of tokens are neighbours: together they read whole rows
    const int ch = blockIdx.x % (2 * heads);
    const int win = blockIdx.x / (2 * heads) % a.windows;
    const int b = blockIdx.x / (2 * heads) / a.windows;
    wait_for_previous();
    const int q = ld(a.req + b), start = ld(a.start + b), count = ld(a.count + b);
    if (q < 0 || q >= a.R || start < 0 || count < 0 || count > a.max_count ||
        start > a.L - count) {
        if constexpr (CACHE)
            if (threadIdx.x == 0) atomicOr(a.status, HS_STATUS_BAD_APPEND);
        return;
    }
    const int blk = start / T + win;
    const long long first = (long long)blk * T;
    if (first >= start + count || count == 0) return;
    const int end = start + count;
    const int lo = first > start ? (int)first : start;
    const int hi = first + T < end ? (int)first + T : end;
    const int parts = D >> 4;
    const int part = threadIdx.x % parts, j0 = threadIdx.x / parts, step = blockDim.x / parts;
    const int tokens = j0 < step ? hi - lo : 0;  // a part of a warp may be left over
    const int c = ch >= heads, h = c ? ch - heads : ch;
    const void* base = c ? a.in.v_dev : a.in.k_dev;
    const int64_t* stride = c ? a.in.v_stride : a.in.k_stride;
    const long long at0 =
        b * stride[0] + (lo - start) * stride[1] + h * stride[2] + part * 16;

    float* scale_at = a.scales + (((long long)q * a.NB + blk) * 2 + c) * heads + h;
    const bool begun = first < lo;  // the block has tokens from before this call
    const float was = begun ? *scale_at : 0.f;
    constexpr int HELD = DTYPE == HS_DTYPE_FP32 ? kHeld / 2 : kHeld;  // the same registers
    Raw<DTYPE> held[HELD];
    float peak = 0.f;
#pragma unroll
    for (int i = 0; i < HELD; ++i) {
        const int j = j0 + i * step;
        if (j < tokens) held[i].load(base, at0 + j * stride[1], a.vec_in);
    }
#pragma unroll
    for (int i = 0; i < HELD; ++i)
        if (j0 + i * step < tokens) peak = fmaxf(peak, held[i].magnitude());
    for (int j = j0 + HELD * step; j < tokens; j += step) {
        Raw<DTYPE> x;
        x.load(base, at0 + j * stride[1], a.vec_in);
        peak = fmaxf(peak, x.magnitude());
    }
    const float now = fmaxf(was, scale_of<CODE>(block_max(peak, s_tmp)));
    const float r = reciprocal_or_zero(now);
    if (threadIdx.x == 0) *scale_at = now;
    const int off = c * heads * D + h * D + part * 16;
#pragma unroll
    for (int i = 0; i < HELD; ++i) {
        const int j = j0 + i * step;
        if (j < tokens)
            store_row<CACHE>(a, q, lo + j, end, off, held[i].template encode<CODE>(r));
    }
    for (int j = j0 + HELD * step; j < tokens; j += step) {
        Raw<DTYPE> x;
        x.load(base, at0 + j * stride[1], a.vec_in);
        store_row<CACHE>(a, q, lo + j, end, off, x.template encode<CODE>(r));
    }
    if (!begun || !(now > was)) return;
    // The scale grew: the block's older codes are rounded again under it.
    const int old_tokens = j0 < step ? (int)(lo - first) : 0;
    for (int j = j0; j < old_tokens; j += step) {
        const int t = (int)first + j;
        const uint4 x = *reinterpret_cast<const uint4*>(
            a.rows + ((long long)q * a.L + t) * a.f.item_size_bytes + off);
        store_row<CACHE>(a, q, t, end, off, recode<CODE, false>(x, was, r));
    }
}

template <int CODE>
__global__ void __launch_bounds__(kCompactThreads, 2) compact_kernel(const CompactArgs a) {
    __shared__ float s_tmp[32];
    const int heads = a.f.num_kv_heads, D = a.f.head_dim, T = a.f.block_tokens;
    const int W = a.f.item_size_bytes;
    const int ch = blockIdx.x % (2 * heads);
    const int win = blockIdx.x / (2 * heads) % a.windows;
    const int b = blockIdx.x / (2 * heads) / a.windows;
    wait_for_previous();
    const int sq = ld(a.src_req + b), dq = ld(a.dst_req + b);
    int kept = ld(a.kept + b);
    if (sq < 0 || sq >= a.src_R || dq < 0 || dq >= a.dst_R) return;
    kept = min(kept, min(a.budget, a.dst_L));
    const int first = win * T;
    int tokens = min(T, kept - first);
    if (tokens <= 0) return;
    const int parts = D >> 4;
    const int part = threadIdx.x % parts, j0 = threadIdx.x / parts, step = blockDim.x / parts;
    if (j0 >= step) tokens = 0;  // a part of a warp may be left over
    const int off = ch * D + part * 16;
    const uint8_t* src = a.src + (long long)sq * a.src_L * W + off;
    uint8_t* dst = a.dst + ((long long)dq * a.dst_L + first) * W + off;
    const int32_t* keep = a.keep + (long long)b * a.budget + first;
    const float* scales = a.src_scales + (long long)sq * a.src_NB * 2 * heads + ch;

    uint4 held[kHeld];
    float scale[kHeld];
    float peak = 0.f;
    auto load = [&](int t, uint4& x, float& s) {
        x = make_uint4(0, 0, 0, 0);
        s = 0.f;
        if (t >= 0 && t < a.src_L) {
            x = ld_once_v4(src + (long long)t * W);
            s = ld(scales + (long long)a.block.of(t) * (2 * heads));
        }
    };
    int t[kHeld];
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
        const int j = j0 + i * step;
        t[i] = j < tokens ? ld(keep + j) : -1;
    }
#pragma unroll
    for (int i = 0; i < kHeld; ++i) load(t[i], held[i], scale[i]);
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
        peak = fmaxf(peak, magnitude<CODE>(held[i], scale[i]));
        // the codes are decoded anew below: kept, the values would take four times the registers
        asm volatile("" : "+r"(held[i].x), "+r"(held[i].y), "+r"(held[i].z), "+r"(held[i].w));
    }
    for (int j = j0 + kHeld * step; j < tokens; j += step) {
        uint4 x;
        float s;
        load(ld(keep + j), x, s);
        peak = fmaxf(peak, magnitude<CODE>(x, s));
    }
    const float now = scale_of<CODE>(block_max(peak, s_tmp));
    const float r = reciprocal_or_zero(now);
    if (threadIdx.x == 0)
        a.dst_scales[((long long)dq * a.dst_NB + win) * 2 * heads + ch] = now;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
        const int j = j0 + i * step;
        if (j < tokens)
            st_v4(dst + (long long)j * W, recode<CODE, true>(held[i], scale[i], r));
    }
    for (int j = j0 + kHeld * step; j < tokens; j += step) {
        uint4 x;
        float s;
        load(ld(keep + j), x, s);
        st_v4(dst + (long long)j * W, recode<CODE, true>(x, s, r));
    }
}

template <int CODE, bool CACHE>
cudaError_t quantize_dtype(const QuantizeArgs& a, int grid, int threads, cudaStream_t s) {
    if (a.in.dtype == HS_DTYPE_BF16)
        return launch_chained(quantize_kernel<CODE, HS_DTYPE_BF16, CACHE>, grid, threads, 0, 0, s, a);
    if (a.in.dtype == HS_DTYPE_FP16)
        return launch_chained(quantize_kernel<CODE, HS_DTYPE_FP16, CACHE>, grid, threads, 0, 0, s, a);
    return launch_chained(quantize_kernel<CODE, HS_DTYPE_FP32, CACHE>, grid, threads, 0, 0, s, a);
}

bool grid_of(long long ctas, int* grid) {
    if (ctas > 0x7fffffffLL) return false;
    *grid = (int)ctas;
    return true;
}

}  // namespace

cudaError_t launch_quantize(QuantizeArgs a, bool cache, cudaStream_t s) {
    const int T = a.f.block_tokens;
    a.windows = (int)(((long long)a.max_count + T - 2) / T + 1);
    const int esz = a.in.dtype == HS_DTYPE_FP32 ? 4 : 2;
    bool vec = ((uintptr_t)a.in.k_dev | (uintptr_t)a.in.v_dev) % 16 == 0;
    for (int i = 0; i < 3; ++i)
        vec = vec && (a.in.k_stride[i] * esz) % 16 == 0 && (a.in.v_stride[i] * esz) % 16 == 0;
    a.vec_in = vec;
    int grid;
    if (!grid_of((long long)a.batch * a.windows * 2 * a.f.num_kv_heads, &grid))
        return cudaErrorInvalidConfiguration;
    const int parts = a.f.head_dim / 16;
    const int threads = group_threads(a.max_count < T ? a.max_count : T, parts,
                                      a.in.dtype == HS_DTYPE_FP32 ? kHeld / 2 : kHeld,
                                      kQuantizeThreads);
    if (a.f.code == HS_KV_E4M3)
        return cache ? quantize_dtype<HS_KV_E4M3, true>(a, grid, threads, s)
                     : quantize_dtype<HS_KV_E4M3, false>(a, grid, threads, s);
    return cache ? quantize_dtype<HS_KV_INT8, true>(a, grid, threads, s)
                 : quantize_dtype<HS_KV_INT8, false>(a, grid, threads, s);
}

cudaError_t launch_compact(CompactArgs a, cudaStream_t s) {
    const int T = a.f.block_tokens;
    const int most = a.budget < a.dst_L ? a.budget : a.dst_L;
    a.windows = (most + T - 1) / T;
    int grid;
    if (!grid_of((long long)a.batch * a.windows * 2 * a.f.num_kv_heads, &grid))
        return cudaErrorInvalidConfiguration;
    a.block = Divisor::by(T);
    const int parts = a.f.head_dim / 16;
    const int threads = group_threads(most < T ? most : T, parts, kHeld, kCompactThreads);
    return launch_chained(
        a.f.code == HS_KV_E4M3 ? compact_kernel<HS_KV_E4M3> : compact_kernel<HS_KV_INT8>, grid,
        threads, 0, 0, s, a);
}

}  // namespace hs
