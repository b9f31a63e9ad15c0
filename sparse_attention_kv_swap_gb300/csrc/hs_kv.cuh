// Shared by the calls that give the KV rows a content (8-bit keys and values
// with a scale for each block of tokens and head): codes, scales and the
// launchers.  The row and scale layouts are in include/hisparse_swap.h.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "hs_internal.cuh"

namespace hs {

// Launchers (each returns the launch's error code).
struct QuantizeArgs {
    hs_kv_format f;
    hs_kv_input in;
    const int32_t* req;
    const int32_t* start;
    const int32_t* count;
    int32_t batch, max_count;
    uint8_t* rows;  // [R][L][W] the store, or the device mapping of the host pool
    float* scales;  // [R][NB][2][Hkv]
    int32_t R, L, NB;
    int32_t windows;  // blocks of T tokens that max_count tokens can touch
    int32_t vec_in;   // 1: 16-byte loads of the input are aligned
    // hs_append_kv: the other copies of a row, and where to report bad entries
    Dims d;
    LayerView lv;
    uint32_t* status;
};
cudaError_t launch_quantize(QuantizeArgs a, bool cache, cudaStream_t s);

// Division of 0 <= t < 2^31 by a constant d: with 2^l >= d > 2^(l-1), m = ceil(2^(31 + l) / d) is
// below 2^32 and m / 2^(31 + l) above 1 / d by less than 2^-(31 + l).  So the product is above t / d by less
// than 2^-l <= 1 / d, too little to reach the next integer.
struct Divisor {
    uint32_t m;
    int32_t shift;
    static Divisor by(int32_t d) {
        int l = 0;
        while ((1ll << l) < d) ++l;
        Divisor x;
        x.m = (uint32_t)(((1ull << (31 + l)) + (uint32_t)d - 1) / (uint32_t)d);
        x.shift = 31 + l;
        return x;
    }
#ifdef __CUDACC__
    __device__ __forceinline__ int32_t of(int32_t t) const {
        return (int32_t)(((uint64_t)(uint32_t)t * m) >> shift);
    }
#endif
};

struct CompactArgs {
    hs_kv_format f;
    const uint8_t* src;
    const float* src_scales;
    const int32_t* src_req;
    const int32_t* keep;
    const int32_t* kept;
    uint8_t* dst;
    float* dst_scales;
    const int32_t* dst_req;
    int32_t batch, budget;
    int32_t src_R, src_L, src_NB, dst_R, dst_L, dst_NB;
    int32_t windows;
    Divisor block;  // by block_tokens
};
cudaError_t launch_compact(CompactArgs a, cudaStream_t s);

cudaError_t launch_accumulate(const float* weights, const int32_t* topk, const int32_t* req,
                              const int32_t* counts, int32_t B, int32_t S, int32_t K, float* acc,
                              int32_t R, int32_t L, bool after_attend, cudaStream_t s);
cudaError_t launch_evict(const float* acc, const int32_t* req, const int32_t* seq_lens, int32_t B,
                         int32_t recent, int32_t budget, int32_t R, int32_t L, int32_t* keep,
                         int32_t* kept, float* kept_acc, cudaStream_t s);

size_t attend_workspace(const hs_kv_format& f, const hs_attend_args& a);
cudaError_t launch_attend(const hs_kv_format& f, const hs_attend_args& a, cudaStream_t s);

// ---- device helpers ---------------------------------------------------------
#ifdef __CUDACC__

// The kernels of these calls run one after the other on a stream, some for a few microseconds:
// each may be launched while the one before it still runs (launch_chained) and waits for its
// end, memory included, before it touches memory that the one before or any earlier one writes
// (wait_for_previous).  The next launch is let go at the end of this kernel, or where all its CTAs
// have come to release_next: there the next one's CTAs may take the place that is left.
__device__ __forceinline__ void wait_for_previous() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void release_next() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Reads of what an earlier kernel may have written: ordinary loads, because those of read-only data
// may be moved ahead of the wait and keep what the kernel before has left in an SM's L1.
template <typename T>
__device__ __forceinline__ T ld(const T* p) {
    return *p;
}
__device__ __forceinline__ uint4 ld_once_v4(const void* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

template <typename... P, typename... A>
cudaError_t launch_chained(void (*kernel)(P...), int grid, int block, size_t smem, int cluster,
                           cudaStream_t s, const A&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 0 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

constexpr float kScaleFloor = 7.888609052210118e-31f;  // 2^-100

// Four codes as two pairs of f16 (e4m3).
__device__ __forceinline__ void decode_halves(uint32_t w, __half2& lo, __half2& hi) {
    uint32_t x, y;
    asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n"
        " cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}"
        : "=r"(x), "=r"(y)
        : "r"(w));
    lo = *reinterpret_cast<__half2*>(&x);
    hi = *reinterpret_cast<__half2*>(&y);
}

// Four codes as 32-bit values.
template <int CODE>
__device__ __forceinline__ void decode4(uint32_t w, float (&x)[4]) {
    if constexpr (CODE == HS_KV_E4M3) {
        __half2 lo, hi;
        decode_halves(w, lo, hi);
        const float2 p = __half22float2(lo), q = __half22float2(hi);
        x[0] = p.x;
        x[1] = p.y;
        x[2] = q.x;
        x[3] = q.y;
    } else {
        // 0x4b000000 | b is the float 2^23 + b of a byte b: with the sign bit flipped, b is the
        // code + 128.
        const uint32_t u = w ^ 0x80808080u;
        x[0] = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7540)) - 8388736.f;
        x[1] = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7541)) - 8388736.f;
        x[2] = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7542)) - 8388736.f;
        x[3] = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7543)) - 8388736.f;
    }
}

// Four codes of y (already divided by the scale): to nearest, ties to even,
// clamped to the largest code.  NaN becomes the e4m3 NaN, or 0 in int8.  With
// INSIDE, every y is known to be finite and to round to a code.
template <int CODE, bool INSIDE = false>
__device__ __forceinline__ uint32_t encode4(const float (&y)[4]) {
    uint32_t w;
    if constexpr (CODE == HS_KV_E4M3) {
        asm("{\n .reg .b16 a, b;\n cvt.rn.satfinite.e4m3x2.f32 a, %2, %1;\n"
            " cvt.rn.satfinite.e4m3x2.f32 b, %4, %3;\n mov.b32 %0, {a, b};\n}"
            : "=r"(w)
            : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]));
    } else {
        // Adding 1.5 * 2^23 leaves the rounded integer in the low bits.
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float x = y[i];
            if (!INSIDE) x = x == x ? fminf(fmaxf(x, -127.f), 127.f) : 0.f;
            u[i] = __float_as_uint(x + 12582912.f);
        }
        w = __byte_perm(__byte_perm(u[0], u[1], 0x0040), __byte_perm(u[2], u[3], 0x0040), 0x5410);
    }
    return w;
}

// Scale of a block whose largest magnitude is a (finite, >= 0).
template <int CODE>
__device__ __forceinline__ float scale_of(float a) {
    if (!(a > 0.f)) return 0.f;
    a = fmaxf(a, kScaleFloor);
    if constexpr (CODE == HS_KV_E4M3) {
        // a = m * 2^e with 1 <= m < 2; 448 = 1.75 * 2^8
        const uint32_t u = __float_as_uint(a);
        int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
        e = e < -100 ? -100 : e;
        return __uint_as_float((uint32_t)(e + 127) << 23);
    } else {
        return __fdiv_rn(a, 127.f);
    }
}

__device__ __forceinline__ float reciprocal_or_zero(float s) {
    return s > 0.f ? __frcp_rn(s) : 0.f;
}

__device__ __forceinline__ float finite_magnitude(float x) {
    const float a = fabsf(x);
    return a <= 3.402823466e38f ? a : 0.f;  // false for NaN too
}

// Largest of a value >= 0 over the block; every thread gets it.  `tmp`: 32 floats.
__device__ __forceinline__ float block_max(float a, float* tmp) {
    // bit patterns of floats >= 0 order like the floats
    const unsigned w = __reduce_max_sync(0xffffffffu, __float_as_uint(a));
    const int nwarps = (blockDim.x + 31) >> 5;
    if (nwarps == 1) return __uint_as_float(w);
    if ((threadIdx.x & 31) == 0) tmp[threadIdx.x >> 5] = __uint_as_float(w);
    __syncthreads();
    const int lane = threadIdx.x & 31;
    return __uint_as_float(
        __reduce_max_sync(0xffffffffu, lane < nwarps ? __float_as_uint(tmp[lane]) : 0u));
}

#endif  // __CUDACC__

}  // namespace hs
