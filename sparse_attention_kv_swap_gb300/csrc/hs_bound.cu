// Least and greatest key of every block of tokens, K/V head and channel (sm_103a).
//
// A CTA takes 256 channels of one block of a request; a lane holds 8 of them, the warps share the
// tokens, and least and greatest are joined in shared memory.  Minima and maxima of 16-bit
// keys are keys: nothing is rounded, so that bounds kept up token by token are those of the whole
// block.  Memory bound for prompts (each key is read once): 4 of 8192 tokens, 8 heads of 128, take
// 14.6 us, 4.7 TB/s; latency for tokens (8.0 us for one of each of 64 requests, through Python).
#include "hs_step.cuh"

namespace hs {
namespace {

constexpr int kWarps = 8;
constexpr int kAhead = 8;  // tokens a lane has under way

struct F16 {
    static constexpr uint32_t kHigh = 0x7c007c00u, kLow = 0xfc00fc00u;  // two infinities
    static __device__ __forceinline__ uint32_t least(uint32_t a, uint32_t b) {
        const __half2 x = __hmin2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
        return *reinterpret_cast<const uint32_t*>(&x);
    }
    static __device__ __forceinline__ uint32_t greatest(uint32_t a, uint32_t b) {
        const __half2 x = __hmax2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
        return *reinterpret_cast<const uint32_t*>(&x);
    }
};
struct B16 {
    static constexpr uint32_t kHigh = 0x7f807f80u, kLow = 0xff80ff80u;
    static __device__ __forceinline__ uint32_t least(uint32_t a, uint32_t b) {
        const __nv_bfloat162 x = __hmin2(*reinterpret_cast<__nv_bfloat162*>(&a),
                                         *reinterpret_cast<__nv_bfloat162*>(&b));
        return *reinterpret_cast<const uint32_t*>(&x);
    }
    static __device__ __forceinline__ uint32_t greatest(uint32_t a, uint32_t b) {
        const __nv_bfloat162 x = __hmax2(*reinterpret_cast<__nv_bfloat162*>(&a),
                                         *reinterpret_cast<__nv_bfloat162*>(&b));
        return *reinterpret_cast<const uint32_t*>(&x);
    }
};

// Eight consecutive 16-bit elements.
__device__ __forceinline__ uint4 load16x8(const uint8_t* p, bool vec) {
    if (vec) return ld_once_v4(p);
    const uint16_t* e = reinterpret_cast<const uint16_t*>(p);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = (uint32_t)ld(e + 2 * i) | (uint32_t)ld(e + 2 * i + 1) << 16;
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void store16x8(uint8_t* p, const uint32_t (&w)[4], bool vec) {
    if (vec) {
        st_v4(p, make_uint4(w[0], w[1], w[2], w[3]));
        return;
    }
    uint16_t* e = reinterpret_cast<uint16_t*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) e[2 * i] = (uint16_t)w[i], e[2 * i + 1] = (uint16_t)(w[i] >> 16);
}

template <typename E>
__device__ __forceinline__ void join(uint32_t (&low)[4], uint32_t (&high)[4], const uint4& a,
                                     const uint4& b) {
    const uint32_t l[4] = {a.x, a.y, a.z, a.w}, h[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        low[i] = E::least(low[i], l[i]);
        high[i] = E::greatest(high[i], h[i]);
    }
}

template <typename E>
__global__ void __launch_bounds__(32 * kWarps) bound_kernel(const BoundArgs a) {
    __shared__ uint4 s_low[kWarps][32], s_high[kWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int slab = blockIdx.x % a.slabs, bw = blockIdx.x / a.slabs;
    const int window = bw % a.windows, b = bw / a.windows;
    const int channel = slab * 256 + lane * 8, h = channel / a.D, d = channel - h * a.D;
    const bool used = channel < a.Hkv * a.D;
    wait_for_previous();
    release_next();
    const int r = ld(a.req + b), start = ld(a.start + b), count = ld(a.count + b);
    if (r < 0 || r >= a.R || start < 0 || count <= 0 || count > a.max_count ||
        start > a.L - count)
        return;
    if (window > (start + count - 1) / a.T - start / a.T) return;
    const int block = start / a.T + window;
    const long long t0 = (long long)block * a.T;
    const int lo = t0 > start ? (int)(t0 - start) : 0;  // the block's first new token
    const int n = (int)min((long long)count, t0 + a.T - start) - lo;
    uint32_t low[4], high[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) low[i] = E::kHigh, high[i] = E::kLow;
    if (used) {
        const uint8_t* p = a.k + 2 * (b * a.stride[0] + lo * a.stride[1] + h * a.stride[2] + d);
        for (int i0 = warp; i0 < n; i0 += kWarps * kAhead) {
            uint4 x[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u)  // past the last one, the first again
                x[u] = load16x8(p + 2 * (i0 + u * kWarps < n ? i0 + u * kWarps : i0) * a.stride[1],
                                a.vec_k);
#pragma unroll
            for (int u = 0; u < kAhead; ++u) join<E>(low, high, x[u], x[u]);
        }
    }
    s_low[warp][lane] = make_uint4(low[0], low[1], low[2], low[3]);
    s_high[warp][lane] = make_uint4(high[0], high[1], high[2], high[3]);
    __syncthreads();
    if (warp > 0 || !used) return;
#pragma unroll
    for (int w = 1; w < kWarps; ++w) join<E>(low, high, s_low[w][lane], s_high[w][lane]);
    uint8_t* to = a.bounds + 2 * ((((long long)r * a.NB + block) * a.Hkv + h) * 2 * a.D + d);
    if (t0 < start)  // begun before: its bounds so far count
        join<E>(low, high, load16x8(to, a.vec_bounds), load16x8(to + 2 * a.D, a.vec_bounds));
    store16x8(to, low, a.vec_bounds);
    store16x8(to + 2 * a.D, high, a.vec_bounds);
}

}  // namespace

cudaError_t launch_bound(BoundArgs a, cudaStream_t s) {
    const int grid = a.batch * a.windows * a.slabs;
    return launch_chained(a.fp16 ? bound_kernel<F16> : bound_kernel<B16>, grid, 32 * kWarps, 0, 0, s,
                          a);
}

}  // namespace hs
