// RMS norm of every query and key head and the position rotation, in one pass
// (sm_103a).
//
// D / 16 lanes hold a head, 16 elements each: two pieces of 8 that lie rot / 2
// apart, so that a lane holds both elements of its pairs whichever way they are
// paired.  The sum of squares goes over the lanes by shuffles; nothing is read twice.
//
// Angles: position * frequency would lose what matters in 32 bits (at position 131072 an angle
// is off by 2^-8) and take sines of large numbers.  The frequency comes as a part of a turn in
// 64-bit fixed point, the product is taken modulo 2^64, that is modulo whole turns, and
// is off by |position| * 2^-65 turns.  What is left of an eighth of a turn goes through sincospif, the
// quadrant is put back by exchange and sign.  A CTA
// computes the cosines and sines of its tile of tokens once for all their heads.
//
// What bounds it: 2 * size bytes an element, for about 10 operations: memory.  32768 tokens of 40 heads
// of 128 bf16 elements take 117 us, 5.7 TB/s read and written; with one head at a time and its addresses
// computed anew for each they took 199 us (438 instructions for 16 elements of a lane, 300 now: the
// rest of the time is still half of what the schedulers can issue).
#include "hs_step.cuh"

namespace hs {
namespace {

constexpr int kThreads = 256;
constexpr int kTile = 24;  // tokens of a CTA, at most
// CTAs of an SM, by registers: of 32-bit elements twice as many are under way in each.
constexpr int ctas_per_sm(size_t element) { return element == 4 ? 2 : 3; }

struct RopeArgs {
    const void* in[2];  // queries, keys
    void* out[2];
    int64_t in_stride[2][3], out_stride[2][3];
    const float* weight[2];
    float eps;
    int32_t rot, adjacent, axes, M, Hq, heads;  // heads: of queries and keys
    long long tokens;  // batch * M
    int32_t tile, run;  // tokens of a CTA, and of a lane group at a time
    Divisor by_heads;
    const int32_t* pos;
    const int64_t* turns;
    const int32_t* axis;
    const int32_t* count;
    int32_t vec_in, vec_out;
};

// Eight consecutive elements as they lie in memory.
template <typename T>
struct Raw {
    uint4 v[sizeof(T) / 2];
};

template <typename T>
__device__ __forceinline__ void load8(Raw<T>& x, const T* p, bool vec) {
    constexpr int kEach = 16 / sizeof(T);
    if (vec) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) x.v[i] = ld_once_v4(p + i * kEach);
    } else {
        alignas(16) T y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = ld(p + i);
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) x.v[i] = reinterpret_cast<const uint4*>(y)[i];
    }
}

template <typename T>
__device__ __forceinline__ void decode8(float (&x)[8], const Raw<T>& raw) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            x[4 * i] = __uint_as_float(raw.v[i].x), x[4 * i + 1] = __uint_as_float(raw.v[i].y);
            x[4 * i + 2] = __uint_as_float(raw.v[i].z), x[4 * i + 3] = __uint_as_float(raw.v[i].w);
        }
    } else {
        const uint32_t w[4] = {raw.v[0].x, raw.v[0].y, raw.v[0].z, raw.v[0].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (__is_same(T, __half)) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
                x[2 * i] = f.x, x[2 * i + 1] = f.y;
            } else {
                x[2 * i] = __uint_as_float(w[i] << 16);
                x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        }
    }
}

template <typename T>
__device__ __forceinline__ T from_float(float x);
template <>
__device__ __forceinline__ float from_float<float>(float x) { return x; }
template <>
__device__ __forceinline__ __half from_float<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float x) {
    return __float2bfloat16_rn(x);
}

template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&x)[8], bool vec) {
    if (vec) {
        alignas(16) T y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = from_float<T>(x[i]);
        const uint4* v = reinterpret_cast<const uint4*>(y);
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) st_v4(p + i * (16 / sizeof(T)), v[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = from_float<T>(x[i]);
    }
}

// (cos, sin) of the angle of a position, whose frequency is `turn` * 2^-64 turns.
__device__ __forceinline__ float2 rotation(int32_t pos, int64_t turn) {
    const uint64_t phase = (uint64_t)(int64_t)pos * (uint64_t)turn + 0x80000000ull;
    const uint32_t t = (uint32_t)(phase >> 32);
    const uint32_t quadrant = (t + 0x20000000u) >> 30;
    const int32_t rest = (int32_t)(t - (quadrant << 30));  // within an eighth of a turn
    float s, c;
    sincospif((float)rest * 0x1p-31f, &s, &c);
    if (quadrant & 1) {
        const float x = c;
        c = -s;
        s = x;
    }
    return quadrant & 2 ? make_float2(-c, -s) : make_float2(c, s);
}

__device__ __forceinline__ void turn(float& y0, float& y1, float c, float s) {
    const float z = y0;
    y0 = z * c - y1 * s;
    y1 = z * s + y1 * c;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(sizeof(T))) norm_rope_kernel(const RopeArgs a) {
    constexpr int kUsed = D / 16;                                        // lanes of a head
    constexpr int kLanes = kUsed <= 2 ? 2 : kUsed <= 4 ? 4 : kUsed <= 8 ? 8 : 16;  // padded
    constexpr int kGroups = kThreads / kLanes;
    // Cosines and sines, [token][4][rot / 16 lanes][2]: the 8 pairs of a lane two at a time, so that
    // lanes side by side read side by side.
    extern __shared__ __align__(16) float2 s_turn[];
    __shared__ __align__(16) float s_weight[2 * D];  // [queries, keys][4][lanes][4] likewise
    const int tid = threadIdx.x, lane = tid % kLanes, group = tid / kLanes;
    const int tiles = (a.M + a.tile - 1) / a.tile, b = blockIdx.x / tiles;
    const int m0 = (blockIdx.x - b * tiles) * a.tile;
    const int half = a.rot / 2, pairs = a.rot / 16;
    // This lane's pieces of 8 elements: a pair of them that turns together, or two that do not turn.
    const bool turns = lane < pairs, used = lane < kUsed;
    const int p0 = 8 * (turns ? lane : 2 * lane), p1 = turns ? half : 8;
    wait_for_previous();
    const int tokens = min(a.tile, (a.count ? min(a.M, ld(a.count + b)) : a.M) - m0);
    if (tokens <= 0) return;
    // Heads are taken in runs of the same head of consecutive tokens, run after run of all heads.
    const int units = (tokens + a.run - 1) / a.run * a.heads;
    struct Cursor {
        int unit, token, left;  // the token's number in the tile, tokens left of the run
    };
    const auto head_of = [&](Cursor& c) {  // starts a run
        const int unit = min(c.unit, units - 1), sub = a.by_heads.of(unit);
        c.token = sub * a.run;
        c.left = a.run;
        return unit - sub * a.heads;
    };
    Cursor in = {group, 0, 0}, out = in;
    const T* from = nullptr;
    T* to = nullptr;
    long long from_step = 0, to_step = 0;
    const float* weight = s_weight;
    bool norm = false;
    const auto enter_in = [&] {
        const int head = head_of(in), w = head >= a.Hq, h = head - (w ? a.Hq : 0);
        from = static_cast<const T*>(a.in[w]) + b * a.in_stride[w][0] +
               (m0 + in.token) * a.in_stride[w][1] + h * a.in_stride[w][2] + p0;
        from_step = a.in_stride[w][1];
    };
    const auto enter_out = [&] {
        const int head = head_of(out), w = head >= a.Hq, h = head - (w ? a.Hq : 0);
        to = static_cast<T*>(a.out[w]) + b * a.out_stride[w][0] +
             (m0 + out.token) * a.out_stride[w][1] + h * a.out_stride[w][2] + p0;
        to_step = a.out_stride[w][1];
        norm = a.weight[w];
        weight = s_weight + w * D;
    };
    struct Item {
        Raw<T> x[2];
    };
    const auto fetch = [&](Item& it) {
        if (in.left == 0) enter_in();
        if (used && in.unit < units && in.token < tokens) {
            load8(it.x[0], from, a.vec_in);
            load8(it.x[1], from + p1, a.vec_in);
        }
        from += from_step;
        ++in.token;
        if (--in.left == 0) in.unit += kGroups;
    };
    const auto step = [&](Item& it) {
        if (out.left == 0) enter_out();
        const bool live = used && out.unit < units && out.token < tokens;
        float x[2][8];
#pragma unroll
        for (int c = 0; c < 2; ++c) decode8<T>(x[c], it.x[c]);
        fetch(it);
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) sum += x[0][k] * x[0][k] + x[1][k] * x[1][k];
        if (!live) sum = 0.f;
#pragma unroll
        for (int o = 1; o < kLanes; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (live) {
            if (norm) {
                const float r = rsqrtf(sum * (1.f / D) + a.eps);
                const float4* wt = reinterpret_cast<const float4*>(weight) + lane;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float4 v = wt[k * kUsed];
                    float* y = x[k / 2] + k % 2 * 4;
                    y[0] *= r * v.x, y[1] *= r * v.y, y[2] *= r * v.z, y[3] *= r * v.w;
                }
            }
            if (turns) {
                const float4* cs = reinterpret_cast<const float4*>(s_turn + out.token * half) + lane;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float4 t = cs[k * pairs];
                    if (a.adjacent) {
                        turn(x[k / 2][4 * (k % 2)], x[k / 2][4 * (k % 2) + 1], t.x, t.y);
                        turn(x[k / 2][4 * (k % 2) + 2], x[k / 2][4 * (k % 2) + 3], t.z, t.w);
                    } else {
                        turn(x[0][2 * k], x[1][2 * k], t.x, t.y);
                        turn(x[0][2 * k + 1], x[1][2 * k + 1], t.z, t.w);
                    }
                }
            }
            store8(to, x[0], a.vec_out);
            store8(to + p1, x[1], a.vec_out);
        }
        to += to_step;
        ++out.token;
        if (--out.left == 0) out.unit += kGroups;
    };
    // Two heads are under way ahead of the one that is worked on, the first ones while the angles are.
    Item even, odd;
    fetch(even);
    fetch(odd);
    for (int i = tid; i < 2 * D; i += kThreads) {
        const int w = i / D, d = i - w * D, l = d / 4 % kUsed, k = d / 4 / kUsed;
        // number 4 k + d % 4 of lane l
        const int at = (l < pairs ? 8 * l + k / 2 * half : 16 * l + k / 2 * 8) + k % 2 * 4 + d % 4;
        if (a.weight[w]) s_weight[i] = ld(a.weight[w] + at);
    }
    for (int i = tid; i < tokens * half; i += kThreads) {
        const int t = i / half, j = i - t * half;
        int x = a.axis ? ld(a.axis + j) : 0;
        x = min(max(x, 0), a.axes - 1);
        // pair j is number u of lane l
        const int quarter = j / 4, l = a.adjacent ? quarter % pairs : j / 8;
        const int u = a.adjacent ? quarter / pairs * 4 + j % 4 : j % 8;
        s_turn[t * half + (u / 2 * pairs + l) * 2 + u % 2] =
            rotation(ld(a.pos + x * a.tokens + (long long)b * a.M + m0 + t), ld(a.turns + j));
    }
    __syncthreads();
    release_next();
    const int steps = (units + kGroups - 1) / kGroups * a.run;  // the same for all lanes
    for (int i = 0; i < steps; i += 2) {
        step(even);
        if (i + 1 < steps) step(odd);
    }
}

template <typename T, int D>
cudaError_t run(RopeArgs a, cudaStream_t s) {
    constexpr int kUsed = D / 16;
    constexpr int kLanes = kUsed <= 2 ? 2 : kUsed <= 4 ? 4 : kUsed <= 8 ? 8 : 16;
    constexpr int kGroups = kThreads / kLanes;
    // A CTA takes all heads of a tile of tokens: no angle is computed twice.  Tiles are as large as fills
    // the SMs once, or, up to kTile tokens, a whole number of times.  A run computes its addresses
    // once and steps through memory; four rounds of runs spread the heads over the lane groups evenly
    // enough.
    const int half = a.rot / 2;
    const long long held = 152 * ctas_per_sm(sizeof(T));
    const long long waves = (a.tokens + held * kTile - 1) / (held * kTile);
    a.tile = (int)((a.tokens + held * waves - 1) / (held * waves));
    if (a.tile > a.M) a.tile = a.M;
    const int tiles = (a.M + a.tile - 1) / a.tile;
    a.tile = (a.M + tiles - 1) / tiles;
    int runs = (4 * kGroups + a.heads - 1) / a.heads;
    if (runs > a.tile) runs = a.tile;
    a.run = (a.tile + runs - 1) / runs;
    const size_t smem = (size_t)a.tile * half * sizeof(float2);
    const int grid = (int)(a.tokens / a.M * tiles);
    return launch_chained(norm_rope_kernel<T, D>, grid, kThreads, smem, 0, s, a);
}

template <typename T>
cudaError_t run_dim(const RopeArgs& a, int D, cudaStream_t s) {
    switch (D) {
        case 32: return run<T, 32>(a, s);
        case 64: return run<T, 64>(a, s);
        case 96: return run<T, 96>(a, s);
        case 128: return run<T, 128>(a, s);
        case 192: return run<T, 192>(a, s);
        case 256: return run<T, 256>(a, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace

cudaError_t launch_norm_rope(const hs_norm_rope_args& x, cudaStream_t s) {
    RopeArgs a = {};
    const int esz = x.dtype == HS_DTYPE_FP32 ? 4 : 2;
    const void* in[2] = {x.q_dev, x.k_dev};
    void* out[2] = {x.q_out_dev, x.k_out_dev};
    const float* weight[2] = {x.q_weight_dev, x.k_weight_dev};
    const int64_t* strides[4] = {x.q_stride, x.k_stride, x.q_out_stride, x.k_out_stride};
    a.vec_in = a.vec_out = 1;
    for (int w = 0; w < 2; ++w) {
        a.in[w] = in[w];
        a.out[w] = out[w];
        a.weight[w] = weight[w];
        a.vec_in &= (uintptr_t)in[w] % 16 == 0;
        a.vec_out &= (uintptr_t)out[w] % 16 == 0;
        if (!(w ? x.num_kv_heads : x.num_heads)) continue;
        for (int i = 0; i < 3; ++i) {
            a.in_stride[w][i] = strides[w][i];
            a.out_stride[w][i] = strides[2 + w][i];
            a.vec_in &= strides[w][i] * esz % 16 == 0;
            a.vec_out &= strides[2 + w][i] * esz % 16 == 0;
        }
    }
    a.eps = x.eps;
    a.rot = x.rot_dim;
    a.adjacent = x.adjacent;
    a.axes = x.num_axes;
    a.M = x.tokens;
    a.Hq = x.num_heads;
    a.heads = x.num_heads + x.num_kv_heads;
    a.tokens = (long long)x.batch * x.tokens;
    a.by_heads = Divisor::by(a.heads);
    a.pos = x.pos_dev;
    a.turns = x.turns_dev;
    a.axis = x.axis_dev;
    a.count = x.count_dev;
    if (x.dtype == HS_DTYPE_BF16) return run_dim<__nv_bfloat16>(a, x.head_dim, s);
    if (x.dtype == HS_DTYPE_FP16) return run_dim<__half>(a, x.head_dim, s);
    return run_dim<float>(a, x.head_dim, s);
}

}  // namespace hs
