// Attention of decode queries over 8-bit rows at device locations (sm_103a);
// the contract is hs_attend's in include/hisparse_swap.h.
//
// A thread-block cluster of P CTAs serves one query position (b, s); the CTAs
// take its selected rows in turns of 16, for all heads, and drop the masked
// ones.  A warp's task is one K/V head (and up to 16 of the query heads that
// share it) over tiles of 16 tokens:
//   1. scores: S^T[token, head] = K[token, d] Q^T[d, head] with f16
//      m16n8k16 products summed in 32 bits.  A selected row is read by exactly
//      one warp per K/V head, so K goes from global memory straight into the
//      operand registers: lane (g, c) loads 16 bytes out of each 64 of the rows
//      g and g + 8, and because a product may visit d in any order, the four
//      bytes of a word are four d of one step.  Codes are exact in f16;
//      the query is scaled by a power of two per head into f16's range, which
//      keeps bf16's and f16's significands whole.  Scores go to shared memory
//      in 32 bits.
//   2. softmax over the task's own tokens: all scores are known, so there is
//      no running rescale.
//   3. O^T[d, head] = V^T[d, token] P^T[token, head]: lane (g, c) loads its
//      16 bytes out of each 128 of the rows of tokens 4 c .. 4 c + 3, a byte
//      permute pairs neighbouring tokens.  P is exp(s - max) times the token's
//      V scale over the largest V scale of the task, so it lies in [0, 1] and
//      is rounded to f16 (11 bits): its rounding error, at most 2^-12 of each
//      term, is far below the output's own 8 or 11 bits.
// Then the CTAs of the cluster exchange maxima and sums over distributed
// shared memory, each adds up a share of the output over the CTAs in rank
// order, and each turns its own scores into weights with the query's final
// sums.  Nothing goes through global memory but inputs and outputs, and no
// result depends on timing.
//
// What bounds it: every row is read once per step, 2 * Hkv * D bytes, for
// 4 * Hq * D operations, i.e. 2 * (Hq / Hkv) operations a byte: memory, with
// the products far below the tensor rate even on mma.sync; tcgen05 would want
// 128 rows of one operand in shared memory, which here would mean writing
// every code back to shared memory as f16 first.
#pragma once

#include <cooperative_groups.h>

#include "hs_kv.cuh"

namespace hs {

struct AttendKernelArgs {
    const void* q;
    void* out;
    int32_t fp16, B, S, K, Hq, Hkv, G, R, L, NB, T, W;
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
    uint8_t* spill;  // per-token arrays of every CTA if shared memory cannot hold them
    // launch shape
    int32_t vec_q, vec_out;
    int32_t TS, TC, TL;      // tokens of a CTA at most; strides of the scale and score rows
    int32_t ngroups, nsub;   // query-head groups of a K/V head; parts of a CTA's tokens
    int32_t alias;           // 1: the output partials reuse the scales' memory
    int32_t token_bytes;     // bytes of the per-token arrays in the workspace
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

// Warps of a CTA at most: 128 registers a thread, more where the arrays are in the workspace
// (64-bit addresses).
constexpr int attend_warps(bool spill) { return spill ? 8 : 16; }

// Passes of the V phase, each for a piece of d.
constexpr int attend_value_passes(int D, int nt) {
    return D * nt <= 128 ? 1 : (D == 96 ? 3 : 2);
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

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A lane's share of a row piece that LANES lanes read together: WORDS words in
// loads of V words, load i at V * (i * LANES + lane), so that each load of the
// lanes covers contiguous bytes.
template <int WORDS>
constexpr int load_words() {
    return WORDS % 4 == 0 ? 4 : (WORDS % 2 == 0 ? 2 : 1);
}

// Byte (element) offset of word w of lane l's share.
template <int WORDS, int LANES>
__device__ __forceinline__ int word_at(int w, int l) {
    constexpr int V = load_words<WORDS>();
    return 4 * (V * ((w / V) * LANES + l) + w % V);
}

// `p` is the address of the lane's first load; zeros where off.
template <int WORDS, int LANES>
__device__ __forceinline__ void load_share(uint32_t (&r)[WORDS], const uint8_t* p, bool on) {
    constexpr int V = load_words<WORDS>();
#pragma unroll
    for (int i = 0; i < WORDS; i += V) {
        const uint8_t* at = p + 4 * LANES * i;
        if constexpr (V == 4) {
            uint4 x = make_uint4(0, 0, 0, 0);
            if (on) x = __ldg(reinterpret_cast<const uint4*>(at));
            r[i] = x.x;
            r[i + 1] = x.y;
            r[i + 2] = x.z;
            r[i + 3] = x.w;
        } else if constexpr (V == 2) {
            uint2 x = make_uint2(0, 0);
            if (on) x = __ldg(reinterpret_cast<const uint2*>(at));
            r[i] = x.x;
            r[i + 1] = x.y;
        } else {
            r[i] = on ? __ldg(reinterpret_cast<const uint32_t*>(at)) : 0u;
        }
    }
}

// The 16-bit elements that belong to a lane's words of a K row, as pairs.
template <int WORDS>
__device__ __forceinline__ void load_query(uint32_t (&r)[2 * WORDS], const uint16_t* p, int c,
                                           bool on, bool vec) {
#pragma unroll
    for (int w = 0; w < WORDS; ++w) {
        const uint16_t* at = p + word_at<WORDS, 4>(w, c);
        if (vec) {
            uint2 x = make_uint2(0, 0);
            if (on) x = __ldg(reinterpret_cast<const uint2*>(at));
            r[2 * w] = x.x;
            r[2 * w + 1] = x.y;
        } else {
            r[2 * w] = on ? (uint32_t)__ldg(at) | ((uint32_t)__ldg(at + 1) << 16) : 0u;
            r[2 * w + 1] = on ? (uint32_t)__ldg(at + 2) | ((uint32_t)__ldg(at + 3) << 16) : 0u;
        }
    }
}

// A pair of bf16 or f16 elements as 32-bit values.
__device__ __forceinline__ float2 pair(uint32_t w, int fp16) {
    if (fp16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// Largest over the 8 lanes that share c (lanes differ in g).
__device__ __forceinline__ float max_over_g(float x) {
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}

template <int CODE, int D, int NT, bool SPILL>
__global__ void __launch_bounds__(32 * attend_warps(SPILL), 1)
    attend_kernel(const AttendKernelArgs a) {
    // A K row is taken in KP pieces and the V phase in VP passes over the tokens, each for a
    // piece of d, so that the tiles in flight and the accumulators fit 128 registers.
    constexpr int KP = D > 128 ? 2 : 1;
    constexpr int KW = D / 16 / KP;       // words of a lane's share of a K piece = steps
    constexpr int VP = attend_value_passes(D, NT);
    constexpr int VD = D / VP;
    constexpr int VW = VD / 32;           // words of a lane's share of a V piece
    // tiles (K: pieces of tiles) in flight in registers
    constexpr int KRING = KP > 1 || (NT == 2 && D > 64) ? 2 : 3;
    constexpr int VRING = D > 128 || (NT == 2 && D > 64) ? 2 : 3;
    extern __shared__ __align__(16) uint8_t smem[];
    cg::cluster_group cluster = cg::this_cluster();
    const int P = (int)cluster.num_blocks();
    const int rank = (int)cluster.block_rank();
    const int bs = blockIdx.x / P;
    const int b = bs / a.S, st = bs - b * a.S;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int nthreads = blockDim.x, nwarps = nthreads >> 5;
    const int g = lane >> 2, c = lane & 3;
    const int GP = a.ngroups * 8 * NT;    // padded query heads of a K/V head
    const int HP = a.Hkv * GP;

    // Shared memory: maxima and sums [nsub][HP], factors [P][Hq], the query's log2-sum-exp
    // [Hq], output partials [Hq][D]; then (or in the workspace) the per-token arrays.
    __shared__ int s_scan[33];
    float* s_max = reinterpret_cast<float*>(smem);
    float* s_sum = s_max + a.nsub * HP;
    float* s_factor = s_sum + a.nsub * HP;
    float* s_lse = s_factor + ((P * a.Hq + 3) & ~3);
    float* s_out = s_lse + ((a.Hq + 3) & ~3);
    const int out_floats = a.alias ? max(a.Hq * D, 2 * a.Hkv * a.TC) : a.Hq * D;
    uint8_t* token = SPILL ? a.spill + (size_t)blockIdx.x * a.token_bytes
                           : reinterpret_cast<uint8_t*>(s_out + out_floats);
    int* t_loc = reinterpret_cast<int*>(token);  // [TS] row, -1 past the last
    int* t_pos = t_loc + a.TS;                   // [TS] position in the sequence
    int* t_src = t_pos + a.TS;                   // [TS] entry of the selection
    float* t_score = reinterpret_cast<float*>(t_src + a.TS);           // [Hq][TL], base-2 logits
    float* t_scale = !SPILL && a.alias ? s_out : t_score + a.Hq * a.TL;  // [2 Hkv][TC]

    const long long entry0 = (long long)bs * a.K;
    const int req = __ldg(a.req + b);
    const bool known = req >= 0 && req < a.R;
    // The CTA's entries, masked ones dropped.
    int live = 0;
    for (int i0 = 0; i0 < a.TS; i0 += nthreads) {
        const int i = i0 + tid;
        const int j = ((i >> 4) * P + rank) * 16 + (i & 15);
        int loc = -1, t = 0;
        if (i < a.TS && j < a.K) {
            loc = __ldg(a.locs + entry0 + j);
            t = __ldg(a.topk + entry0 + j);
            if (!known || loc < 0 || loc >= a.num_rows || t < 0 || t >= a.L) {
                loc = -1;
                if (a.weights) a.weights[entry0 + j] = 0.f;
            }
        }
        int n = __syncthreads_count(loc >= 0);
        int at = live + tid;  // a full turn, or one that only lacks its end, stays in place
        if (__syncthreads_or(loc >= 0 && tid >= n)) {
            at = live + block_exclusive_scan(loc >= 0, s_scan, &n);
        }
        if (loc >= 0) {
            t_loc[at] = loc;
            t_pos[at] = t;
            t_src[at] = j;
        }
        live += n;
    }
    const int tiles = (live + 15) >> 4;
    for (int i = live + tid; i < tiles * 16; i += nthreads) t_loc[i] = -1;
    __syncthreads();
    {
        const int per = 2 * a.Hkv;
        const float* base = a.scales + (long long)(known ? req : 0) * a.NB * per;
        for (int i = tid; i < tiles * 16 * per; i += nthreads) {
            const int tok = i / per, ch = i - tok * per;
            t_scale[ch * a.TC + tok] =
                tok < live ? __ldg(base + (long long)(t_pos[tok] / a.T) * per + ch) : 0.f;
        }
    }
    __syncthreads();

    const int groups = a.Hkv * a.ngroups;
    for (int task = warp; task < groups * a.nsub; task += nwarps) {
        const int sub = task / groups, hg = task - sub * groups;
        const int h = hg / a.ngroups, j0 = (hg - h * a.ngroups) * 8 * NT;
        const int tile0 = tiles * sub / a.nsub, tile1 = tiles * (sub + 1) / a.nsub;
        const float* sk = t_scale + h * a.TC;
        const float* sv = t_scale + (a.Hkv + h) * a.TC;
        float* score = t_score + (h * a.G + j0) * a.TL;

        // ---- scores --------------------------------------------------------------
        float top[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) top[nt][0] = top[nt][1] = -INFINITY;
        {
            const uint8_t* kbase = a.rows + h * D + word_at<KW, 4>(0, c);
            uint32_t kr[KRING][2][KW];
            // piece u: part u % KP of tile u / KP
            auto load_k = [&](uint32_t (&r)[2][KW], int u) {
                const int tile = tile0 + u / KP;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int loc = tile < tile1 ? t_loc[tile * 16 + g + 8 * i] : -1;
                    load_share<KW, 4>(r[i], kbase + (u % KP) * (D / KP) + (long long)loc * a.W,
                                      loc >= 0);
                }
            };
            if constexpr (KP == 1) {
#pragma unroll
                for (int i = 0; i < KRING; ++i) load_k(kr[i], i);
            }

            // Queries as the B operand: lane (g, c) holds head g's elements of its words.
            uint32_t qf[NT][KP][KW][2];
            float factor[NT][2];  // of the scores of heads 2 c and 2 c + 1
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int j = j0 + nt * 8 + g;
                const long long at = b * a.q_stride[0] + st * a.q_stride[1] +
                                     (long long)(h * a.G + j) * a.q_stride[2];
                float peak = 0.f;
#pragma unroll
                for (int p = 0; p < KP; ++p) {
                    uint32_t raw[2 * KW];
                    load_query<KW>(raw, static_cast<const uint16_t*>(a.q) + at + p * (D / KP), c,
                                   j < a.G, a.vec_q);
#pragma unroll
                    for (int w = 0; w < KW; ++w) {
                        qf[nt][p][w][0] = raw[2 * w];
                        qf[nt][p][w][1] = raw[2 * w + 1];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float2 x = pair(raw[2 * w + i], a.fp16);
                            peak = fmaxf(peak, fmaxf(fabsf(x.x), fabsf(x.y)));
                        }
                    }
                }
                peak = fmaxf(peak, __shfl_xor_sync(0xffffffffu, peak, 1));
                peak = fmaxf(peak, __shfl_xor_sync(0xffffffffu, peak, 2));
                // the head's largest element goes to [2^14, 2^15), f16's top
                int e = (int)(__float_as_uint(peak) >> 23) - 127;
                e = e < -100 ? -100 : e;
                const float up = __uint_as_float((uint32_t)(14 - e + 127) << 23);
#pragma unroll
                for (int p = 0; p < KP; ++p) {
#pragma unroll
                    for (int w = 0; w < KW; ++w) {
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float2 x = pair(qf[nt][p][w][i], a.fp16);
                            qf[nt][p][w][i] = pack_half2(x.x * up, x.y * up);
                        }
                    }
                }
                const float down =
                    __uint_as_float((uint32_t)(e - 14 + 127) << 23) * a.scale_log2;
                factor[nt][0] = __shfl_sync(0xffffffffu, down, 8 * c);
                factor[nt][1] = __shfl_sync(0xffffffffu, down, 8 * c + 4);
            }

            if constexpr (KP > 1) {  // no registers for them before
#pragma unroll
                for (int i = 0; i < KRING; ++i) load_k(kr[i], i);
            }

            const int pieces = (tile1 - tile0) * KP;
            float s[NT][2][4];
            for (int u = 0; u < pieces; u += KRING) {
#pragma unroll
                for (int i = 0; i < KRING; ++i) {
                    if (u + i >= pieces) break;
                    const int part = i % KP;
                    if (part == 0) {
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int k = 0; k < 4; ++k) s[nt][0][k] = s[nt][1][k] = 0.f;
                    }
#pragma unroll
                    for (int w = 0; w < KW; ++w) {
                        uint32_t a0, a1, a2, a3;
                        halves<CODE>(kr[i][0][w], a0, a2);
                        halves<CODE>(kr[i][1][w], a1, a3);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma(s[nt][w & 1], a0, a1, a2, a3, qf[nt][part][w][0],
                                qf[nt][part][w][1]);
                    }
                    load_k(kr[i], u + i + KRING);
                    if (part != KP - 1) continue;
                    const int t0 = (tile0 + (u + i) / KP) * 16 + g;
                    const bool on0 = t0 < live, on1 = t0 + 8 < live;
                    const float k0 = sk[t0], k1 = sk[t0 + 8];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const float f = factor[nt][k];
                            const float v0 =
                                on0 ? (s[nt][0][k] + s[nt][1][k]) * (k0 * f) : -INFINITY;
                            const float v1 =
                                on1 ? (s[nt][0][k + 2] + s[nt][1][k + 2]) * (k1 * f) : -INFINITY;
                            top[nt][k] = fmaxf(top[nt][k], fmaxf(v0, v1));
                            const int j = nt * 8 + 2 * c + k;
                            if (j0 + j < a.G) {
                                score[j * a.TL + t0] = v0;
                                score[j * a.TL + t0 + 8] = v1;
                            }
                        }
                    }
                }
            }
        }

        // ---- values --------------------------------------------------------------
        const uint8_t* vbase = a.rows + (a.Hkv + h) * D + word_at<VW, 8>(0, g);
        uint32_t vr[VRING][4][VW];
        auto load_v = [&](uint32_t (&r)[4][VW], int tile, int part) {
            int4 loc = make_int4(-1, -1, -1, -1);
            if (tile < tile1) loc = *reinterpret_cast<const int4*>(t_loc + tile * 16 + 4 * c);
            const uint8_t* p = vbase + part * VD;
            load_share<VW, 8>(r[0], p + (long long)loc.x * a.W, loc.x >= 0);
            load_share<VW, 8>(r[1], p + (long long)loc.y * a.W, loc.y >= 0);
            load_share<VW, 8>(r[2], p + (long long)loc.z * a.W, loc.z >= 0);
            load_share<VW, 8>(r[3], p + (long long)loc.w * a.W, loc.w >= 0);
        };
#pragma unroll
        for (int i = 0; i < VRING; ++i) load_v(vr[i], tile0 + i, 0);

        float head_max[NT], head_sum[NT];  // of head g of each 8-head tile
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const float m0 = max_over_g(top[nt][0]), m1 = max_over_g(top[nt][1]);
            // head g's maximum lies with lanes c = g / 2
            const float from0 = __shfl_sync(0xffffffffu, m0, g >> 1);
            const float from1 = __shfl_sync(0xffffffffu, m1, g >> 1);
            head_max[nt] = g & 1 ? from1 : from0;
        }
        float ref = 0.f;  // largest V scale of the task's tokens
        for (int i = tile0 * 16 + lane; i < tile1 * 16; i += 32) ref = fmaxf(ref, sv[i]);
        ref = max_over_g(ref);
        ref = fmaxf(ref, __shfl_xor_sync(0xffffffffu, ref, 1));
        ref = fmaxf(ref, __shfl_xor_sync(0xffffffffu, ref, 2));
        const float inv = ref > 0.f ? 1.f / ref : 0.f;
        __syncwarp();  // the warp's scores are in shared memory

        float fold[NT][2];  // of the partial outputs of heads 2 c and 2 c + 1
#pragma unroll
        for (int part = 0; part < VP; ++part) {
            float o[2 * VW][NT][4] = {};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) head_sum[nt] = 0.f;
            for (int tile = tile0; tile < tile1; tile += VRING) {
#pragma unroll
                for (int i = 0; i < VRING; ++i) {
                    if (tile + i >= tile1) break;
                    const int t0 = (tile + i) * 16 + 4 * c;
                    const float4 scale = *reinterpret_cast<const float4*>(sv + t0);
                    uint32_t pf[NT][2];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (j0 + nt * 8 + g < a.G)
                            z = *reinterpret_cast<const float4*>(score + (nt * 8 + g) * a.TL + t0);
                        const float m = head_max[nt] == -INFINITY ? 0.f : head_max[nt];
                        const float p0 = exp2_fast(z.x - m), p1 = exp2_fast(z.y - m);
                        const float p2 = exp2_fast(z.z - m), p3 = exp2_fast(z.w - m);
                        head_sum[nt] += (p0 + p1) + (p2 + p3);
                        pf[nt][0] = pack_half2(p0 * (scale.x * inv), p1 * (scale.y * inv));
                        pf[nt][1] = pack_half2(p2 * (scale.z * inv), p3 * (scale.w * inv));
                    }
#pragma unroll
                    for (int w = 0; w < VW; ++w) {
                        // bytes of neighbouring tokens side by side: d, d + 1 | d + 2, d + 3
                        const uint32_t x0 = __byte_perm(vr[i][0][w], vr[i][1][w], 0x5140);
                        const uint32_t y0 = __byte_perm(vr[i][0][w], vr[i][1][w], 0x7362);
                        const uint32_t x1 = __byte_perm(vr[i][2][w], vr[i][3][w], 0x5140);
                        const uint32_t y1 = __byte_perm(vr[i][2][w], vr[i][3][w], 0x7362);
                        uint32_t a0, a1, a2, a3;
                        halves<CODE>(x0, a0, a1);
                        halves<CODE>(x1, a2, a3);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma(o[2 * w][nt], a0, a1, a2, a3, pf[nt][0], pf[nt][1]);
                        halves<CODE>(y0, a0, a1);
                        halves<CODE>(y1, a2, a3);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma(o[2 * w + 1][nt], a0, a1, a2, a3, pf[nt][0], pf[nt][1]);
                    }
                    load_v(vr[i], tile + i + VRING, part);
                }
            }
            if (part + 1 < VP) {
#pragma unroll
                for (int i = 0; i < VRING; ++i) load_v(vr[i], tile0 + i, part + 1);
            }
            if (part == 0) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float x = head_sum[nt];
                    x += __shfl_xor_sync(0xffffffffu, x, 1);
                    x += __shfl_xor_sync(0xffffffffu, x, 2);
                    if (c == 0) {
                        const int at = sub * HP + h * GP + j0 + nt * 8 + g;
                        s_max[at] = head_max[nt];
                        s_sum[at] = x;
                    }
                }
            }
            // The output may take the scales' place: then every warp has one task and VP is 1,
            // and all are done with the scales here.  Several parts of a slice have one task a
            // warp too; their outputs are added in order, relative to their common maximum.
            if (a.alias || a.nsub > 1) __syncthreads();
            if (part == 0) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        fold[nt][k] = ref;
                        if (a.nsub > 1) {
                            const int at = h * GP + j0 + nt * 8 + 2 * c + k;
                            float m = -INFINITY;
                            for (int u = 0; u < a.nsub; ++u) m = fmaxf(m, s_max[u * HP + at]);
                            fold[nt][k] *=
                                exp2_fast(s_max[sub * HP + at] - (m == -INFINITY ? 0.f : m));
                        }
                    }
                }
            }
            for (int u = 0; u < a.nsub; ++u) {
                if (u == sub) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const int j = j0 + nt * 8 + 2 * c + k;
                            if (j >= a.G) continue;
                            const float f = fold[nt][k];
                            float* row = s_out + (h * a.G + j) * D + part * VD;
#pragma unroll
                            for (int w = 0; w < VW; ++w) {
                                float4* dst =
                                    reinterpret_cast<float4*>(row + word_at<VW, 8>(w, g));
                                float4 x =
                                    make_float4(o[2 * w][nt][k] * f, o[2 * w][nt][k + 2] * f,
                                                o[2 * w + 1][nt][k] * f,
                                                o[2 * w + 1][nt][k + 2] * f);
                                if (u > 0) {
                                    const float4 y = *dst;
                                    x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
                                }
                                *dst = x;
                            }
                        }
                    }
                }
                if (a.nsub > 1) __syncthreads();
            }
        }
    }
    if (a.nsub > 1) {  // one maximum and sum per head of the slice
        for (int i = tid; i < HP; i += nthreads) {
            float m = -INFINITY, l = 0.f;
            for (int u = 0; u < a.nsub; ++u) m = fmaxf(m, s_max[u * HP + i]);
            const float safe = m == -INFINITY ? 0.f : m;
            for (int u = 0; u < a.nsub; ++u)
                l += s_sum[u * HP + i] * exp2_fast(s_max[u * HP + i] - safe);
            s_max[i] = m;
            s_sum[i] = l;
        }
    }

    // ---- the cluster's result ----------------------------------------------------
    cluster.sync();
    for (int i = tid; i < a.Hq; i += nthreads) {
        const int at = (i / a.G) * GP + i % a.G;
        float m = -INFINITY, l = 0.f;
        for (int r = 0; r < P; ++r) m = fmaxf(m, cluster.map_shared_rank(s_max, r)[at]);
        const float safe = m == -INFINITY ? 0.f : m;
        for (int r = 0; r < P; ++r) {
            const float f = exp2_fast(cluster.map_shared_rank(s_max, r)[at] - safe);
            s_factor[r * a.Hq + i] = f;
            l += cluster.map_shared_rank(s_sum, r)[at] * f;
        }
        const float norm = l == 0.f ? 0.f : 1.f / l;
        for (int r = 0; r < P; ++r) s_factor[r * a.Hq + i] *= norm;
        const float lse2 = m + log2f(l);
        s_lse[i] = l == 0.f ? INFINITY : lse2;  // weights of an empty query: 0
        if (rank == 0 && a.lse)
            a.lse[(long long)bs * a.Hq + i] = l == 0.f ? -INFINITY : lse2 * 0.69314718056f;
    }
    __syncthreads();
    {
        const int quads = a.Hq * (D / 4);
        const int lo = quads * rank / P, hi = quads * (rank + 1) / P;
        for (int i = lo + tid; i < hi; i += nthreads) {
            const int head = i / (D / 4), d = (i - head * (D / 4)) * 4;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int r = 0; r < P; ++r) {
                const float4 y =
                    reinterpret_cast<const float4*>(cluster.map_shared_rank(s_out, r))[i];
                const float f = s_factor[r * a.Hq + head];
                x = make_float4(x.x + y.x * f, x.y + y.y * f, x.z + y.z * f, x.w + y.w * f);
            }
            const long long at = b * a.out_stride[0] + st * a.out_stride[1] +
                                 head * a.out_stride[2] + d;
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
            uint16_t* dst = static_cast<uint16_t*>(a.out) + at;
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
    if (a.weights || a.acc) {
        for (int i = tid; i < live; i += nthreads) {
            float w = 0.f;
#pragma unroll 4
            for (int j = 0; j < a.Hq; ++j) w += exp2_fast(t_score[j * a.TL + i] - s_lse[j]);
            if (a.acc) atomicAdd(a.acc + (long long)req * a.L + t_pos[i], w);
            if (a.weights) a.weights[entry0 + t_src[i]] = w;
        }
    }
    cluster.sync();  // no CTA leaves while another reads its shared memory
}

template <int CODE, int D, int NT, bool SPILL>
cudaError_t run_one(const AttendShape& sh, cudaStream_t s) {
    static SmemOptIn opt;
    auto* kernel = attend_kernel<CODE, D, NT, SPILL>;
    cudaError_t e = ensure_smem(kernel, sh.smem, &opt);
    if (e != cudaSuccess) return e;
    if (sh.P > 8) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(sh.a.B * sh.a.S * sh.P);
    cfg.blockDim = dim3(sh.threads);
    cfg.dynamicSmemBytes = sh.smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = sh.P;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, sh.a);
}

template <int CODE, int D>
cudaError_t run_dim(const AttendShape& sh, cudaStream_t s) {
    if (sh.spill) return run_one<CODE, D, 1, true>(sh, s);
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
