// Launch of hs_attend_prefix (the kernel is in hs_prefix.cuh), and the kernel that puts
// together the rows whose tokens fell to several CTAs.
//
// A CTA takes 32 rows of a K/V head, a lane a row, and 16 quads of their elements, a warp a quad, or 4
// quads, four warps a quad; partial outputs lie with consecutive rows side by side.  They come
// mostly out of L2; latencies bound it, so its launch and its plan overlap the end of
// prefix_kernel and the first parts are loaded while their factors are worked out.
#include "hs_prefix.cuh"

namespace hs {
namespace {

using prefix::Joined;
using prefix::Plan;

constexpr int kWarps = 16;
constexpr int kParts = 2 * kPrefixCtas;  // of a row at most

__global__ void __launch_bounds__(32 * kWarps, 2) combine_kernel(const PrefixArgs a, int D,
                                                              int groups, int split) {
    __shared__ Plan plan;
    __shared__ float s_factor[kParts][32];  // of a part of a row
    __shared__ float s_tmp[kWarps][32];
    __shared__ float4 s_y[kWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int pipes = prefix_pipes(D), tile_rows = kPrefixRows * pipes;
    // The plan's inputs come from before prefix_kernel, which lets this one start only after it has
    // itself waited for them (without prefixes there is no plan, and nothing is read).
    if (warp == 0) prefix::fill_plan(plan, a, tile_rows, kPrefixTokens);
    __syncthreads();
    const int units = plan.unit[a.P], ctas = prefix::working(units, a.ctas);
    const int slice = blockIdx.x / (a.Hkv * groups), hg = blockIdx.x - slice * a.Hkv * groups;
    const int h = hg / groups, all = a.B * a.S * a.G;
    const int i = (hg - h * groups) * 32 + lane;  // row of all batch rows
    const bool on = i < all;
    const prefix::Row at(a, 0, h, on ? i : 0);
    const long long out_row = ((long long)at.b * a.S + at.s) * a.Hq + at.head;
    int p = a.P - 1;  // the row's prefix: the last that begins at its batch row or before, and has rows
    while (p >= 0 && (plan.lo[p] > at.b || plan.hi[p] <= plan.lo[p])) --p;
    const bool some = on && p >= 0 && at.b < plan.hi[p] && plan.len[p] > 0;
    int first = 0, last = -1;  // CTAs with units of the row's tile
    int unit0 = 0, tile_row = 0, halves = 1;
    if (some) {
        const int rows = (plan.hi[p] - plan.lo[p]) * a.S * a.G;
        const int tiles = prefix::tiles_of(plan.len[p], kPrefixTokens);
        const int r = i - plan.lo[p] * a.S * a.G, row_tiles = (rows + tile_rows - 1) / tile_rows;
        tile_row = r % tile_rows;
        // Two pipelines that share the tile's rows leave a part each.
        if (pipes == 2 && rows - (r - tile_row) <= kPrefixRows) halves = 2;
        unit0 = plan.unit[p] + (h * row_tiles + r / tile_rows) * tiles;
        const int each = units / ctas, more = units % ctas;  // the first `more` CTAs have one more
        auto owner = [&](int unit) {
            const int edge = more * (each + 1);
            return unit < edge ? unit / (each + 1) : more + (unit - edge) / each;
        };
        first = owner(unit0);
        last = owner(unit0 + tiles - 1);
    }
    // Where one CTA has the whole tile, it has written the outputs.
    const bool mine = on && (!some || last > first);
    const int parts = some && mine ? (last - first + 1) * halves : 0;
    // A CTA's part lies in the place of its first segment if it begins within the tile, as all but the
    // tile's first CTA do; the second pipeline's, 128 rows on.
    const int later = some && prefix::first_unit(units, first, ctas) < unit0 ? 1 : 0;
    auto slot = [&](int c) {
        const int n = halves == 2 ? c >> 1 : c;
        return 2 * (first + n) + (n == 0 ? later : 0);
    };
    auto row_of = [&](int c) { return tile_row + (halves == 2 && (c & 1) ? kPrefixRows : 0); };
    wait_for_previous();
    release_next();
    // The first parts' outputs, on their way while the factors are worked out.
    const int quads = D / 4, d = (slice * kWarps + warp) / split, sub = warp % split;
    const float4* part = reinterpret_cast<const float4*>(a.part) + (long long)d * tile_rows;
    constexpr int kAhead = 6;
    float4 z[kAhead];
    const auto fetch = [&](int c0) {
#pragma unroll
        for (int c = 0; c < kAhead; ++c) {
            z[c] = make_float4(0.f, 0.f, 0.f, 0.f);
            const int at = sub + (c0 + c) * split;
            if (at < parts && d < quads)
                z[c] = ld(part + (long long)slot(at) * quads * tile_rows + row_of(at));
        }
    };
    fetch(0);
    // The factors of a row's parts, a warp every 16th of them: sums relative to the largest.
    float top = -INFINITY, first_sum = 0.f;
    bool nan = false;
    for (int c = warp; c < parts; c += kWarps) {
        const float2 x = ld(a.part_sum + slot(c) * tile_rows + row_of(c));
        if (c == warp) first_sum = x.y;
        const float y = x.x + log2f(x.y);  // -inf for a part without tokens
        s_factor[c][lane] = x.x;
        top = fmaxf(top, y);
        nan = nan || !(y == y);
    }
    s_tmp[warp][lane] = nan ? NAN : top;
    __syncthreads();
    top = s_tmp[0][lane];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) {
        const float y = s_tmp[w][lane];
        top = y == y && top == top ? fmaxf(top, y) : NAN;
    }
    __syncthreads();
    float sum = 0.f;
    for (int c = warp; c < parts; c += kWarps) {
        const float f = exp2f(s_factor[c][lane] - top);
        s_factor[c][lane] = f;
        sum += (c == warp ? first_sum : ld(a.part_sum + slot(c) * tile_rows + row_of(c)).y) * f;
    }
    s_tmp[warp][lane] = sum;
    // lse may be the given one itself, and a row's slices are CTAs of their own, which nothing orders: what
    // one of them writes must not be where the others read.  They read the copy that lies with the
    // parts then (copying always would cost 0.6 of 31.6 us for 21 requests of 3 steps), and a row without
    // parts keeps the given lse.
    const bool in_place = a.lse == a.join_lse;
    float other = -INFINITY;
    if (mine && a.join)
        other = parts > 0 && in_place ? ld(a.part_join + slot(0) * tile_rows + row_of(0))
                                      : ld(a.join_lse + out_row);
    __syncthreads();
    sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) sum += s_tmp[w][lane];
    const Joined j(some ? top + log2f(sum) : -INFINITY, other);
    if (mine && warp == 0 && slice == 0 && a.lse && (parts > 0 || !in_place)) a.lse[out_row] = j.lse;
    const float by = some ? j.mine / sum : 0.f;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c0 = 0; sub + c0 * split < parts; c0 += kAhead) {
        if (c0 > 0) fetch(c0);
#pragma unroll
        for (int c = 0; c < kAhead; ++c) {
            const int at = sub + (c0 + c) * split;
            const float f = at < parts ? s_factor[at][lane] : 0.f;
            if (f == 0.f) continue;  // a part without tokens is not written
            y = make_float4(y.x + z[c].x * f, y.y + z[c].y * f, y.z + z[c].z * f, y.w + z[c].w * f);
        }
    }
    if (split > 1) {
        s_y[warp][lane] = y;
        __syncthreads();
        if (sub > 0) return;
        for (int i = 1; i < split; ++i) {
            const float4 x = s_y[warp + i][lane];
            y = make_float4(y.x + x.x, y.y + x.y, y.z + x.z, y.w + x.w);
        }
    }
    if (!mine || d >= quads) return;
    y = make_float4(y.x * by, y.y * by, y.z * by, y.w * by);
    if (j.other > 0.f) {
        const uint2 z = prefix::load4(a.join + at.at(a.join_stride) + 4 * d, a.vec_join);
        const float2 z0 = prefix::pair(z.x, a.fp16), z1 = prefix::pair(z.y, a.fp16);
        y = make_float4(y.x + z0.x * j.other, y.y + z0.y * j.other, y.z + z1.x * j.other,
                        y.w + z1.y * j.other);
    }
    prefix::store4(a.out + at.at(a.out_stride) + 4 * d, prefix::unpair(y.x, y.y, a.fp16),
                   prefix::unpair(y.z, y.w, a.fp16), a.vec_out);
}

// CTAs of the kernel: one an SM of the current device.
int prefix_ctas() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1) {
        cudaGetLastError();
        sms = 152;
    }
    return sms < kPrefixCtas ? sms : kPrefixCtas;
}

// The tensor map of the store.  The encoder is the driver's; its entry point is looked up once.
cudaError_t make_map(const hs_kv_format& f, const hs_prefix_args& x, CUtensorMap* map) {
    using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static std::atomic<void*> known{nullptr};
    void* fn = known.load(std::memory_order_acquire);
    if (!fn) {
        cudaDriverEntryPointQueryResult found;
        const cudaError_t e = cudaGetDriverEntryPointByVersion(
            "cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found);
        if (e != cudaSuccess) return e;
        if (!fn || found != cudaDriverEntryPointSuccess) return cudaErrorNotSupported;
        known.store(fn, std::memory_order_release);
    }
    const int D = f.head_dim, box_bytes = prefix_box(D);
    const cuuint64_t W = (cuuint64_t)f.item_size_bytes;
    const cuuint64_t dims[3] = {W, (cuuint64_t)x.max_seq_len, (cuuint64_t)x.num_requests};
    const cuuint64_t strides[2] = {W, W * (cuuint64_t)x.max_seq_len};
    const cuuint32_t box[3] = {(cuuint32_t)box_bytes, (cuuint32_t)kPrefixTokens, 1};
    const cuuint32_t step[3] = {1, 1, 1};
    const CUresult r = reinterpret_cast<Encode>(fn)(
        map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(x.rows_dev), dims, strides, box,
        step, CU_TENSOR_MAP_INTERLEAVE_NONE,
        box_bytes == 128  ? CU_TENSOR_MAP_SWIZZLE_128B
        : box_bytes == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                          : CU_TENSOR_MAP_SWIZZLE_32B,
        CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

size_t part_bytes(const hs_kv_format& f, int ctas) {
    return (size_t)ctas * 2 * kPrefixRows * prefix_pipes(f.head_dim) * f.head_dim * sizeof(float);
}

}  // namespace

size_t prefix_workspace(const hs_kv_format& f) {
    const int ctas = prefix_ctas();
    return part_bytes(f, ctas) + (size_t)ctas * 2 * kPrefixRows * prefix_pipes(f.head_dim) *
                                     (sizeof(float2) + sizeof(float));
}

cudaError_t launch_prefix(const hs_kv_format& f, const hs_prefix_args& x, cudaStream_t s) {
    PrefixArgs a = {};
    a.q = static_cast<const uint16_t*>(x.q_dev);
    a.out = static_cast<uint16_t*>(x.out_dev);
    a.fp16 = x.dtype == HS_DTYPE_FP16;
    a.B = x.batch;
    a.S = x.steps;
    a.Hq = x.num_heads;
    a.Hkv = f.num_kv_heads;
    a.G = x.num_heads / f.num_kv_heads;
    a.R = x.num_requests;
    a.L = x.max_seq_len;
    a.NB = (x.max_seq_len - 1) / f.block_tokens + 1;
    a.W = f.item_size_bytes;
    a.P = x.num_prefixes;
    a.block = Divisor::by(f.block_tokens);
    a.even = f.block_tokens % 16 == 0 && x.sm_scale >= 0.f;
    a.scale_log2 = fabsf(x.sm_scale) * 1.4426950408889634f;
    a.k_sign = x.sm_scale < 0.f ? -1.f : 1.f;
    a.vec_q = (uintptr_t)x.q_dev % 16 == 0;
    a.vec_out = (uintptr_t)x.out_dev % 8 == 0;
    a.vec_join = (uintptr_t)x.join_out_dev % 8 == 0;
    for (int i = 0; i < 3; ++i) {
        a.q_stride[i] = x.q_stride[i];
        a.out_stride[i] = x.out_stride[i];
        a.join_stride[i] = x.join_stride[i];
        a.vec_q = a.vec_q && x.q_stride[i] % 8 == 0;
        a.vec_out = a.vec_out && x.out_stride[i] % 4 == 0;
        a.vec_join = a.vec_join && x.join_stride[i] % 4 == 0;
    }
    a.rows = static_cast<const uint8_t*>(x.rows_dev);
    a.scales = x.scales_dev;
    a.prefix = x.prefix_dev;
    a.lens = x.lens_dev;
    a.starts = x.starts_dev;
    a.lse = x.lse_dev;
    a.join = static_cast<const uint16_t*>(x.join_out_dev);
    a.join_lse = x.join_lse_dev;
    a.ctas = prefix_ctas();
    uint8_t* ws = static_cast<uint8_t*>(x.workspace_dev);
    a.part = reinterpret_cast<float*>(ws);
    a.part_sum = reinterpret_cast<float2*>(ws + part_bytes(f, a.ctas));
    a.part_join = reinterpret_cast<float*>(a.part_sum + (size_t)a.ctas * 2 * kPrefixRows *
                                                            prefix_pipes(f.head_dim));
    if (a.P > 0) {
        CUtensorMap map;
        cudaError_t e = make_map(f, x, &map);
        if (e != cudaSuccess) return e;
        e = f.code == HS_KV_E4M3 ? prefix_run_e4m3(a, map, f.head_dim, s)
                                 : prefix_run_int8(a, map, f.head_dim, s);
        if (e != cudaSuccess) return e;
    }
    const int groups = (int)(((long long)a.B * a.S * a.G + 31) / 32);
    // Where that leaves SMs idle, four warps share a quad's parts.
    const int quads = f.head_dim / 4;
    const int split = (long long)a.Hkv * groups * ((quads + kWarps - 1) / kWarps) * 4 <= a.ctas ? 4 : 1;
    const int slices = (quads * split + kWarps - 1) / kWarps;
    return launch_chained(combine_kernel, a.Hkv * groups * slices, 32 * kWarps, 0, 0, s, a,
                          f.head_dim, groups, split);
}

}  // namespace hs
