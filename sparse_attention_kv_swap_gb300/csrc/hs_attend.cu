// Launch shape of hs_attend (the kernel is in hs_attend.cuh).
#include <cmath>
#include <cstring>

#include "hs_attend.cuh"

namespace hs {
namespace {

constexpr int kSms = 152;
constexpr int kMaxCluster = 16;
constexpr size_t kMaxSmem = 227 * 1024;

// Shared-memory layout of a CTA: bytes without the per-token arrays, and theirs.
void sizes(const hs_kv_format& f, const hs_attend_args& a, int P, AttendShape* sh, size_t* fixed,
           size_t* token) {
    AttendKernelArgs& k = sh->a;
    k.TS = (int)((((long long)a.top_k + P - 1) / P + 15) / 16 * 16);
    if (k.TS == 0) k.TS = 16;
    // Score rows 4 floats past a multiple of 32 and scale rows 4 past their length: the rows
    // that a warp's lanes touch together fall into different banks.
    k.TL = (k.TS + 31) / 32 * 32 + 4;
    k.TC = k.TS + 4;
    const int D = f.head_dim, G = a.num_heads / f.num_kv_heads;
    k.ngroups = (G + 8 * sh->nt - 1) / (8 * sh->nt);
    const int groups = f.num_kv_heads * k.ngroups;
    // Warps: one task each where they fit; with few heads, a slice is split into parts so
    // that a CTA has 8 warps or a few more; with many, a warp takes several in turn.
    const int most = attend_max_warps(D, sh->nt);
    int nsub = groups >= 8 ? 1 : (8 + groups - 1) / groups;
    if (groups * nsub > most) nsub = most / groups > 0 ? most / groups : 1;
    if (nsub > k.TS / 16) nsub = k.TS / 16;
    k.nsub = nsub;
    const int rounds = (groups * nsub + most - 1) / most;
    sh->threads = 32 * ((groups * nsub + rounds - 1) / rounds);
    const size_t HP = (size_t)groups * 8 * sh->nt;
    *fixed = 4 * ((size_t)a.num_heads * D + 2 * nsub * HP +
                  (((size_t)P * a.num_heads + 3) & ~(size_t)3) + ((a.num_heads + 3) & ~3));
    *token = 4 * ((size_t)2 * k.TS + (size_t)2 * f.num_kv_heads * k.TC +
                  (size_t)a.num_heads * k.TL);
}

// P: enough CTAs that every SM has two, in slices of 64 tokens or more, and
// slices of at most 256 tokens while a portable cluster allows; twice the
// cluster where the scores do not fit; the workspace where that is not enough.
AttendShape shape_of(const hs_kv_format& f, const hs_attend_args& a) {
    AttendShape sh;
    std::memset(&sh, 0, sizeof(sh));
    const int G = a.num_heads / f.num_kv_heads;
    sh.nt = G > 8 && f.head_dim <= 128 ? 2 : 1;
    const long long queries = (long long)a.batch * a.steps;
    int P = 1;
    while (P < 8 && (a.top_k > 256 * P || (a.top_k > 64 * P && queries * P < 2 * kSms))) P *= 2;
    size_t fixed, token;
    sizes(f, a, P, &sh, &fixed, &token);
    while (fixed + token > kMaxSmem && P < kMaxCluster) {
        P *= 2;
        sizes(f, a, P, &sh, &fixed, &token);
    }
    if (fixed + token > kMaxSmem) {
        sh.nt = 1;
        sh.spill = true;
        sizes(f, a, P, &sh, &fixed, &token);
    }
    token = (token + 15) & ~(size_t)15;
    sh.P = P;
    sh.smem = fixed + (sh.spill ? 0 : token);
    sh.a.token_bytes = (int32_t)token;
    return sh;
}

}  // namespace

size_t attend_workspace(const hs_kv_format& f, const hs_attend_args& a) {
    const AttendShape sh = shape_of(f, a);
    return sh.spill ? (size_t)a.batch * a.steps * sh.P * sh.a.token_bytes : 0;
}

cudaError_t launch_attend(const hs_kv_format& f, const hs_attend_args& a, cudaStream_t s) {
    AttendShape sh = shape_of(f, a);
    AttendKernelArgs& k = sh.a;
    k.q = a.q_dev;
    k.out = a.out_dev;
    k.fp16 = a.dtype == HS_DTYPE_FP16;
    k.B = a.batch;
    k.S = a.steps;
    k.K = a.top_k;
    k.Hq = a.num_heads;
    k.Hkv = f.num_kv_heads;
    k.G = a.num_heads / f.num_kv_heads;
    k.R = a.num_requests;
    k.L = a.max_seq_len;
    k.T = f.block_tokens;
    k.NB = (a.max_seq_len - 1) / f.block_tokens + 1;
    k.W = f.item_size_bytes;
    k.scale_log2 = a.sm_scale * 1.4426950408889634f;
    k.vec_q = (uintptr_t)a.q_dev % 16 == 0;
    k.vec_out = (uintptr_t)a.out_dev % 8 == 0;
    for (int i = 0; i < 3; ++i) {
        k.q_stride[i] = a.q_stride[i];
        k.out_stride[i] = a.out_stride[i];
        k.vec_q = k.vec_q && a.q_stride[i] % 8 == 0;
        k.vec_out = k.vec_out && a.out_stride[i] % 4 == 0;
    }
    k.rows = static_cast<const uint8_t*>(a.rows_dev);
    k.num_rows = a.num_rows;
    k.locs = a.locs_dev;
    k.topk = a.topk_dev;
    k.req = a.req_dev;
    k.scales = a.scales_dev;
    k.lse = a.lse_dev;
    k.weights = a.weights_dev;
    k.acc = a.steps == 1 ? a.acc_dev : nullptr;
    k.spill = static_cast<uint8_t*>(a.workspace_dev);
    const cudaError_t e = f.code == HS_KV_E4M3 ? attend_run_e4m3(sh, f.head_dim, s)
                                               : attend_run_int8(sh, f.head_dim, s);
    if (e != cudaSuccess || !a.acc_dev || a.steps == 1) return e;
    // A token may be selected in several steps: its sums follow the steps.
    return launch_accumulate(a.weights_dev, a.topk_dev, a.req_dev, nullptr, a.batch, a.steps,
                             a.top_k, a.acc_dev, a.num_requests, a.max_seq_len, s);
}

}  // namespace hs
