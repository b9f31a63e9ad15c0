// Launch shape of hs_attend (the kernel is in hs_attend.cuh).
#include <atomic>
#include <cmath>
#include <cstring>

#include "hs_attend.cuh"

namespace hs {
namespace {

constexpr size_t kSmSmem = 228 * 1024;             // of an SM; a CTA takes 1 KB more than it asks
constexpr int kSmCols = 512;                       // tensor-memory columns of an SM
constexpr size_t kStatic = 512;                    // static arrays of the kernel, rounded up
constexpr size_t kMaxSmem = kSmSmem - 1024 - kStatic;
constexpr size_t kHalfSmem = kSmSmem / 2 - 1024 - kStatic;  // two CTAs an SM

// Memory of a CTA for a cluster of P with at most `most` warps a CTA, and the shape that follows.
void set_cluster(const hs_kv_format& f, const hs_attend_args& a, int P, int most, AttendShape* sh) {
    AttendKernelArgs& k = sh->a;
    sh->P = P;
    const long long chunks = ((long long)a.top_k + 15) / 16;
    k.TS = (int)(16 * ((chunks + P - 1) / P));
    if (k.TS == 0) k.TS = 16;
    k.TC = k.TS + 4;  // scale rows in different banks
    const int D = f.head_dim, G = a.num_heads / f.num_kv_heads;
    int columns, groups, nsub, task_tiles;
    const auto split = [&](int nt) {
        sh->nt = nt;
        columns = nt == 0 ? 4 : 8 * nt;  // query heads of a task
        k.ngroups = (G + columns - 1) / columns;
        groups = f.num_kv_heads * k.ngroups;
        // Warps: one task each where they fit; with few heads, a CTA's tokens are split into parts
        // so that it has 8 warps or a few more; with many, a warp takes several in turn.
        nsub = groups >= 8 ? 1 : (8 + groups - 1) / groups;
        if (nsub > 1 && groups * nsub > most) nsub = most / groups;
        if (nsub > k.TS / 16) nsub = k.TS / 16;
        if (nsub < 1) nsub = 1;
        task_tiles = (k.TS / 16 + nsub - 1) / nsub;
    };
    // Query heads a warp serves with one reading of keys and values.  Up to 4 heads, a fragment of
    // 8 columns holds two tiles (nt 0), which halves the scores' tensor memory: slices twice as
    // long fit, and fit two CTAs an SM (16 requests of 8192 tokens, 8 heads of 64, 4 query heads each:
    // 48.5 us; 59.4 with one tile and columns left empty).  Above 8 heads, 16 columns (nt 2)
    // convert every code once instead of twice (128 requests of 2048 tokens, one K/V head of 64, 32
    // query heads: 29.2 us against 37.1), but leave half the tasks, and with under 4 tiles a task the
    // warps run short (64 requests of 512 tokens, one K/V head of 128, 16 query heads: 15.1 us
    // against 12.7).  Wider heads have the registers for one tile and 8 columns only.
    if (sh->spill) {
        split(1);
    } else if (G <= 4 && D <= 192) {
        split(0);
    } else if (G > 8 && D <= 128) {
        split(2);
        if (task_tiles < 4) split(1);
    } else {
        split(1);
    }
    k.nsub = nsub;
    const int rounds = (groups * nsub + most - 1) / most;
    const int warps = (groups * nsub + rounds - 1) / rounds;
    sh->threads = 32 * warps;
    k.alias = rounds == 1;
    k.task_cols = sh->nt == 0 ? 4 * ((task_tiles + 1) / 2) : 4 * sh->nt * task_tiles;
    const long long need = (long long)rounds * ((warps + 3) / 4) * k.task_cols;
    int cols = 32;
    while (cols < need && cols < 2 * kSmCols) cols *= 2;
    k.cols = cols;
    const size_t HP = (size_t)groups * columns;
    const size_t fixed = 4 * ((2 * nsub + 1) * HP + (((size_t)P * a.num_heads + 3) & ~(size_t)3));
    const size_t scale = (size_t)2 * f.num_kv_heads * k.TC, weight = (size_t)groups * k.TS;
    const size_t token = 4 * ((size_t)3 * k.TS + (scale > weight ? scale : weight));
    const size_t out = 4 * (size_t)a.num_heads * (D + 4);
    const size_t queue = (size_t)warps * attend_stages(D) * 16 * D;
    const size_t rest = k.alias ? (out > queue ? out : queue) : out + queue;
    if (sh->spill) {
        sh->smem = fixed + rest;
        const size_t score = (size_t)rounds * warps * k.task_cols * 128;
        k.token_bytes = (int32_t)((token + score + 15) & ~(size_t)15);
        k.cols = 0;
    } else {
        sh->smem = fixed + token + rest;
        // Tensor memory is handed out to CTAs as they ask and a cluster must not wait for it while
        // another cluster's CTA waits elsewhere: a CTA takes shared memory in proportion to
        // its columns, so that an SM never holds CTAs of these kernels with more columns than it has.
        const size_t share = kSmSmem / kSmCols * (size_t)cols - 1024 - kStatic;
        if (sh->smem < share) sh->smem = share;
        // Kernels of other libraries, on another stream, follow no such rule.  A lone CTA then waits for
        // its columns until theirs end.  But CTAs of a cluster wait for one another with their columns
        // held, and two kernels that both do could wait for each other.  So they take half an SM:
        // beside them fits only what takes the other half at most, and that blocks them only if
        // its clusters hold over half of the columns.  (In CTAs of under 8 warps more than two
        // would fit an SM: 1000 requests of 64 rows, one K/V head of 64, 4 query heads, take 19 us, and
        // 33 us if single CTAs took half an SM too.)
        if (P > 1 && sh->smem < kHalfSmem) sh->smem = kHalfSmem;
    }
}

bool fits(const AttendShape& sh, size_t smem) {
    return sh.smem <= smem && sh.a.cols <= kSmCols;
}

// CTAs in clusters of P that the current device runs at once with one CTA an SM: fewer than
// SMs where P does not divide a group of SMs (on one GB300, 152 in clusters of 1 or 2, 144 of
// 4, 120 of 8, 112 of 16).  Asked once per device and cluster size.
int resident(int P) {
    constexpr int kDevices = 64;
    static std::atomic<int> known[kDevices][kMaxCluster + 1];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) dev = kDevices;
    int n = dev < kDevices ? known[dev][P].load(std::memory_order_relaxed) : 0;
    if (n == 0) {
        n = attend_resident(P, kMaxSmem);
        if (n <= 0) n = 112;
        if (dev < kDevices) known[dev][P].store(n, std::memory_order_relaxed);
    }
    return n;
}

// The same for a shape: registers leave room for two CTAs of up to 8 warps an SM, and then a
// cluster of an even P needs P / 2 SMs.
int slots(const AttendShape& sh) {
    if (sh.threads > 256 || sh.smem > kHalfSmem) return resident(sh.P);
    return 2 * resident(sh.P % 2 == 0 ? sh.P / 2 : sh.P);
}

// Estimated time of a call in us.  The CTAs run in rounds, with one CTA an SM or, if there are more
// than that, two.  A round has a start and an end of about 10 us; a token takes 9 ns and 10 ns for
// every KB gathered (16 with two CTAs an SM, which each get 60% of the speed of one), where the work
// on a head's codes counts as 0.125 KB and a query head as 2.5 bytes.  The constants are fitted to all
// cluster sizes of 44 calls with weights, of 1 to 256 queries and 512 to 8192 tokens, whole and
// with rows left out: the size of the least estimate is 0.5% slower than the fastest one on
// average, 9% at worst.  64 requests of 2048 tokens and 8 heads of 128, for one, took 62.5 us in
// clusters of 4, 63.5 of 2, 75.8 of 6 and 67.1 of 8.
double cost(const hs_kv_format& f, const hs_attend_args& a, const AttendShape& sh) {
    const int one = resident(sh.P), two = slots(sh);
    const double kb =
        f.num_kv_heads * (2e-3 * f.head_dim + 0.125 * sh.a.ngroups) + 2.5e-3 * a.num_heads;
    double t = 0;
    for (long long left = (long long)a.batch * a.steps * sh.P; left > 0;) {
        const bool shared = left > one && two > one;
        t += shared ? 11.5 + sh.a.TS * (0.009 + 0.016 * kb) : 10 + sh.a.TS * (0.009 + 0.010 * kb);
        left -= shared ? two : one;
    }
    return t;
}

// The cluster sizes tried for a call: CTAs of 64 tokens or more, if any of those fit.
bool worth(const hs_attend_args& a, int P) { return P == 1 || a.top_k >= 64 * P; }

// The first cluster size that fits, among those worth it or else among all; with the scores and
// the arrays by token in the workspace if none does.  Host only.
AttendShape first_shape(const hs_kv_format& f, const hs_attend_args& a) {
    AttendShape sh;
    std::memset(&sh, 0, sizeof(sh));
    for (int pass = 0; pass < 2; ++pass) {
        for (int P = 1; P <= kMaxCluster && (pass == 1 || worth(a, P)); ++P) {
            set_cluster(f, a, P, attend_warps(f.head_dim, false), &sh);
            if (fits(sh, kMaxSmem)) return sh;
        }
    }
    // Wide outputs of many heads leave no room for the queues of that many warps (128 heads of 256
    // are 133 KB, the queues of 8 warps 98): as many as fit, and at least one does, take more turns.
    sh.spill = true;
    for (int most = attend_warps(f.head_dim, true); most > 0; --most) {
        set_cluster(f, a, kMaxCluster, most, &sh);
        if (fits(sh, kMaxSmem)) break;
    }
    return sh;
}

// Of the cluster sizes that fit and are worth it, the one of the least estimated time.
AttendShape shape_of(const hs_kv_format& f, const hs_attend_args& a) {
    AttendShape best = first_shape(f, a);
    if (best.spill || best.P == kMaxCluster || !worth(a, best.P + 1)) return best;
    double least = cost(f, a, best);
    AttendShape sh = best;
    for (int P = best.P + 1; P <= kMaxCluster && worth(a, P); P += P < 8 ? 1 : 2) {
        set_cluster(f, a, P, attend_warps(f.head_dim, false), &sh);
        if (!fits(sh, kMaxSmem)) continue;
        const double t = cost(f, a, sh);
        if (t < least) least = t, best = sh;
    }
    return best;
}

}  // namespace

size_t attend_workspace(const hs_kv_format& f, const hs_attend_args& a) {
    const AttendShape sh = first_shape(f, a);
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
    k.block = Divisor::by(f.block_tokens);
    k.NB = (a.max_seq_len - 1) / f.block_tokens + 1;
    k.W = f.item_size_bytes;
    k.scale_log2 = a.sm_scale * 1.4426950408889634f;
    k.vec_q = (uintptr_t)a.q_dev % 8 == 0;
    k.vec_out = (uintptr_t)a.out_dev % 8 == 0;
    k.vec_scale = (uintptr_t)a.scales_dev % 16 == 0 && f.num_kv_heads % 2 == 0;
    for (int i = 0; i < 3; ++i) {
        k.q_stride[i] = a.q_stride[i];
        k.out_stride[i] = a.out_stride[i];
        k.vec_q = k.vec_q && a.q_stride[i] % 4 == 0;
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
                             a.top_k, a.acc_dev, a.num_requests, a.max_seq_len, true, s);
}

}  // namespace hs
