// Launch shapes of hs_attend over everything that hs_attend accepts, evaluated on the host: every
// shape has to fit an SM and the kernel's layout has to fit the shape.  Prints "ok" and the
// number of shapes, or what does not fit.
#include "hs_attend.cu"

#include <cstdio>
#include <initializer_list>

namespace hs {
cudaError_t attend_run_e4m3(const AttendShape&, int, cudaStream_t) { return cudaErrorUnknown; }
cudaError_t attend_run_int8(const AttendShape&, int, cudaStream_t) { return cudaErrorUnknown; }
// the CTAs that a GB300 runs at once
int attend_resident(int P, size_t) { return P <= 2 ? 152 / P * P : P <= 4 ? 144 / P * P : 112 / P * P; }
cudaError_t launch_accumulate(const float*, const int32_t*, const int32_t*, const int32_t*, int32_t,
                              int32_t, int32_t, float*, int32_t, int32_t, bool, cudaStream_t) {
    return cudaErrorUnknown;
}
}  // namespace hs

using namespace hs;

static const char* wrong(const hs_kv_format& f, const hs_attend_args& a, const AttendShape& sh) {
    const AttendKernelArgs& k = sh.a;
    const int D = f.head_dim, G = a.num_heads / f.num_kv_heads;
    const int columns = sh.nt == 0 ? 4 : 8 * sh.nt, warps = sh.threads / 32;
    if (sh.smem > 227 * 1024 - kStatic) return "shared memory of an SM";
    if (sh.P < 1 || sh.P > 16 || sh.threads % 32 != 0 || warps < 1 || warps > attend_warps(D, sh.spill))
        return "cluster and threads";
    if ((sh.nt == 0 && D > 192) || (sh.nt == 2 && D > 128) || (sh.spill && sh.nt != 1)) return "kernel";
    if (k.TS % 16 != 0 || k.TS < 16 || (long long)k.TS * sh.P < a.top_k) return "tokens of a CTA";
    if (k.ngroups * columns < G || k.nsub < 1 || k.nsub > k.TS / 16) return "groups";
    const int groups = f.num_kv_heads * k.ngroups, tasks = groups * k.nsub;
    const int rounds = (tasks + warps - 1) / warps;
    if (k.alias && rounds != 1) return "outputs over queues in use";
    if ((k.alias || k.nsub > 1) && tasks != warps) return "block barriers that some warps skip";
    const int tiles = (k.TS / 16 + k.nsub - 1) / k.nsub;
    if (k.task_cols < (sh.nt == 0 ? 4 * ((tiles + 1) / 2) : 4 * sh.nt * tiles)) return "scores";
    const size_t HP = (size_t)groups * columns;
    const size_t scale = (size_t)2 * f.num_kv_heads * k.TC, weight = (size_t)groups * k.TS;
    const size_t token = 4 * ((size_t)3 * k.TS + (scale > weight ? scale : weight));
    const size_t queue = (size_t)warps * attend_stages(D) * 16 * D;
    const size_t out = (size_t)4 * a.num_heads * (D + 4);
    size_t bytes = 4 * ((2 * k.nsub + 1) * HP + (((size_t)sh.P * a.num_heads + 3) & ~(size_t)3));
    bytes += k.alias ? (queue > out ? queue : out) : queue + out;
    if (sh.spill) {
        if (k.token_bytes % 16 != 0 ||
            (size_t)k.token_bytes < token + (size_t)rounds * warps * k.task_cols * 128)
            return "workspace of a CTA";
        if (attend_workspace(f, a) != (size_t)a.batch * a.steps * sh.P * k.token_bytes)
            return "workspace";
    } else {
        bytes += token;
        if (attend_workspace(f, a) != 0) return "workspace that is not used";
        if (k.cols < 32 || k.cols > 512 || (k.cols & (k.cols - 1)) != 0 ||
            k.cols < rounds * ((warps + 3) / 4) * k.task_cols)
            return "tensor memory";
        // CTAs that wait for one another leave others half an SM at most
        if (sh.P > 1 && 2 * (sh.smem + 1024 + kStatic) < (size_t)228 * 1024) return "half of an SM";
        // as much of the SM's shared memory as of its tensor memory
        if ((sh.smem + 1024 + kStatic) * 512 < (size_t)228 * 1024 * k.cols) return "share of an SM";
    }
    return bytes > sh.smem ? "layout" : nullptr;
}

int main() {
    long long shapes = 0, bad = 0;
    for (int D : {32, 64, 96, 128, 192, 256}) {
        for (int heads = 1; heads <= HS_MAX_KV_HEADS; ++heads) {
            hs_kv_format f = {heads, D, 64, HS_KV_E4M3, 2 * heads * D};
            for (int G = 1; heads * G <= HS_MAX_KV_HEADS; ++G) {
                for (int K : {0, 1, 15, 16, 64, 100, 333, 512, 1000, 2048, 3000, 4096, 5300, 8192, 12000,
                              16384, 20000, 40000, 65536, 131072, 1 << 20, 1 << 22}) {
                    for (int batch : {1, 40, 1000}) {
                        hs_attend_args a;
                        std::memset(&a, 0, sizeof(a));
                        a.batch = batch;
                        a.steps = 1;
                        a.top_k = K;
                        a.num_heads = heads * G;
                        ++shapes;
                        const char* w = wrong(f, a, shape_of(f, a));
                        if (w && ++bad <= 20)
                            std::printf("D %d, %d x %d heads, %d entries, batch %d: %s (%zu bytes)\n", D,
                                        heads, G, K, batch, w, shape_of(f, a).smem);
                    }
                }
            }
        }
    }
    if (bad == 0) std::printf("ok %lld\n", shapes);
    else std::printf("%lld of %lld shapes\n", bad, shapes);
    return bad != 0;
}
