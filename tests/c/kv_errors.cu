// A call of the 8-bit rows whose launch fails returns HS_ERR_CUDA and takes the runtime's last
// error with it: the next call that asks for it would report a failure of its own otherwise.
// The launches and the last error are stand-ins; nothing runs on a GPU.
#include <cuda_runtime.h>

#include <cstdio>

static cudaError_t device(int* d) { return *d = 0, cudaSuccess; }
#define cudaGetDevice device

#include "hs_kv.cuh"

static cudaError_t last = cudaSuccess;
static cudaError_t take_last() {
    const cudaError_t e = last;
    last = cudaSuccess;
    return e;
}
#define cudaGetLastError take_last

#include "hs_kv_api.cu"

namespace hs {
static cudaError_t fail() { return last = cudaErrorInvalidValue; }
LayerView layer_view(const Dims&, unsigned char*, int, const unsigned char*, unsigned char*) { return {}; }
Workspace workspace_view(const Dims&, unsigned char*) { return {}; }
cudaError_t launch_quantize(QuantizeArgs, bool, cudaStream_t) { return fail(); }
cudaError_t launch_compact(CompactArgs, cudaStream_t) { return fail(); }
cudaError_t launch_accumulate(const float*, const int32_t*, const int32_t*, const int32_t*, int32_t,
                              int32_t, int32_t, float*, int32_t, int32_t, bool, cudaStream_t) {
    return fail();
}
cudaError_t launch_evict(const float*, const int32_t*, const int32_t*, int32_t, int32_t, int32_t,
                         int32_t, int32_t, int32_t*, int32_t*, float*, cudaStream_t) {
    return fail();
}
size_t attend_workspace(const hs_kv_format&, const hs_attend_args&) { return 0; }
cudaError_t launch_attend(const hs_kv_format&, const hs_attend_args&, cudaStream_t) { return fail(); }
}  // namespace hs

static int bad = 0;
static void check(const char* what, int rc) {
    if (rc != HS_ERR_CUDA || last != cudaSuccess) {
        std::printf("%s: returned %d, last error %d\n", what, rc, (int)last);
        bad = 1;
    }
    last = cudaSuccess;
}

int main() {
    hs_kv_format f = {2, 64, 16, HS_KV_E4M3, 256};
    char *at = reinterpret_cast<char*>(0x100000), *far = reinterpret_cast<char*>(0x900000);
    float *x = reinterpret_cast<float*>(at), *y = reinterpret_cast<float*>(far);
    int32_t* i = reinterpret_cast<int32_t*>(at);
    hs_kv_input in = {at, at, HS_DTYPE_BF16, {1, 1, 1}, {1, 1, 1}};
    check("hs_quantize_kv", hs_quantize_kv(&f, &in, i, i, i, 1, 1, at, x, 1, 64, nullptr));
    hs_state st = {};
    st.d.W = 256, st.d.layers = 1, st.d.R = 1, st.d.L = 64;
    st.host_pool_dev.push_back(nullptr);
    st.device_kv.push_back(nullptr);
    check("hs_append_kv", hs_append_kv(&st, 0, &f, &in, i, i, i, 1, 1, x, nullptr));
    hs_attend_args a = {};
    a.q_dev = at, a.out_dev = at, a.batch = 1, a.steps = 1, a.top_k = 4, a.num_heads = 2;
    a.num_requests = 1, a.max_seq_len = 64, a.rows_dev = at, a.num_rows = 4, a.locs_dev = i;
    a.topk_dev = i, a.req_dev = i, a.scales_dev = x;
    check("hs_attend", hs_attend(&f, &a, nullptr));
    check("hs_accumulate", hs_accumulate(x, i, i, nullptr, 1, 1, 4, x, 1, 64, nullptr));
    check("hs_evict", hs_evict(x, i, i, 1, 0, 4, 1, 64, i, i, nullptr, nullptr));
    check("hs_compact_kv",
          hs_compact_kv(&f, at, x, 1, 64, i, i, i, 1, 4, far, y, 1, 64, i, nullptr));
    // scales side by side (one request with 4 blocks of 2 x 2: 64 bytes) are not refused
    for (char* to : {at + 64, at - 16})
        check("hs_compact_kv beside its source's scales",
              hs_compact_kv(&f, at, x, 1, 64, i, i, i, 1, 4, far, reinterpret_cast<float*>(to), 1,
                            16, i, nullptr));
    if (!bad) std::printf("ok\n");
    return bad;
}
