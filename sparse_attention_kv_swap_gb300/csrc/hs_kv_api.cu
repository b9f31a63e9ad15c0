// Host side of the 8-bit key/value row calls of include/hisparse_swap.h:
// argument validation and launches on the caller's stream.
#include "hs_kv.cuh"

using namespace hs;

namespace {

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

bool overlap(const void* p, size_t p_bytes, const void* q, size_t q_bytes) {
    return (uintptr_t)p < (uintptr_t)q + q_bytes && (uintptr_t)q < (uintptr_t)p + p_bytes;
}

int32_t blocks_of(const hs_kv_format* f, int32_t L) { return (L - 1) / f->block_tokens + 1; }

// The runtime keeps a failure as its last error, which the next call that asks for it would
// report as its own.
int result(cudaError_t e) {
    if (e == cudaSuccess) return HS_OK;
    cudaGetLastError();
    return HS_ERR_CUDA;
}

constexpr int32_t kMaxCtas = 0x7fffffff;

// The input and the per-entry arrays of the two quantising calls.
int check_input(const hs_kv_format* f, const hs_kv_input* in, const int32_t* req,
                const int32_t* start, const int32_t* count, const float* scales, int32_t batch,
                int32_t max_count) {
    if (in->dtype < HS_DTYPE_BF16 || in->dtype > HS_DTYPE_FP32) return HS_ERR_INVALID_ARG;
    const size_t esz = in->dtype == HS_DTYPE_FP32 ? 4 : 2;
    if (!in->k_dev || !in->v_dev || !req || !start || !count || !scales)
        return HS_ERR_INVALID_ARG;
    if (!aligned(in->k_dev, esz) || !aligned(in->v_dev, esz) || !aligned(req, 4) ||
        !aligned(start, 4) || !aligned(count, 4) || !aligned(scales, 4))
        return HS_ERR_INVALID_ARG;
    const long long windows = ((long long)max_count + f->block_tokens - 2) / f->block_tokens + 1;
    if ((long long)batch * windows * 2 * f->num_kv_heads > kMaxCtas) return HS_ERR_UNSUPPORTED;
    return HS_OK;
}

int check_attend(const hs_kv_format* f, const hs_attend_args* a) {
    const int rc = hs_kv_format_check(f);
    if (rc != HS_OK) return rc;
    if (!a || a->batch < 0 || a->steps < 1 || a->top_k < 0 || a->num_heads < 1 ||
        a->num_heads % f->num_kv_heads != 0)
        return HS_ERR_INVALID_ARG;
    if (a->num_heads > HS_MAX_KV_HEADS) return HS_ERR_UNSUPPORTED;
    // clusters of up to 16 CTAs in one grid, and a slice's arrays counted in 32 bits
    if ((long long)a->batch * a->steps * 16 > kMaxCtas || a->top_k > (1 << 22))
        return HS_ERR_UNSUPPORTED;
    return HS_OK;
}

}  // namespace

extern "C" {

int hs_kv_format_check(const hs_kv_format* f) {
    if (!f) return HS_ERR_INVALID_ARG;
    if (f->num_kv_heads < 1 || f->head_dim < 1 || f->block_tokens < 1) return HS_ERR_INVALID_ARG;
    if (f->code != HS_KV_E4M3 && f->code != HS_KV_INT8) return HS_ERR_INVALID_ARG;
    if (f->num_kv_heads > HS_MAX_KV_HEADS || f->block_tokens > HS_MAX_KV_BLOCK)
        return HS_ERR_UNSUPPORTED;
    switch (f->head_dim) {
        case 32: case 64: case 96: case 128: case 192: case 256: break;
        default: return HS_ERR_UNSUPPORTED;
    }
    if (f->item_size_bytes % 16 != 0 || f->item_size_bytes < 2 * f->num_kv_heads * f->head_dim)
        return HS_ERR_INVALID_ARG;
    if (f->item_size_bytes > HS_MAX_ITEM_BYTES) return HS_ERR_UNSUPPORTED;
    return HS_OK;
}

int hs_quantize_kv(const hs_kv_format* fmt, const hs_kv_input* in, const int32_t* req_dev,
                   const int32_t* start_dev, const int32_t* count_dev, int32_t batch,
                   int32_t max_count, void* rows_dev, float* scales_dev, int32_t num_requests,
                   int32_t max_seq_len, void* stream) {
    int rc = hs_kv_format_check(fmt);
    if (rc != HS_OK) return rc;
    if (!in || batch < 0 || max_count < 0 || num_requests < 1 || max_seq_len < 1)
        return HS_ERR_INVALID_ARG;
    if (batch == 0 || max_count == 0) return HS_OK;
    rc = check_input(fmt, in, req_dev, start_dev, count_dev, scales_dev, batch, max_count);
    if (rc != HS_OK) return rc;
    if (!rows_dev || !aligned(rows_dev, 16)) return HS_ERR_INVALID_ARG;
    QuantizeArgs a = {};
    a.f = *fmt;
    a.in = *in;
    a.req = req_dev;
    a.start = start_dev;
    a.count = count_dev;
    a.batch = batch;
    a.max_count = max_count;
    a.rows = static_cast<uint8_t*>(rows_dev);
    a.scales = scales_dev;
    a.R = num_requests;
    a.L = max_seq_len;
    a.NB = blocks_of(fmt, max_seq_len);
    return result(launch_quantize(a, false, static_cast<cudaStream_t>(stream)));
}

int hs_append_kv(hs_state* st, int32_t layer_id, const hs_kv_format* fmt, const hs_kv_input* in,
                 const int32_t* req_dev, const int32_t* start_dev, const int32_t* count_dev,
                 int32_t batch, int32_t max_count, float* scales_dev, void* stream) {
    if (!st) return HS_ERR_INVALID_ARG;
    int rc = hs_kv_format_check(fmt);
    if (rc != HS_OK) return rc;
    if (!on_handle_device(st)) return HS_ERR_INVALID_ARG;
    const Dims& d = st->d;
    if (layer_id < 0 || layer_id >= d.layers || !in || batch < 0 || max_count < 0 ||
        fmt->item_size_bytes != d.W)
        return HS_ERR_INVALID_ARG;
    if (batch == 0 || max_count == 0) return HS_OK;
    rc = check_input(fmt, in, req_dev, start_dev, count_dev, scales_dev, batch, max_count);
    if (rc != HS_OK) return rc;
    QuantizeArgs a = {};
    a.f = *fmt;
    a.in = *in;
    a.req = req_dev;
    a.start = start_dev;
    a.count = count_dev;
    a.batch = batch;
    a.max_count = max_count;
    // the caller's writable memory, as in hs_append_rows
    a.rows = const_cast<uint8_t*>(st->host_pool_dev[layer_id]);
    a.scales = scales_dev;
    a.R = d.R;
    a.L = d.L;
    a.NB = blocks_of(fmt, d.L);
    a.d = d;
    a.lv = layer_view(d, st->state, layer_id, st->host_pool_dev[layer_id],
                      st->device_kv[layer_id]);
    a.status = workspace_view(d, st->ws).status;
    return result(launch_quantize(a, true, static_cast<cudaStream_t>(stream)));
}

size_t hs_attend_workspace_bytes(const hs_kv_format* fmt, const hs_attend_args* args) {
    if (check_attend(fmt, args) != HS_OK) return (size_t)-1;
    if (args->batch == 0) return 0;
    return attend_workspace(*fmt, *args);
}

int hs_attend(const hs_kv_format* fmt, const hs_attend_args* a, void* stream) {
    const int rc = check_attend(fmt, a);
    if (rc != HS_OK) return rc;
    if (a->dtype != HS_DTYPE_BF16 && a->dtype != HS_DTYPE_FP16) return HS_ERR_INVALID_ARG;
    if (a->num_requests < 1 || a->max_seq_len < 1 || a->num_rows < 0) return HS_ERR_INVALID_ARG;
    if (a->acc_dev && a->steps > 1 && !a->weights_dev) return HS_ERR_INVALID_ARG;
    if (a->batch == 0) return HS_OK;
    if (!a->q_dev || !a->out_dev || !a->req_dev) return HS_ERR_INVALID_ARG;
    if (a->top_k > 0 && (!a->locs_dev || !a->topk_dev || !a->scales_dev ||
                         (!a->rows_dev && a->num_rows > 0)))
        return HS_ERR_INVALID_ARG;
    if (!aligned(a->q_dev, 2) || !aligned(a->out_dev, 2) || !aligned(a->rows_dev, 16) ||
        !aligned(a->locs_dev, 4) || !aligned(a->topk_dev, 4) || !aligned(a->req_dev, 4) ||
        !aligned(a->scales_dev, 4) || !aligned(a->lse_dev, 4) || !aligned(a->weights_dev, 4) ||
        !aligned(a->acc_dev, 4) || !aligned(a->workspace_dev, 16))
        return HS_ERR_INVALID_ARG;
    const size_t need = attend_workspace(*fmt, *a);
    if (need > 0 && (!a->workspace_dev || a->workspace_bytes < need)) return HS_ERR_INVALID_ARG;
    return result(launch_attend(*fmt, *a, static_cast<cudaStream_t>(stream)));
}

int hs_accumulate(const float* weights_dev, const int32_t* topk_dev, const int32_t* req_dev,
                  const int32_t* counts_dev, int32_t batch, int32_t num_steps, int32_t top_k,
                  float* acc_dev, int32_t num_requests, int32_t max_seq_len, void* stream) {
    if (batch < 0 || num_steps < 1 || top_k < 0 || num_requests < 1 || max_seq_len < 1)
        return HS_ERR_INVALID_ARG;
    if (top_k > (1 << 22) || (long long)batch * 4 > kMaxCtas) return HS_ERR_UNSUPPORTED;
    if (batch == 0 || top_k == 0) return HS_OK;
    if (!weights_dev || !topk_dev || !req_dev || !acc_dev) return HS_ERR_INVALID_ARG;
    if (!aligned(weights_dev, 4) || !aligned(topk_dev, 4) || !aligned(req_dev, 4) ||
        !aligned(counts_dev, 4) || !aligned(acc_dev, 4))
        return HS_ERR_INVALID_ARG;
    return result(launch_accumulate(weights_dev, topk_dev, req_dev, counts_dev, batch, num_steps,
                                    top_k, acc_dev, num_requests, max_seq_len, false,
                                    static_cast<cudaStream_t>(stream)));
}

int hs_evict(const float* acc_dev, const int32_t* req_dev, const int32_t* seq_lens_dev,
             int32_t batch, int32_t recent, int32_t budget, int32_t num_requests,
             int32_t max_seq_len, int32_t* keep_dev, int32_t* kept_dev, float* kept_acc_dev,
             void* stream) {
    if (batch < 0 || budget < 1 || recent < 0 || recent > budget || num_requests < 1 ||
        max_seq_len < 1)
        return HS_ERR_INVALID_ARG;
    // the kernel counts positions, and CTAs of clusters of 8, in 32 bits
    if (max_seq_len > (1 << 30) || budget > (1 << 30) || (long long)batch * 8 > kMaxCtas)
        return HS_ERR_UNSUPPORTED;
    if (batch == 0) return HS_OK;
    if (!acc_dev || !req_dev || !seq_lens_dev || !keep_dev || !kept_dev)
        return HS_ERR_INVALID_ARG;
    if (!aligned(acc_dev, 4) || !aligned(req_dev, 4) || !aligned(seq_lens_dev, 4) ||
        !aligned(keep_dev, 4) || !aligned(kept_dev, 4) || !aligned(kept_acc_dev, 4))
        return HS_ERR_INVALID_ARG;
    return result(launch_evict(acc_dev, req_dev, seq_lens_dev, batch, recent, budget, num_requests,
                               max_seq_len, keep_dev, kept_dev, kept_acc_dev,
                               static_cast<cudaStream_t>(stream)));
}

int hs_compact_kv(const hs_kv_format* fmt, const void* src_rows_dev, const float* src_scales_dev,
                  int32_t src_requests, int32_t src_seq_len, const int32_t* src_req_dev,
                  const int32_t* keep_dev, const int32_t* kept_dev, int32_t batch, int32_t budget,
                  void* dst_rows_dev, float* dst_scales_dev, int32_t dst_requests,
                  int32_t dst_seq_len, const int32_t* dst_req_dev, void* stream) {
    const int rc = hs_kv_format_check(fmt);
    if (rc != HS_OK) return rc;
    if (batch < 0 || budget < 1 || src_requests < 1 || src_seq_len < 1 || dst_requests < 1 ||
        dst_seq_len < 1)
        return HS_ERR_INVALID_ARG;
    if (batch == 0) return HS_OK;
    if (!src_rows_dev || !src_scales_dev || !src_req_dev || !keep_dev || !kept_dev ||
        !dst_rows_dev || !dst_scales_dev || !dst_req_dev)
        return HS_ERR_INVALID_ARG;
    if (!aligned(src_rows_dev, 16) || !aligned(dst_rows_dev, 16) || !aligned(src_scales_dev, 4) ||
        !aligned(dst_scales_dev, 4) || !aligned(src_req_dev, 4) || !aligned(keep_dev, 4) ||
        !aligned(kept_dev, 4) || !aligned(dst_req_dev, 4))
        return HS_ERR_INVALID_ARG;
    const size_t W = fmt->item_size_bytes, block = sizeof(float) * 2 * fmt->num_kv_heads;
    if (overlap(src_rows_dev, (size_t)src_requests * src_seq_len * W, dst_rows_dev,
                (size_t)dst_requests * dst_seq_len * W) ||
        overlap(src_scales_dev, (size_t)src_requests * blocks_of(fmt, src_seq_len) * block,
                dst_scales_dev, (size_t)dst_requests * blocks_of(fmt, dst_seq_len) * block))
        return HS_ERR_INVALID_ARG;
    const int32_t most = budget < dst_seq_len ? budget : dst_seq_len;
    if ((long long)batch * blocks_of(fmt, most) * 2 * fmt->num_kv_heads > kMaxCtas)
        return HS_ERR_UNSUPPORTED;
    CompactArgs a = {};
    a.f = *fmt;
    a.src = static_cast<const uint8_t*>(src_rows_dev);
    a.src_scales = src_scales_dev;
    a.src_req = src_req_dev;
    a.keep = keep_dev;
    a.kept = kept_dev;
    a.dst = static_cast<uint8_t*>(dst_rows_dev);
    a.dst_scales = dst_scales_dev;
    a.dst_req = dst_req_dev;
    a.batch = batch;
    a.budget = budget;
    a.src_R = src_requests;
    a.src_L = src_seq_len;
    a.src_NB = blocks_of(fmt, src_seq_len);
    a.dst_R = dst_requests;
    a.dst_L = dst_seq_len;
    a.dst_NB = blocks_of(fmt, dst_seq_len);
    return result(launch_compact(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
