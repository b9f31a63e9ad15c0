// Host side of the calls around a decode step of include/hisparse_swap.h: argument
// validation and launches on the caller's stream.
#include "hs_step.cuh"

using namespace hs;

namespace {

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

int result(cudaError_t e) {
    if (e == cudaSuccess) return HS_OK;
    cudaGetLastError();  // not the next call's
    return HS_ERR_CUDA;
}

constexpr long long kMaxCtas = 0x7fffffff;

bool known_dim(int32_t d) {
    return d == 32 || d == 64 || d == 96 || d == 128 || d == 192 || d == 256;
}

// Sizes that hs_select_workspace_bytes and hs_select_blocks share.
int check_select_sizes(int32_t batch, int32_t steps, int32_t max_seq_len, int32_t block_tokens) {
    if (batch < 0 || steps < 1 || max_seq_len < 1 || block_tokens < 1) return HS_ERR_INVALID_ARG;
    if (steps > HS_MAX_STEPS || block_tokens > HS_MAX_KV_BLOCK ||
        (max_seq_len - 1) / block_tokens + 1 > HS_MAX_SELECT_BLOCKS)
        return HS_ERR_UNSUPPORTED;
    // CTAs are counted in 32 bits
    if ((long long)batch * (HS_MAX_SELECT_BLOCKS / kSelectChunk) > kMaxCtas) return HS_ERR_UNSUPPORTED;
    return HS_OK;
}

// Bytes of error bounds: one for every step of a CTA that scores.
size_t select_bytes(int32_t batch, int32_t steps, int32_t max_seq_len, int32_t block_tokens) {
    const size_t blocks = (size_t)(max_seq_len - 1) / block_tokens + 1;
    return 4 * (size_t)batch * steps * ((blocks + kSelectChunk - 1) / kSelectChunk);
}

int check_prefix(const hs_kv_format* f, const hs_prefix_args* a) {
    const int rc = hs_kv_format_check(f);
    if (rc != HS_OK) return rc;
    if (!a || a->batch < 0 || a->steps < 1 || a->num_heads < 1 || a->num_prefixes < 0 ||
        a->num_heads % f->num_kv_heads != 0)
        return HS_ERR_INVALID_ARG;
    if (a->num_heads > HS_MAX_KV_HEADS || a->num_prefixes > HS_MAX_PREFIXES)
        return HS_ERR_UNSUPPORTED;
    // rows are counted in 32 bits, with those that a last tile lacks
    if (a->batch > 0 && a->steps > (kMaxCtas - 4096) / a->num_heads / a->batch)
        return HS_ERR_UNSUPPORTED;
    return HS_OK;
}

}  // namespace

extern "C" {

int hs_norm_rope(const hs_norm_rope_args* a, void* stream) {
    if (!a || a->batch < 0 || a->tokens < 0 || a->num_heads < 0 || a->num_kv_heads < 0 ||
        a->dtype < HS_DTYPE_BF16 || a->dtype > HS_DTYPE_FP32 || a->rot_dim < 0 ||
        a->rot_dim > a->head_dim || a->rot_dim % 16 != 0 || a->num_axes < 1 ||
        (a->adjacent != 0 && a->adjacent != 1))
        return HS_ERR_INVALID_ARG;
    if (a->head_dim < 1) return HS_ERR_INVALID_ARG;
    if (!known_dim(a->head_dim) || a->num_axes > HS_MAX_ROPE_AXES) return HS_ERR_UNSUPPORTED;
    if ((a->q_weight_dev || a->k_weight_dev) && !(a->eps > 0.f)) return HS_ERR_INVALID_ARG;
    const long long heads = (long long)a->num_heads + a->num_kv_heads;
    const long long tokens = (long long)a->batch * a->tokens;
    if (tokens == 0 || heads == 0) return HS_OK;
    // items, with those that a last CTA looks at past the end, are counted in 32 bits
    if (heads > (1 << 20) || tokens > kMaxCtas / heads - (1 << 14)) return HS_ERR_UNSUPPORTED;
    const size_t esz = a->dtype == HS_DTYPE_FP32 ? 4 : 2;
    if ((a->num_heads > 0 && (!a->q_dev || !a->q_out_dev)) ||
        (a->num_kv_heads > 0 && (!a->k_dev || !a->k_out_dev)) ||
        (a->rot_dim > 0 && (!a->pos_dev || !a->turns_dev)))
        return HS_ERR_INVALID_ARG;
    if (!aligned(a->q_dev, esz) || !aligned(a->k_dev, esz) || !aligned(a->q_out_dev, esz) ||
        !aligned(a->k_out_dev, esz) || !aligned(a->q_weight_dev, 4) ||
        !aligned(a->k_weight_dev, 4) || !aligned(a->pos_dev, 4) || !aligned(a->turns_dev, 8) ||
        !aligned(a->axis_dev, 4) || !aligned(a->count_dev, 4))
        return HS_ERR_INVALID_ARG;
    return result(launch_norm_rope(*a, static_cast<cudaStream_t>(stream)));
}

int hs_bound_keys(const void* k_dev, const int64_t* k_stride, int32_t dtype, int32_t num_kv_heads,
                  int32_t head_dim, int32_t block_tokens, const int32_t* req_dev,
                  const int32_t* start_dev, const int32_t* count_dev, int32_t batch,
                  int32_t max_count, void* bounds_dev, int32_t num_requests, int32_t max_seq_len,
                  void* stream) {
    if (!k_stride || batch < 0 || max_count < 0 || num_requests < 1 || max_seq_len < 1 ||
        num_kv_heads < 1 || head_dim < 1 || block_tokens < 1 ||
        (dtype != HS_DTYPE_BF16 && dtype != HS_DTYPE_FP16))
        return HS_ERR_INVALID_ARG;
    if (!known_dim(head_dim) || num_kv_heads > HS_MAX_KV_HEADS || block_tokens > HS_MAX_KV_BLOCK)
        return HS_ERR_UNSUPPORTED;
    if (batch == 0 || max_count == 0) return HS_OK;
    if (!k_dev || !req_dev || !start_dev || !count_dev || !bounds_dev) return HS_ERR_INVALID_ARG;
    if (!aligned(k_dev, 2) || !aligned(bounds_dev, 2) || !aligned(req_dev, 4) ||
        !aligned(start_dev, 4) || !aligned(count_dev, 4))
        return HS_ERR_INVALID_ARG;
    BoundArgs a = {};
    const long long windows = ((long long)max_count + block_tokens - 2) / block_tokens + 1;
    const long long slabs = ((long long)num_kv_heads * head_dim + 255) / 256;
    if (windows > kMaxCtas / slabs / batch) return HS_ERR_UNSUPPORTED;
    a.k = static_cast<const uint8_t*>(k_dev);
    a.vec_k = aligned(k_dev, 16);
    for (int i = 0; i < 3; ++i) {
        a.stride[i] = k_stride[i];
        a.vec_k = a.vec_k && k_stride[i] % 8 == 0;
    }
    a.vec_bounds = aligned(bounds_dev, 16);
    a.fp16 = dtype == HS_DTYPE_FP16;
    a.Hkv = num_kv_heads;
    a.D = head_dim;
    a.T = block_tokens;
    a.batch = batch;
    a.max_count = max_count;
    a.R = num_requests;
    a.L = max_seq_len;
    a.NB = (max_seq_len - 1) / block_tokens + 1;
    a.req = req_dev;
    a.start = start_dev;
    a.count = count_dev;
    a.bounds = static_cast<uint8_t*>(bounds_dev);
    a.windows = (int32_t)windows;
    a.slabs = (int32_t)slabs;
    return result(launch_bound(a, static_cast<cudaStream_t>(stream)));
}

size_t hs_select_workspace_bytes(int32_t batch, int32_t steps, int32_t max_seq_len,
                                 int32_t block_tokens) {
    if (check_select_sizes(batch, steps, max_seq_len, block_tokens) != HS_OK) return (size_t)-1;
    return select_bytes(batch, steps, max_seq_len, block_tokens);
}

int hs_select_blocks(const hs_select_args* a, void* stream) {
    if (!a || a->num_kv_heads < 1 || a->num_heads < 1 || a->num_heads % a->num_kv_heads != 0 ||
        a->head_dim < 1 || a->num_requests < 1 || a->select < 1 || a->first < 0 || a->last < 0 ||
        a->first > a->select || a->last > a->select - a->first ||
        (a->dtype != HS_DTYPE_BF16 && a->dtype != HS_DTYPE_FP16))
        return HS_ERR_INVALID_ARG;
    const int rc = check_select_sizes(a->batch, a->steps, a->max_seq_len, a->block_tokens);
    if (rc != HS_OK) return rc;
    const int32_t width = a->num_kv_heads > HS_MAX_KV_HEADS ? 0 : a->num_kv_heads * a->head_dim;
    if (width == 0 || !known_dim(a->head_dim) || a->num_heads > HS_MAX_KV_HEADS ||
        width > HS_MAX_SELECT_WIDTH || width * a->steps > 2 * HS_MAX_SELECT_WIDTH ||
        a->select > HS_MAX_SELECT_BLOCKS || (long long)a->select * a->block_tokens > (1 << 30))
        return HS_ERR_UNSUPPORTED;
    if (a->batch == 0) return HS_OK;
    if (!a->q_dev || !a->bounds_dev || !a->req_dev || !a->seq_lens_dev || !a->topk_dev ||
        !a->scores_dev || !a->workspace_dev)
        return HS_ERR_INVALID_ARG;
    if (!aligned(a->q_dev, 2) || !aligned(a->bounds_dev, 2) || !aligned(a->req_dev, 4) ||
        !aligned(a->seq_lens_dev, 4) || !aligned(a->blocks_dev, 4) || !aligned(a->topk_dev, 4) ||
        !aligned(a->scores_dev, 4) || !aligned(a->workspace_dev, 4))
        return HS_ERR_INVALID_ARG;
    if (a->workspace_bytes < select_bytes(a->batch, a->steps, a->max_seq_len, a->block_tokens))
        return HS_ERR_INVALID_ARG;
    return result(launch_select(*a, static_cast<cudaStream_t>(stream)));
}

size_t hs_prefix_workspace_bytes(const hs_kv_format* fmt, const hs_prefix_args* args) {
    if (check_prefix(fmt, args) != HS_OK) return (size_t)-1;
    if (args->batch == 0) return 0;
    return prefix_workspace(*fmt);
}

int hs_attend_prefix(const hs_kv_format* fmt, const hs_prefix_args* a, void* stream) {
    const int rc = check_prefix(fmt, a);
    if (rc != HS_OK) return rc;
    if (a->dtype != HS_DTYPE_BF16 && a->dtype != HS_DTYPE_FP16) return HS_ERR_INVALID_ARG;
    if (a->num_requests < 1 || a->max_seq_len < 1 || !a->join_out_dev != !a->join_lse_dev)
        return HS_ERR_INVALID_ARG;
    // tiles of rows and tokens are counted in 32 bits; a copy's strides have 40
    const long long rows = (long long)a->batch * a->steps * (a->num_heads / fmt->num_kv_heads);
    const long long tiles = (a->max_seq_len - 1) / kPrefixTokens + 1;
    const long long row_tiles = (rows + kPrefixRows - 1) / kPrefixRows + a->num_prefixes;
    if (row_tiles * fmt->num_kv_heads > INT32_MAX / tiles ||
        (long long)fmt->item_size_bytes > ((1ll << 40) - 1) / a->max_seq_len)
        return HS_ERR_UNSUPPORTED;
    if (a->batch == 0) return HS_OK;
    if (!a->q_dev || !a->out_dev) return HS_ERR_INVALID_ARG;
    if (a->num_prefixes > 0 && (!a->rows_dev || !a->scales_dev || !a->prefix_dev || !a->lens_dev ||
                                !a->starts_dev))
        return HS_ERR_INVALID_ARG;
    if (!aligned(a->q_dev, 2) || !aligned(a->out_dev, 2) || !aligned(a->join_out_dev, 2) ||
        !aligned(a->rows_dev, 16) || !aligned(a->scales_dev, 4) || !aligned(a->prefix_dev, 4) ||
        !aligned(a->lens_dev, 4) || !aligned(a->starts_dev, 4) || !aligned(a->lse_dev, 4) ||
        !aligned(a->join_lse_dev, 4) || !aligned(a->workspace_dev, 16))
        return HS_ERR_INVALID_ARG;
    const size_t need = prefix_workspace(*fmt);
    if (need > 0 && (!a->workspace_dev || a->workspace_bytes < need)) return HS_ERR_INVALID_ARG;
    return result(launch_prefix(*fmt, *a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
