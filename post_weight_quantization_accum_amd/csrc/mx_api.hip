// C entry points of the microscaled operators: argument checks and dispatch.
// Contracts are in include/gptq.h.
#include "mx.hpp"

using namespace gptq;

namespace {

constexpr int64_t MAX_DIM = int64_t(1) << 20;

bool is_float(gptq_dtype dt) { return dt == GPTQ_F32 || dt == GPTQ_F16 || dt == GPTQ_BF16; }
bool is_half(gptq_dtype dt) { return dt == GPTQ_F16 || dt == GPTQ_BF16; }
bool is_mx(gptq_mx_format f) { return f == GPTQ_MX_FP8 || f == GPTQ_MX_FP4; }
bool in(int64_t v, int64_t lo, int64_t hi) { return v >= lo && v <= hi; }
bool on(const void* p, size_t n) { return p && (uintptr_t)p % n == 0; }
// elements start on their own size
bool elems(const void* p, gptq_dtype dt) { return on(p, dt == GPTQ_F32 ? 4 : 2); }

gptq_status check_cache(const gptq_kv_cache* c) {
    if (!c) return GPTQ_ERR_INVALID_ARG;
    if (c->format != GPTQ_MX_NONE && !is_mx(c->format)) return GPTQ_ERR_INVALID_ARG;
    if (c->format == GPTQ_MX_NONE && !is_half(c->dtype)) return GPTQ_ERR_INVALID_ARG;
    if (c->n_pages < 1 || c->page_size < 1 || c->n_kv_heads < 1 || c->head_dim < 1) return GPTQ_ERR_INVALID_ARG;
    if (c->n_pages > INT32_MAX || (int64_t)c->page_size * c->n_kv_heads > INT32_MAX / c->n_pages)
        return GPTQ_ERR_INVALID_ARG;
    if (c->head_dim % 32 != 0 || c->head_dim > 128) return GPTQ_ERR_UNSUPPORTED;
    if ((int64_t)c->n_kv_heads * c->head_dim > MAX_DIM) return GPTQ_ERR_INVALID_ARG;
    if (!on(c->k, 16) || !on(c->v, 16)) return GPTQ_ERR_INVALID_ARG;
    if (c->format != GPTQ_MX_NONE && (!c->k_scales || !c->v_scales)) return GPTQ_ERR_INVALID_ARG;
    return GPTQ_OK;
}

bool check_shape(const gptq_kv_cache* c, int64_t n_tok, int64_t n_heads, int64_t n_seq, int64_t max_pages,
                 int64_t max_q, int64_t window) {
    return in(n_tok, 0, MAX_DIM) && in(n_heads, 1, MAX_DIM) && n_heads % c->n_kv_heads == 0 &&
           n_heads * c->head_dim <= MAX_DIM && in(n_seq, 0, MAX_DIM) && in(max_pages, 0, INT32_MAX) &&
           in(max_q, 0, MAX_DIM) && in(window, 0, int64_t(1) << 30);
}

}  // namespace

extern "C" {

int64_t gptq_mx_codes_per_row(int64_t n_cols, gptq_mx_format format) {
    return n_cols < 0 || !is_mx(format) ? -1 : mx_code_bytes(n_cols, format);
}

int64_t gptq_mx_scales_per_row(int64_t n_cols) { return n_cols < 0 ? -1 : mx_scale_bytes(n_cols); }

gptq_status gptq_mx_quantize(const void* X, gptq_dtype x_dtype, int64_t n_rows, int64_t n_cols, int64_t ld_x,
                             gptq_mx_format format, uint8_t* codes, uint8_t* scales, hipStream_t stream) {
    if (!is_float(x_dtype) || !is_mx(format)) return GPTQ_ERR_INVALID_ARG;
    if (!in(n_rows, 0, MAX_DIM) || !in(n_cols, 1, MAX_DIM) || ld_x < n_cols) return GPTQ_ERR_INVALID_ARG;
    if (n_rows == 0) return GPTQ_OK;
    if (!elems(X, x_dtype) || !on(codes, 16) || !on(scales, 4)) return GPTQ_ERR_INVALID_ARG;
    return mx_quantize_launch(X, x_dtype, n_rows, n_cols, ld_x, format, codes, scales, stream);
}

gptq_status gptq_mx_dequantize(const uint8_t* codes, const uint8_t* scales, gptq_mx_format format, int64_t n_rows,
                               int64_t n_cols, void* Y, gptq_dtype y_dtype, int64_t ld_y, hipStream_t stream) {
    if (!is_float(y_dtype) || !is_mx(format)) return GPTQ_ERR_INVALID_ARG;
    if (!in(n_rows, 0, MAX_DIM) || !in(n_cols, 1, MAX_DIM) || ld_y < n_cols) return GPTQ_ERR_INVALID_ARG;
    if (n_rows == 0) return GPTQ_OK;
    if (!elems(Y, y_dtype) || !on(codes, 16) || !on(scales, 4)) return GPTQ_ERR_INVALID_ARG;
    return mx_dequantize_launch(codes, scales, format, n_rows, n_cols, Y, y_dtype, ld_y, stream);
}

gptq_status gptq_mx_matmul(const void* X, gptq_dtype x_dtype, int64_t n_tok, int64_t d_in, int64_t ld_x,
                           const uint8_t* codes, const uint8_t* scales, int64_t d_out, float* Y, int64_t ld_y,
                           hipStream_t stream) {
    if (!is_float(x_dtype)) return GPTQ_ERR_INVALID_ARG;
    if (!in(n_tok, 0, MAX_DIM) || !in(d_in, 1, MAX_DIM) || !in(d_out, 0, MAX_DIM)) return GPTQ_ERR_INVALID_ARG;
    if (ld_x < d_in || ld_y < d_out) return GPTQ_ERR_INVALID_ARG;
    if (n_tok == 0 || d_out == 0) return GPTQ_OK;
    if (!elems(X, x_dtype) || !on(codes, 16) || !on(scales, 4) || !on(Y, 4)) return GPTQ_ERR_INVALID_ARG;
    return mx_matmul_launch(X, x_dtype, n_tok, d_in, ld_x, codes, scales, d_out, Y, ld_y, stream);
}

gptq_status gptq_mx_matmul_quantized(const uint8_t* x_codes, const uint8_t* x_scales, gptq_mx_format x_format,
                                     int64_t n_tok, int64_t d_in, const uint8_t* codes, const uint8_t* scales,
                                     int64_t d_out, float* Y, int64_t ld_y, hipStream_t stream) {
    if (!is_mx(x_format)) return GPTQ_ERR_INVALID_ARG;
    if (!in(n_tok, 0, MAX_DIM) || !in(d_in, 1, MAX_DIM) || !in(d_out, 0, MAX_DIM)) return GPTQ_ERR_INVALID_ARG;
    if (ld_y < d_out) return GPTQ_ERR_INVALID_ARG;
    if (n_tok == 0 || d_out == 0) return GPTQ_OK;
    if (!on(x_codes, 16) || !on(x_scales, 4) || !on(codes, 16) || !on(scales, 4) || !on(Y, 4))
        return GPTQ_ERR_INVALID_ARG;
    return mx_matmul_quantized_launch(x_codes, x_scales, x_format, n_tok, d_in, codes, scales, d_out, Y, ld_y, stream);
}

int32_t gptq_mx_matmul_kernel(gptq_dtype x_dtype, gptq_mx_format x_format, int64_t n_tok, int64_t d_in, int64_t d_out,
                              int32_t aligned) {
    if (x_format == GPTQ_MX_NONE ? !is_float(x_dtype) : !is_mx(x_format)) return -1;
    if (!in(n_tok, 1, MAX_DIM) || !in(d_in, 1, MAX_DIM) || !in(d_out, 1, MAX_DIM)) return -1;
    return mx_matmul_kernel(x_dtype, x_format, n_tok, d_in, d_out, aligned != 0);
}

gptq_status gptq_cache_write(const gptq_kv_cache* cache, const void* K, const void* V, gptq_dtype x_dtype,
                             int64_t n_tok, int64_t ld_k, int64_t ld_v, const int64_t* slots, hipStream_t stream) {
    const gptq_status st = check_cache(cache);
    if (st != GPTQ_OK) return st;
    if (!is_float(x_dtype) || (cache->format == GPTQ_MX_NONE && x_dtype != cache->dtype)) return GPTQ_ERR_INVALID_ARG;
    const int64_t width = (int64_t)cache->n_kv_heads * cache->head_dim;
    if (!in(n_tok, 0, MAX_DIM) || ld_k < width || ld_v < width) return GPTQ_ERR_INVALID_ARG;
    if (n_tok == 0) return GPTQ_OK;
    if (!elems(K, x_dtype) || !elems(V, x_dtype) || !on(slots, 8)) return GPTQ_ERR_INVALID_ARG;
    return cache_write_launch(*cache, K, V, x_dtype, n_tok, ld_k, ld_v, slots, stream);
}

gptq_status gptq_cache_read(const gptq_kv_cache* cache, const int32_t* table, int64_t max_pages, int64_t n_seq,
                            const int32_t* row_start, int64_t n_rows, void* K, void* V, gptq_dtype y_dtype,
                            int64_t ld_k, int64_t ld_v, hipStream_t stream) {
    const gptq_status st = check_cache(cache);
    if (st != GPTQ_OK) return st;
    if (!is_float(y_dtype)) return GPTQ_ERR_INVALID_ARG;
    const int64_t width = (int64_t)cache->n_kv_heads * cache->head_dim;
    if (!in(n_rows, 0, INT32_MAX) || !in(n_seq, 0, MAX_DIM) || !in(max_pages, 0, INT32_MAX)) return GPTQ_ERR_INVALID_ARG;
    if (ld_k < width || ld_v < width) return GPTQ_ERR_INVALID_ARG;
    if (n_rows == 0 || n_seq == 0) return GPTQ_OK;
    if (!elems(K, y_dtype) || !elems(V, y_dtype) || !on(row_start, 4) || (max_pages && !on(table, 4)))
        return GPTQ_ERR_INVALID_ARG;
    return cache_read_launch(*cache, table, max_pages, n_seq, row_start, n_rows, K, V, y_dtype, ld_k, ld_v, stream);
}

size_t gptq_cache_attention_workspace(const gptq_kv_cache* cache, int64_t n_tok, int64_t n_heads, int64_t n_seq,
                                      int64_t max_pages, int64_t max_q, int64_t window) {
    if (check_cache(cache) != GPTQ_OK) return 0;
    if (!check_shape(cache, n_tok, n_heads, n_seq, max_pages, max_q, window)) return 0;
    if (n_tok == 0 || n_seq == 0) return 0;
    return cache_attention_ws(*cache, AttentionShape{n_tok, n_heads, n_seq, max_pages, max_q, window});
}

gptq_status gptq_cache_attention_plan(const gptq_kv_cache* cache, int64_t n_tok, int64_t n_heads, int64_t n_seq,
                                      int64_t max_pages, int64_t max_q, int64_t window, int64_t* plan) {
    const gptq_status st = check_cache(cache);
    if (st != GPTQ_OK) return st;
    if (!plan || !check_shape(cache, n_tok, n_heads, n_seq, max_pages, max_q, window)) return GPTQ_ERR_INVALID_ARG;
    plan[0] = plan[1] = plan[2] = 0;
    if (n_tok == 0 || n_seq == 0) return GPTQ_OK;
    return cache_attention_plan(*cache, AttentionShape{n_tok, n_heads, n_seq, max_pages, max_q, window}, plan);
}

gptq_status gptq_cache_attention(const gptq_kv_cache* cache, const void* Q, gptq_dtype q_dtype, int64_t n_tok,
                                 int64_t n_heads, int64_t ld_q, const int32_t* q_start, const int32_t* kv_len,
                                 const int32_t* table, int64_t max_pages, int64_t n_seq, int64_t max_q,
                                 float scale, int64_t window, void* O, int64_t ld_o, void* workspace,
                                 size_t ws_bytes, hipStream_t stream) {
    const gptq_status st = check_cache(cache);
    if (st != GPTQ_OK) return st;
    if (!is_half(q_dtype) || (cache->format == GPTQ_MX_NONE && q_dtype != cache->dtype)) return GPTQ_ERR_INVALID_ARG;
    if (!check_shape(cache, n_tok, n_heads, n_seq, max_pages, max_q, window)) return GPTQ_ERR_INVALID_ARG;
    if (ld_q < n_heads * cache->head_dim || ld_o < n_heads * cache->head_dim) return GPTQ_ERR_INVALID_ARG;
    if (!(scale >= 0x1p-100f && scale <= 0x1p100f)) return GPTQ_ERR_INVALID_ARG;   // its reciprocal is used, too
    if (n_tok == 0 || n_seq == 0) return GPTQ_OK;
    if (!elems(Q, q_dtype) || !elems(O, q_dtype) || !on(q_start, 4) || !on(kv_len, 4) || (max_pages && !on(table, 4)))
        return GPTQ_ERR_INVALID_ARG;
    const AttentionShape a{n_tok, n_heads, n_seq, max_pages, max_q, window};
    const size_t need = cache_attention_ws(*cache, a);
    if (need && (!on(workspace, 16) || ws_bytes < need)) return GPTQ_ERR_WORKSPACE;
    return cache_attention_launch(*cache, a, Q, q_dtype, ld_q, q_start, kv_len, table, scale, O, ld_o, workspace,
                                  stream);
}

}  // extern "C"
