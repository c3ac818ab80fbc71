// C entry points of the norms around a block: argument checks and dispatch.
// Contracts are in include/gptq.h.
#include "norm.hpp"

#include <cmath>

using namespace gptq;

namespace {

constexpr int64_t MAX_DIM = int64_t(1) << 20;

bool is_float(gptq_dtype dt) { return dt == GPTQ_F32 || dt == GPTQ_F16 || dt == GPTQ_BF16; }
bool in(int64_t v, int64_t lo, int64_t hi) { return v >= lo && v <= hi; }
// elements start on their own size
bool starts(const void* p, gptq_dtype dt) { return (uintptr_t)p % (dt == GPTQ_F32 ? 4 : 2) == 0; }
bool elems(const void* p, gptq_dtype dt) { return p && starts(p, dt); }

bool check_norm(const gptq_norm* c, int64_t n_tok, int64_t d) {
    if (!c || (c->kind != GPTQ_NORM_RMS && c->kind != GPTQ_NORM_LAYER)) return false;
    if (!in(n_tok, 0, MAX_DIM) || !in(d, 1, MAX_DIM)) return false;
    if (!(c->eps >= 0.0f) || !std::isfinite(c->eps) || !std::isfinite(c->residual_scale)) return false;
    if (!is_float(c->vec_dtype)) return false;
    for (const void* p : {c->weight, c->bias, c->post_weight, c->gate})
        if (!starts(p, c->vec_dtype)) return false;
    return c->ld_gate == 0 || (c->gate && c->ld_gate >= d);
}

NormArgs base(const gptq_norm* c, int64_t n_tok, int64_t d) {
    NormArgs a{};
    a.n_tok = n_tok;
    a.d = d;
    a.inv_d = 1.0 / (double)d;
    a.eps = c->eps;
    a.scale = c->residual_scale;
    a.layer = c->kind == GPTQ_NORM_LAYER;
    a.v_dt = c->vec_dtype;
    a.weight = c->weight;
    a.bias = c->bias;
    a.post = c->post_weight;
    a.gate = c->gate;
    a.ld_gate = c->ld_gate;
    return a;
}

}  // namespace

extern "C" {

gptq_status gptq_residual_norm(const gptq_norm* norm, int64_t n_tok, int64_t d, const void* X, gptq_dtype x_dtype,
                               int64_t ld_x, const void* B, gptq_dtype b_dtype, int64_t ld_b, void* H, gptq_dtype h_dtype,
                               int64_t ld_h, void* Y, gptq_dtype y_dtype, int64_t ld_y, hipStream_t stream) {
    if (!check_norm(norm, n_tok, d)) return GPTQ_ERR_INVALID_ARG;
    if (!is_float(x_dtype) || !is_float(h_dtype) || !is_float(y_dtype) || !is_float(b_dtype)) return GPTQ_ERR_INVALID_ARG;
    if (ld_x < d || (H && ld_h < d) || (Y && ld_y < d) || (B && ld_b < d)) return GPTQ_ERR_INVALID_ARG;
    if (n_tok == 0) return GPTQ_OK;
    if (!elems(X, x_dtype) || !starts(B, b_dtype) || !starts(H, h_dtype) || !starts(Y, y_dtype)) return GPTQ_ERR_INVALID_ARG;
    if (!B && (norm->post_weight || norm->gate)) return GPTQ_ERR_INVALID_ARG;
    // in place, a lane writes where it has read
    if (H == X && (h_dtype != x_dtype || (n_tok > 1 && ld_h != ld_x))) return GPTQ_ERR_INVALID_ARG;
    if (!H && !Y) return GPTQ_OK;
    NormArgs a = base(norm, n_tok, d);
    a.X = X;
    a.B = B;
    a.H = H;
    a.Y = Y;
    a.x_dt = x_dtype;
    a.b_dt = b_dtype;
    a.h_dt = h_dtype;
    a.y_dt = y_dtype;
    a.ld_x = ld_x;
    a.ld_b = ld_b;
    a.ld_h = ld_h;
    a.ld_y = ld_y;
    return norm_launch(a, stream);
}

size_t gptq_residual_norm_backward_workspace(int64_t n_tok, int64_t d) {
    return in(n_tok, 1, MAX_DIM) && in(d, 1, MAX_DIM) ? norm_grad_ws(n_tok, d) : 0;
}

gptq_status gptq_residual_norm_backward(const gptq_norm* norm, int64_t n_tok, int64_t d, const void* dY, gptq_dtype dy_dtype,
                                        int64_t ld_dy, const void* H, gptq_dtype h_dtype, int64_t ld_h, const void* B,
                                        gptq_dtype b_dtype, int64_t ld_b, const void* dH, int64_t ld_dh, void* dX,
                                        int64_t ld_dx, void* dB, int64_t ld_db, float* d_weight, float* d_bias,
                                        float* d_post_weight, void* d_gate, int64_t ld_dgate, void* workspace,
                                        size_t ws_bytes, hipStream_t stream) {
    if (!check_norm(norm, n_tok, d)) return GPTQ_ERR_INVALID_ARG;
    if (!is_float(dy_dtype) || !is_float(h_dtype) || !is_float(b_dtype)) return GPTQ_ERR_INVALID_ARG;
    if (ld_dy < d || ld_h < d || (B && ld_b < d) || (dH && ld_dh < d) || (dX && ld_dx < d) || (dB && ld_db < d))
        return GPTQ_ERR_INVALID_ARG;
    const bool rows = norm->gate && norm->ld_gate > 0;
    if (d_gate && (!norm->gate || (rows && ld_dgate < d) || !starts(d_gate, rows ? norm->vec_dtype : GPTQ_F32)))
        return GPTQ_ERR_INVALID_ARG;
    if (d_post_weight && !norm->post_weight) return GPTQ_ERR_INVALID_ARG;
    for (const float* p : {d_weight, d_bias, d_post_weight})
        if (!starts(p, GPTQ_F32)) return GPTQ_ERR_INVALID_ARG;
    const bool needs = norm->post_weight || norm->gate;
    float* gate_sum = rows ? nullptr : (float*)d_gate;
    NormGradArgs a{};
    a.f = base(norm, n_tok, d);
    if (n_tok > 0) {
        if (!elems(dY, dy_dtype) || !elems(H, h_dtype) || !starts(B, b_dtype) || !starts(dH, h_dtype) || !starts(dX, h_dtype) ||
            !starts(dB, b_dtype) || (needs && !B))
            return GPTQ_ERR_INVALID_ARG;
        const bool sums = d_weight || d_bias || d_post_weight || gate_sum;
        if (sums && ((uintptr_t)workspace % 16 != 0 || !workspace || ws_bytes < norm_grad_ws(n_tok, d))) return GPTQ_ERR_WORKSPACE;
    }
    a.f.B = needs ? B : nullptr;
    a.f.b_dt = b_dtype;
    a.f.ld_b = ld_b;
    a.has_b = needs;
    a.dY = dY;
    a.H = H;
    a.dH = dH;
    a.dX = dX;
    a.dB = dB;
    a.d_gate_rows = rows ? d_gate : nullptr;
    a.dy_dt = dy_dtype;
    a.h_dt = h_dtype;
    a.ld_dy = ld_dy;
    a.ld_h = ld_h;
    a.ld_dh = ld_dh;
    a.ld_dx = ld_dx;
    a.ld_db = ld_db;
    a.ld_dgate = ld_dgate;
    a.parts = (float*)workspace;
    return norm_grad_launch(a, d_weight, d_bias, d_post_weight, gate_sum, stream);
}

}  // extern "C"
