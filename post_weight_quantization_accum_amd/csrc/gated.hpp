// Gated products with e2m1 weights and the gradients of products: activation
// functions, arguments and launchers (checked in mx_api.hip).
#pragma once

#include <type_traits>

#include "mx.hpp"

namespace gptq {

// exp(v), 1 / (1 + exp(-v)) (0 and 1 far out).  QUICK: for results of 16 bits, by
// the hardware's power of two and reciprocal: off by some |v| + 3 roundings of
// float32 (the product with log2 e is one), and by nothing that 16 bits see.
template <bool QUICK>
__device__ __forceinline__ float exp_of(float v) { return QUICK ? __builtin_amdgcn_exp2f(v * 1.44269504f) : expf(v); }
template <bool QUICK>
__device__ __forceinline__ float sigmoid(float v) {
    return QUICK ? __builtin_amdgcn_rcpf(1.0f + exp_of<true>(-v)) : 1.0f / (1.0f + expf(-v));
}

constexpr float GELU_C = 0.7978845608028654f, GELU_A = 0.044715f;      // sqrt(2 / pi)

template <bool QUICK>
__device__ __forceinline__ float activate(gptq_activation act, float v) {
    switch (act) {
        case GPTQ_ACT_SILU: return v * sigmoid<QUICK>(v);
        case GPTQ_ACT_GELU: return v * (0.5f * erfcf(v * -0.70710678118654752f));      // no difference of near numbers below 0
        case GPTQ_ACT_GELU_TANH: return v * sigmoid<QUICK>(2.0f * GELU_C * (v + GELU_A * v * v * v));
        default: return v < 0.0f ? 0.0f : v;                                           // a NaN stays one
    }
}

// y = act(g) u of eight values.  The function is chosen once, not for each value:
// code that is unrolled with all four takes longer to come in than to run.
template <bool QUICK>
__device__ __forceinline__ void gate8(gptq_activation act, const float (&g)[8], const float (&u)[8], float (&y)[8]) {
    const auto all = [&](auto a) {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = activate<QUICK>(decltype(a)::value, g[i]) * u[i];
    };
    switch (act) {
        case GPTQ_ACT_SILU: all(std::integral_constant<gptq_activation, GPTQ_ACT_SILU>{}); break;
        case GPTQ_ACT_GELU: all(std::integral_constant<gptq_activation, GPTQ_ACT_GELU>{}); break;
        case GPTQ_ACT_GELU_TANH: all(std::integral_constant<gptq_activation, GPTQ_ACT_GELU_TANH>{}); break;
        default: all(std::integral_constant<gptq_activation, GPTQ_ACT_RELU>{}); break;
    }
}

// v where the slopes' second terms matter: beyond, they are 0, and neither an
// infinity nor an overflow meets that 0.
__device__ __forceinline__ float within(float v) { return __builtin_amdgcn_fmed3f(v, -200.0f, 200.0f); }

// The function's value and slope.
template <bool QUICK>
__device__ __forceinline__ void activate_with_slope(gptq_activation act, float v, float& value, float& slope) {
    switch (act) {
        case GPTQ_ACT_SILU: {
            const float s = sigmoid<QUICK>(v);
            value = v * s;
            slope = s * (1.0f + within(v) * (1.0f - s));
            break;
        }
        case GPTQ_ACT_GELU: {
            const float s = 0.5f * erfcf(v * -0.70710678118654752f);
            value = v * s;
            slope = s + within(v) * (exp_of<QUICK>(-0.5f * within(v) * within(v)) * 0.3989422804014327f);      // 1 / sqrt(2 pi)
            break;
        }
        case GPTQ_ACT_GELU_TANH: {
            const float s = sigmoid<QUICK>(2.0f * GELU_C * (v + GELU_A * v * v * v));
            value = v * s;
            slope = s + within(v) * s * (1.0f - s) * (2.0f * GELU_C * (1.0f + 3.0f * GELU_A * within(v) * within(v)));
            break;
        }
        default:
            value = v < 0.0f ? 0.0f : v;
            slope = v > 0.0f ? 1.0f : v == v ? 0.0f : v;
            break;
    }
}

// Four neighbouring outputs, n of which exist.
__device__ __forceinline__ void put4(void* Y, gptq_dtype dt, int64_t at, int n, const float (&v)[4]) {
    const bool whole = n >= 4;
    if (dt == GPTQ_F32) {
        float* y = (float*)Y + at;
        if (whole) {
            *(f32x4_any_t*)y = f32x4_any_t{v[0], v[1], v[2], v[3]};
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < n) y[i] = v[i];
        }
        return;
    }
    uint16_t* y = (uint16_t*)Y + at;
    u32x2_t w;
    w.x = dt == GPTQ_BF16 ? H16<true>::pack(v[0], v[1]) : H16<false>::pack(v[0], v[1]);
    w.y = dt == GPTQ_BF16 ? H16<true>::pack(v[2], v[3]) : H16<false>::pack(v[2], v[3]);
    if (whole) {
        *(u32x2_any_t*)y = w;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < n) y[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
    }
}
// What a gated product has beside the product of X and the gate.
struct GatedArgs {
    const uint8_t *up_codes, *up_scales;
    gptq_activation act;
    void* Y;
    gptq_dtype y_dt;
    int64_t ld_y;
    void *G, *U;           // may be null
    int64_t ld_gu;
};
gptq_status mx_gated_launch(const void* X, gptq_dtype dt, int64_t n_tok, int64_t d_in, int64_t ld_x, const uint8_t* codes,
                            const uint8_t* scales, int64_t d_ff, const GatedArgs& g, hipStream_t s);
gptq_status mx_gated_quantized_launch(const uint8_t* xc, const uint8_t* xs, gptq_mx_format xf, int64_t n_tok, int64_t d_in,
                                      const uint8_t* codes, const uint8_t* scales, int64_t d_ff, const GatedArgs& g,
                                      hipStream_t s);

int mx_gated_kernel(gptq_dtype dt, gptq_mx_format xf, int64_t n_tok, int64_t d_in, int64_t d_ff, bool aligned);

// The gradient of products for their activations: one matrix of codes, or the
// sum over two.
struct BackArgs {
    gptq_dtype dt;                       // of the gradients
    int64_t n_tok, rows, d_in;           // rows: of each matrix
    const uint8_t *codes[2], *scales[2];
    int matrices;
    const int32_t* exps;                 // null, or for each token the exponent of the power of two that its gradients lack
    void* dX;
    gptq_dtype dx_dt;
    int64_t ld_dx;
};
size_t mx_backward_ws(gptq_dtype dt, int64_t n_tok, int64_t d_in, int64_t rows);
void mx_backward_plan(gptq_dtype dt, int matrices, int64_t n_tok, int64_t d_in, int64_t rows, int64_t* plan);
gptq_status mx_backward_launch(const BackArgs& a, const void* D, int64_t ld, void* ws, hipStream_t s);

struct GatedBackArgs {
    const void *dY, *G, *U;
    gptq_dtype dt;
    int64_t n_tok, d_ff, ld_dy, ld_gu;
    const uint8_t *codes[2], *scales[2];
    int64_t d_in;
    gptq_activation act;
    void* dX;
    gptq_dtype dx_dt;
    int64_t ld_dx;
    void *dG, *dU;                       // may be null
    int64_t ld_dgu;
};
size_t mx_gated_backward_ws(gptq_dtype dt, int64_t n_tok, int64_t d_in, int64_t d_ff);
gptq_status mx_gated_backward_launch(const GatedBackArgs& a, void* ws, hipStream_t s);

}  // namespace gptq
