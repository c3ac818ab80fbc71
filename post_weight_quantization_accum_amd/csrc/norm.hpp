// Norms around a block and their gradient: arguments and launchers (checked in
// norm_api.hip).
#pragma once

#include "mx.hpp"

namespace gptq {

struct NormArgs {
    int64_t n_tok, d;
    double inv_d;
    float eps, scale;
    bool layer;
    gptq_dtype v_dt;                                     // of the vectors
    const void *weight, *bias, *post, *gate;             // may be null
    int64_t ld_gate;
    const void* X;
    const void* B;                                       // may be null
    void* H;                                             // may be null
    void* Y;                                             // may be null
    gptq_dtype x_dt, b_dt, h_dt, y_dt;
    int64_t ld_x, ld_b, ld_h, ld_y;
};

struct NormGradArgs {
    NormArgs f;                                          // of it the sizes, vectors and B
    bool has_b;                                          // B's values are needed
    const void *dY, *H, *dH;                             // dH may be null
    void *dX, *dB, *d_gate_rows;                         // may be null
    gptq_dtype dy_dt, h_dt;                              // dH and dX are of h_dt, dB of B's type
    int64_t ld_dy, ld_h, ld_dh, ld_dx, ld_db, ld_dgate;
    float* parts;                                        // [part][slot][ld_part]
    int n_slots, slot[4];                                // of weight, bias, post, gate; -1: not asked for
    int64_t ld_part;
};

gptq_status norm_launch(const NormArgs& a, hipStream_t s);
size_t norm_grad_ws(int64_t n_tok, int64_t d);
gptq_status norm_grad_launch(NormGradArgs a, float* d_weight, float* d_bias, float* d_post, float* d_gate, hipStream_t s);

}  // namespace gptq
