// Products with e2m1 weights: Y = X W^T (include/gptq.h, gptq_mx_matmul and
// gptq_mx_matmul_quantized).
#include "mx.hpp"

namespace gptq {
namespace {

// Kinds of activations that enter as bfloat16 parts.
enum Act : int { ACT_F32 = GPTQ_F32, ACT_F16 = GPTQ_F16, ACT_BF16 = GPTQ_BF16, ACT_FP8 };

struct MatArgs {
    const void* X;         // values, or e4m3 codes
    const uint8_t* XS;     // scale bytes of the codes
    int64_t n_tok, d_in, ld_x;
    bool aligned;          // X rows start on 16 bytes
    const uint8_t* W;      // codes
    const uint8_t* S;      // scale bytes
    int64_t w_row, s_row;  // bytes per row
    int steps;             // padded 128-column steps
    int64_t d_out, ld_y;
    float* Y;
};

// ---------------------------------------------------------------------------
// Activations as bfloat16 parts.  A float32 is the sum of three bfloat16 cut
// off its top (8 + 8 + 8 of its 24 bits), a float16 of two: no rounding, and
// no overflow.  The parts below an infinity or NaN are 0.  A microscaled e4m3
// value is a bfloat16 as it is.  (v_mfma_scale_f32_32x32x64_f8f6f4 would take
// its codes directly, at twice the rate, but with an e4m3 operand it cuts
// products off some 16 bits below the largest one of an instruction: an
// error of 1e-5 of sum |x w| and more, measured, where these sums keep 1e-7.)
// ---------------------------------------------------------------------------
template <Act DT>
constexpr int parts_of() { return DT == ACT_F16 ? 2 : DT == ACT_F32 ? 3 : 1; }

// Eight activations from (t, k): n of them exist.
template <Act DT>
__device__ __forceinline__ void load_parts(const MatArgs& a, int64_t t, int64_t k, u32x4_t (&p)[parts_of<DT>()]) {
    if constexpr (DT == ACT_FP8) {
        const u32x2_t w = *(const u32x2_t*)((const uint8_t*)a.X + t * a.ld_x + k);
        p[0] = fp8x8<true>(w.x, w.y, mx_scale(a.XS[t * a.s_row + (k >> 5)]));
        return;
    }
    const int n = (int)max((int64_t)0, min((int64_t)8, a.d_in - k));
    const bool vec = a.aligned && n == 8;
    if constexpr (DT == ACT_BF16) {
        const uint16_t* q = (const uint16_t*)a.X + t * a.ld_x + k;
        if (vec) {
            p[0] = *(const u32x4_t*)q;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t lo = 2 * i < n ? q[2 * i] : 0, hi = 2 * i + 1 < n ? q[2 * i + 1] : 0;
                p[0][i] = lo | hi << 16;
            }
        }
    } else if constexpr (DT != ACT_FP8) {
        float v[8];
        load8_f32(a.X, (gptq_dtype)DT, t * a.ld_x + k, n, vec, v);
#pragma unroll
        for (int j = 0; j < parts_of<DT>(); ++j) {
            uint32_t w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t b = __float_as_uint(v[i]);
                const bool fin = (b & 0x7F800000u) != 0x7F800000u;
                // a NaN whose top bits are an infinity's keeps a quiet bit
                w[i] = (b & 0xFFFF0000u) | ((b & 0x7FFFFFFFu) > 0x7F800000u ? 0x00400000u : 0u);
                v[i] = fin ? v[i] - __uint_as_float(b & 0xFFFF0000u) : 0.0f;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) p[j][i] = w[2 * i] >> 16 | (w[2 * i + 1] & 0xFFFF0000u);
        }
    }
}

// ---------------------------------------------------------------------------
// Few tokens: 16 weight rows per workgroup, its eight waves share the
// 128-column steps, and their sums meet in LDS.  v_mfma_f32_16x16x32_bf16
// with a lane's four k-groups of eight chosen as one block of 32 columns:
// lane l holds row l % 16, block l / 16 of the step (16 bytes of codes, one
// scale), and activations of token l % 16 in the same columns.
// ---------------------------------------------------------------------------
constexpr int FEW_WAVES = 8;

template <Act DT, int TT>
__global__ __launch_bounds__(64 * FEW_WAVES) void mx_few_kernel(MatArgs a) {
    constexpr int NP = parts_of<DT>();
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int i16 = lane & 15, g = lane >> 4;
    const int64_t r0 = (int64_t)blockIdx.x * 16, t0 = (int64_t)blockIdx.y * (16 * TT);
    const int64_t row = min(r0 + i16, a.d_out - 1);
    const uint8_t* wp = a.W + row * a.w_row + 16 * g;
    const uint8_t* sp = a.S + row * a.s_row + g;
    f32x4_t acc[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    constexpr int PF = 4;
    u32x4_t w[PF];
    uint32_t s[PF];
    const int last = a.steps - 1;
#pragma unroll
    for (int i = 0; i < PF; ++i) {
        const int st = min(wave + FEW_WAVES * i, last);
        w[i] = *(const u32x4_t*)(wp + 64 * (int64_t)st);
        s[i] = sp[4 * (int64_t)st];
    }
    for (int s0 = wave; s0 < a.steps; s0 += FEW_WAVES * PF) {
#pragma unroll
        for (int i = 0; i < PF; ++i) {
            const int st = s0 + FEW_WAVES * i;
            if (st < a.steps) {
                const int64_t k = 128 * (int64_t)st + 32 * g;
                const float sc = mx_scale(s[i]);
                u32x4_t aw[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) aw[c] = fp4x8<true>(w[i][c], sc);
#pragma unroll
                for (int t = 0; t < TT; ++t) {
                    const int64_t tok = t0 + 16 * t + i16;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        u32x4_t p[NP];
                        if (tok < a.n_tok) {
                            load_parts<DT>(a, tok, k + 8 * c, p);
                        } else {
#pragma unroll
                            for (int j = 0; j < NP; ++j) p[j] = u32x4_t{0u, 0u, 0u, 0u};
                        }
#pragma unroll
                        for (int j = 0; j < NP; ++j) acc[t] = H16<true>::mfma16(aw[c], p[j], acc[t]);
                    }
                }
            }
            const int nx = min(st + FEW_WAVES * PF, last);
            w[i] = *(const u32x4_t*)(wp + 64 * (int64_t)nx);
            s[i] = sp[4 * (int64_t)nx];
        }
    }
    __shared__ f32x4_t part[FEW_WAVES][TT][64];
#pragma unroll
    for (int t = 0; t < TT; ++t) part[wave][t][lane] = acc[t];
    __syncthreads();
    for (int e = threadIdx.x; e < TT * 64; e += 64 * FEW_WAVES) {
        const int t = e >> 6, l = e & 63;
        f32x4_t v = part[0][t][l];
#pragma unroll
        for (int q = 1; q < FEW_WAVES; ++q) v += part[q][t][l];
        const int64_t tok = t0 + 16 * t + (l & 15), r = r0 + 4 * (l >> 4);
        if (tok < a.n_tok) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (r + j < a.d_out) a.Y[tok * a.ld_y + r + j] = v[j];
        }
    }
}

// ---------------------------------------------------------------------------
// Many tokens: 128 weight rows x 128 tokens per workgroup of four waves, each
// 64 x 64 of v_mfma_f32_32x32x16_bf16.  Activations go through LDS (split
// into their parts on the way), weights straight from memory into the lanes
// that multiply them: lane l holds row l % 32 and, of every 64 columns, block
// l / 32.
// ---------------------------------------------------------------------------
constexpr int MT = 128, MK = 64, X_ROW = MK * 2 + 16;

template <Act DT>
__global__ __launch_bounds__(256) void mx_many_kernel(MatArgs a) {
    constexpr int NP = parts_of<DT>();
    __shared__ __attribute__((aligned(16))) char xs[NP * MT * X_ROW];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int i32 = lane & 31, h = lane >> 5;
    const int64_t r0 = (int64_t)blockIdx.x * MT + 64 * (wave >> 1), t0 = (int64_t)blockIdx.y * MT;
    const int tw = 64 * (wave & 1);
    const uint8_t* wp[2];
    const uint8_t* sp[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int64_t row = min(r0 + 32 * i + i32, a.d_out - 1);
        wp[i] = a.W + row * a.w_row + 16 * h;
        sp[i] = a.S + row * a.s_row + h;
    }
    f16_t acc[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
    for (int st = 0; st < 2 * a.steps; ++st) {
        __syncthreads();
        // 128 tokens x 8 groups of eight columns, four per thread
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int e = threadIdx.x + 256 * q, t = e >> 3, c = e & 7;
            u32x4_t p[NP];
            if (t0 + t < a.n_tok) {
                load_parts<DT>(a, t0 + t, (int64_t)MK * st + 8 * c, p);
            } else {
#pragma unroll
                for (int j = 0; j < NP; ++j) p[j] = u32x4_t{0u, 0u, 0u, 0u};
            }
#pragma unroll
            for (int j = 0; j < NP; ++j) *(u32x4_t*)(xs + (j * MT + t) * X_ROW + 16 * c) = p[j];
        }
        u32x4_t w[2];
        float sc[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            w[i] = *(const u32x4_t*)(wp[i] + 32 * (int64_t)st);
            sc[i] = mx_scale(sp[i][2 * (int64_t)st]);
        }
        __syncthreads();
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            u32x4_t aw[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) aw[i] = fp4x8<true>(w[i][c], sc[i]);
#pragma unroll
            for (int p = 0; p < NP; ++p)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const u32x4_t b = *(const u32x4_t*)(xs + (p * MT + tw + 32 * j + i32) * X_ROW + 64 * h + 16 * c);
#pragma unroll
                    for (int i = 0; i < 2; ++i) acc[i][j] = H16<true>::mfma32(aw[i], b, acc[i][j]);
                }
        }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int64_t t = t0 + tw + 32 * j + i32;
        if (t >= a.n_tok) continue;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int64_t r = r0 + 32 * i + 8 * (e >> 2) + 4 * h + (e & 3);
                if (r < a.d_out) a.Y[t * a.ld_y + r] = acc[i][j][e];
            }
    }
}

// ---------------------------------------------------------------------------
// Both operands e2m1: v_mfma_scale_f32_32x32x64_f8f6f4.  Lane l holds row
// (token) l % 32 and block l / 32 of the 64 columns, 16 bytes, with that
// block's scale.  (Checked on the GPU against float64.)
// ---------------------------------------------------------------------------
struct MxArgs {
    const uint8_t* X;
    const uint8_t* XS;
    MatArgs m;             // X, XS, ld_x, aligned unused
};

__global__ __launch_bounds__(256) void mx_mx_kernel(MxArgs a) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int i32 = lane & 31, h = lane >> 5;
    const int64_t r0 = (int64_t)blockIdx.x * 128 + 64 * (wave >> 1), t0 = (int64_t)blockIdx.y * 128 + 64 * (wave & 1);
    const uint8_t *wp[2], *sp[2], *xp[2], *xsp[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int64_t row = min(r0 + 32 * i + i32, a.m.d_out - 1), tok = min(t0 + 32 * i + i32, a.m.n_tok - 1);
        wp[i] = a.m.W + row * a.m.w_row + 16 * h;
        sp[i] = a.m.S + row * a.m.s_row;
        xp[i] = a.X + tok * a.m.w_row + 16 * h;
        xsp[i] = a.XS + tok * a.m.s_row;
    }
    f16_t acc[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
    for (int st = 0; st < a.m.steps; ++st) {
        int ws[2], xs[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            ws[i] = (int)(*(const uint32_t*)(sp[i] + 4 * (int64_t)st) >> (8 * h));
            xs[i] = (int)(*(const uint32_t*)(xsp[i] + 4 * (int64_t)st) >> (8 * h));
        }
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            i32x8_t w[2], x[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const u32x4_t v = *(const u32x4_t*)(wp[i] + 64 * (int64_t)st + 32 * q);
                const u32x4_t u = *(const u32x4_t*)(xp[i] + 64 * (int64_t)st + 32 * q);
                w[i] = i32x8_t{(int)v.x, (int)v.y, (int)v.z, (int)v.w, 0, 0, 0, 0};
                x[i] = i32x8_t{(int)u.x, (int)u.y, (int)u.z, (int)u.w, 0, 0, 0, 0};
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    if (q == 0)
                        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w[i], x[j], acc[i][j], 4, 4, 0,
                                                                                   ws[i], 0, xs[j]);
                    else
                        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w[i], x[j], acc[i][j], 4, 4, 2,
                                                                                   ws[i], 2, xs[j]);
                }
        }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int64_t t = t0 + 32 * j + i32;
        if (t >= a.m.n_tok) continue;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int64_t r = r0 + 32 * i + 8 * (e >> 2) + 4 * h + (e & 3);
                if (r < a.m.d_out) a.m.Y[t * a.m.ld_y + r] = acc[i][j][e];
            }
    }
}

template <Act DT>
void launch_16bit(const MatArgs& a, hipStream_t s) {
    if (a.n_tok <= 16) {
        hipLaunchKernelGGL((mx_few_kernel<DT, 1>), dim3((unsigned)ceil_div(a.d_out, 16)), dim3(64 * FEW_WAVES), 0, s, a);
    } else if (a.n_tok <= 64) {
        hipLaunchKernelGGL((mx_few_kernel<DT, 2>), dim3((unsigned)ceil_div(a.d_out, 16), (unsigned)ceil_div(a.n_tok, 32)),
                           dim3(64 * FEW_WAVES), 0, s, a);
    } else {
        hipLaunchKernelGGL(mx_many_kernel<DT>, dim3((unsigned)ceil_div(a.d_out, MT), (unsigned)ceil_div(a.n_tok, MT)),
                           dim3(256), 0, s, a);
    }
}

MatArgs mat_args(const uint8_t* codes, const uint8_t* scales, int64_t n_tok, int64_t d_in, int64_t d_out, float* Y,
                 int64_t ld_y) {
    MatArgs a;
    a.X = nullptr;
    a.XS = nullptr;
    a.ld_x = 0;
    a.aligned = false;
    a.n_tok = n_tok;
    a.d_in = d_in;
    a.W = codes;
    a.S = scales;
    a.w_row = mx_code_bytes(d_in, GPTQ_MX_FP4);
    a.s_row = mx_scale_bytes(d_in);
    a.steps = (int)ceil_div(d_in, MX_PAD);
    a.d_out = d_out;
    a.ld_y = ld_y;
    a.Y = Y;
    return a;
}

}  // namespace

gptq_status mx_matmul_launch(const void* X, gptq_dtype dt, int64_t n_tok, int64_t d_in, int64_t ld_x,
                             const uint8_t* codes, const uint8_t* scales, int64_t d_out, float* Y, int64_t ld_y,
                             hipStream_t s) {
    MatArgs a = mat_args(codes, scales, n_tok, d_in, d_out, Y, ld_y);
    a.X = X;
    a.ld_x = ld_x;
    a.aligned = ((uintptr_t)X | (uintptr_t)(ld_x * (dt == GPTQ_F32 ? 4 : 2))) % 16 == 0;
    switch (dt) {
        case GPTQ_BF16: launch_16bit<ACT_BF16>(a, s); break;
        case GPTQ_F16: launch_16bit<ACT_F16>(a, s); break;
        default: launch_16bit<ACT_F32>(a, s); break;
    }
    GPTQ_LAUNCH_CHECK();
    return GPTQ_OK;
}

gptq_status mx_matmul_quantized_launch(const uint8_t* xc, const uint8_t* xs, gptq_mx_format xf, int64_t n_tok,
                                       int64_t d_in, const uint8_t* codes, const uint8_t* scales, int64_t d_out,
                                       float* Y, int64_t ld_y, hipStream_t s) {
    MatArgs m = mat_args(codes, scales, n_tok, d_in, d_out, Y, ld_y);
    if (xf == GPTQ_MX_FP8) {
        m.X = xc;
        m.XS = xs;
        m.ld_x = mx_code_bytes(d_in, xf);
        launch_16bit<ACT_FP8>(m, s);
    } else {
        const MxArgs a{xc, xs, m};
        hipLaunchKernelGGL(mx_mx_kernel, dim3((unsigned)ceil_div(d_out, 128), (unsigned)ceil_div(n_tok, 128)), dim3(256),
                           0, s, a);
    }
    GPTQ_LAUNCH_CHECK();
    return GPTQ_OK;
}

}  // namespace gptq
