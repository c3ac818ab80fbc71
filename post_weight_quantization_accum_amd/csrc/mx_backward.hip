// Gradients of products with e2m1 weights for their activations:
// dX = dY W (include/gptq.h, gptq_mx_matmul_backward), and of gated products,
// dX = dG Wg + dU Wu (gptq_mx_gated_backward).
#include <algorithm>

#include "gated.hpp"

namespace gptq {
namespace {

// float32 as three bfloat16 parts that sum to it (two: of values that two hold,
// as float16 ones); below an infinity or NaN the others are 0.
template <int NP>
__device__ __forceinline__ void cut(const float (&v)[8], u32x4_t (&p)[NP]) {
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = v[i];
#pragma unroll
    for (int j = 0; j < NP; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t w[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float& y = x[2 * i + k];
                w[k] = __float_as_uint(y);
                const bool fin = (w[k] & 0x7F800000u) != 0x7F800000u;
                y = fin ? y - __uint_as_float(w[k] & 0xFFFF0000u) : 0.0f;
                if ((w[k] & 0x7FFFFFFFu) > 0x7F800000u) w[k] |= 0x00400000u;      // a NaN stays one
            }
            p[j][i] = __builtin_amdgcn_perm(w[1], w[0], 0x07060302u);
        }
}

// One call, as the kernels see it: steps of KS rows of the matrices in a row,
// the last of each matrix padded with zeros.
struct Call {
    BackArgs b;
    int64_t w_row, s_row;      // bytes per row
    int steps, per;            // steps of one matrix; steps of one part
    int parts;
    float* sums;               // [part][token][d_in], of more than one part
    bool d_vec, out4;          // D's rows start on 16 bytes; dX's groups of four on their own size
};

// ---------------------------------------------------------------------------
// 128 columns x 128 tokens per workgroup of 2 x 2 waves of 64 x 64 in
// v_mfma_f32_32x32x16, one step of 32 rows at a time through LDS.  The weights'
// rows are the sum's index here, and a lane of the instruction wants eight of
// them in a column: codes are converted eight columns of a row at a time (one
// scale), and the halves of two rows' results make the pairs (two byte permutes
// for four values).
// ---------------------------------------------------------------------------
constexpr int KS = 32, BT = 128, ROW = KS * 2 + 16;

template <gptq_dtype DT>
__global__ __launch_bounds__(256) void mx_back_kernel(Call c) {
    constexpr int NP = DT == GPTQ_F32 ? 3 : DT == GPTQ_F16 ? 2 : 1;
    __shared__ __attribute__((aligned(16))) char wl[BT * ROW], xl[NP * BT * ROW];
    const BackArgs& a = c.b;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i32 = lane & 31, h = lane >> 5;
    const int64_t n0 = (int64_t)blockIdx.x * BT, t0 = (int64_t)blockIdx.y * BT;
    const int nw = 64 * (wave >> 1), tw = 64 * (wave & 1);
    f16_t acc[2][2];
    bool left = false;

    const auto multiply = [&](auto half) {
        constexpr bool HALF = decltype(half)::value;
        constexpr int PARTS = HALF ? 1 : NP;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
        const int first = blockIdx.z * c.per, end = min(first + c.per, c.steps * a.matrices);
        for (int st = first; st < end; ++st) {
            const int m = st >= c.steps;
            const int64_t k0 = (int64_t)(m ? st - c.steps : st) * KS;
            __syncthreads();
            // weights: this thread's two rows and eight columns
            {
                const int o = threadIdx.x & 15, k = 2 * (threadIdx.x >> 4);
                uint32_t w[2] = {0u, 0u};
                float s[2] = {0.f, 0.f};
                const int64_t col = n0 + 8 * o;
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    if (k0 + k + e < a.rows && col < 2 * c.w_row) {
                        w[e] = *(const uint32_t*)(a.codes[m] + (k0 + k + e) * c.w_row + col / 2);
                        uint32_t byte = a.scales[m][(k0 + k + e) * c.s_row + col / 32];
                        if (HALF && byte - 104u > 36u) {
                            left |= w[e] != 0u || byte == 255u;
                            w[e] = 0u;
                            byte = 127u;
                        }
                        s[e] = mx_scale(byte);
                    }
                const u32x4_t r0 = fp4x8<!HALF>(w[0], s[0]), r1 = fp4x8<!HALF>(w[1], s[1]);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    *(uint32_t*)(wl + (8 * o + 2 * q) * ROW + 2 * k) = __builtin_amdgcn_perm(r1[q], r0[q], 0x05040100u);
                    *(uint32_t*)(wl + (8 * o + 2 * q + 1) * ROW + 2 * k) = __builtin_amdgcn_perm(r1[q], r0[q], 0x07060302u);
                }
            }
            // gradients: eight rows of a token at a time
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int e = threadIdx.x + 256 * q, t = e >> 2, k = 8 * (e & 3);
                float v[8];
                const int64_t tok = t0 + t;
                const int n = tok < a.n_tok ? (int)max((int64_t)0, min((int64_t)8, a.rows - k0 - k)) : 0;
                load8_f32(a.D, DT, min(tok, a.n_tok - 1) * a.ld + m * a.d2 + k0 + k, n, c.d_vec && n == 8, v);
                u32x4_t p[PARTS];
                if constexpr (PARTS > 1) {
                    cut(v, p);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) p[0][i] = H16<!HALF>::pack(v[2 * i], v[2 * i + 1]);
                }
#pragma unroll
                for (int j = 0; j < PARTS; ++j) *(u32x4_t*)(xl + (j * BT + t) * ROW + 2 * k) = p[j];
            }
            __syncthreads();
#pragma unroll
            for (int k = 0; k < KS / 16; ++k)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const u32x4_t w = *(const u32x4_t*)(wl + (nw + 32 * i + i32) * ROW + 32 * k + 16 * h);
#pragma unroll
                    for (int p = 0; p < PARTS; ++p)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const u32x4_t x = *(const u32x4_t*)(xl + (p * BT + tw + 32 * j + i32) * ROW + 32 * k + 16 * h);
                            acc[i][j] = H16<!HALF>::mfma32(w, x, acc[i][j]);
                        }
                }
        }
    };
    multiply(std::integral_constant<bool, DT == GPTQ_F16>{});
    if constexpr (DT == GPTQ_F16) {
        if (__syncthreads_or(left)) multiply(std::false_type{});
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int64_t t = t0 + tw + 32 * j + i32;
        if (t >= a.n_tok) continue;
        const int e2 = a.exps ? a.exps[t] : 0;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
                const int64_t n = n0 + nw + 32 * i + 2 * e + 4 * h;
                if (n >= a.d_in) continue;
                float v[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) v[q] = acc[i][j][e + q];
                const int m = (int)min((int64_t)4, a.d_in - n);
                if (c.parts > 1) {
                    put4(c.sums, GPTQ_F32, m == 4 && a.d_in % 4 == 0, ((int64_t)blockIdx.z * a.n_tok + t) * a.d_in + n, m, v);
                } else {
#pragma unroll
                    for (int q = 0; q < 4; ++q) v[q] = ldexpf(v[q], e2);
                    put4(a.dX, a.dx_dt, c.out4 && m == 4, t * a.ld_dx + n, m, v);
                }
            }
    }
}

// dX from the parts' sums, in the order of the parts (zeros of none).
__global__ __launch_bounds__(256) void mx_back_join_kernel(Call c) {
    const BackArgs& a = c.b;
    const int64_t n = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4, t = blockIdx.y;
    if (n >= a.d_in) return;
    const int m = (int)min((int64_t)4, a.d_in - n);
    const bool whole = m == 4 && a.d_in % 4 == 0;
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    for (int p = 0; p < c.parts; ++p) {
        const float* s = c.sums + ((int64_t)p * a.n_tok + t) * a.d_in + n;
        if (whole) {
            const f32x4_t x = *(const f32x4_t*)s;
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] += x[q];
        } else {
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (q < m) v[q] += s[q];
        }
    }
    const int e2 = a.exps ? a.exps[t] : 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = ldexpf(v[q], e2);
    put4(a.dX, a.dx_dt, c.out4 && m == 4, t * a.ld_dx + n, m, v);
}

// ---------------------------------------------------------------------------
// A token's dG and dU.  One workgroup a token, which looks for its largest
// finite value first and scales by a power of two; float32 ones are kept as
// they are.
// ---------------------------------------------------------------------------
struct Gates {
    GatedBackArgs a;
    void* D;                   // [token][2][pad]
    int64_t pad;
    int32_t* exps;             // null for float32
    bool vec, vec_out;
};

__device__ __forceinline__ void gate_gradients(const Gates& c, int64_t t, int64_t k, float (&g)[8], float (&u)[8]) {
    const GatedBackArgs& a = c.a;
    const int n = (int)max((int64_t)0, min((int64_t)8, a.d_ff - k));
    float dy[8], gv[8], uv[8];
    load8_f32(a.dY, a.dt, t * a.ld_dy + k, n, c.vec && n == 8, dy);
    load8_f32(a.G, a.dt, t * a.ld_gu + k, n, c.vec && n == 8, gv);
    load8_f32(a.U, a.dt, t * a.ld_gu + k, n, c.vec && n == 8, uv);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float value, slope;
        activate_with_slope(a.act, gv[i], value, slope);
        g[i] = dy[i] * uv[i] * slope;
        u[i] = dy[i] * value;
    }
}

__global__ __launch_bounds__(256) void mx_gates_kernel(Gates c) {
    __shared__ float top[4];
    const GatedBackArgs& a = c.a;
    const int64_t t = blockIdx.x;
    const auto finite_max = [](float m, float v) { return __builtin_isfinite(v) ? fmaxf(m, fabsf(v)) : m; };
    int e2 = 0;
    if (c.exps) {
        float m = 0.0f;
        for (int64_t k = 8 * threadIdx.x; k < a.d_ff; k += 2048) {
            float g[8], u[8];
            gate_gradients(c, t, k, g, u);
#pragma unroll
            for (int i = 0; i < 8; ++i) m = finite_max(finite_max(m, g[i]), u[i]);
        }
#pragma unroll
        for (int s = 32; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor(m, s, 64));
        if ((threadIdx.x & 63) == 0) top[threadIdx.x >> 6] = m;
        __syncthreads();
        m = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
        if (m > 0.0f) {
            frexpf(m, &e2);                      // m = f 2^e2, f in [1/2, 1)
            e2 = 15 - e2;
        }
        if (threadIdx.x == 0) c.exps[t] = -e2;
    }
    for (int64_t k = 8 * threadIdx.x; k < c.pad; k += 2048) {
        float g[8], u[8];
        gate_gradients(c, t, k, g, u);
        const int n = (int)max((int64_t)0, min((int64_t)8, a.d_ff - k));
        if (a.dG) {
            store8(a.dG, a.dt, t * a.ld_dgu + k, n, c.vec_out && n == 8, g);
            store8(a.dU, a.dt, t * a.ld_dgu + k, n, c.vec_out && n == 8, u);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {            // past d_ff: zeros, whatever act(0) is
            g[i] = i < n ? ldexpf(g[i], e2) : 0.0f;
            u[i] = i < n ? ldexpf(u[i], e2) : 0.0f;
        }
        const gptq_dtype dt = c.exps ? GPTQ_F16 : GPTQ_F32;
        store8(c.D, dt, t * 2 * c.pad + k, 8, true, g);
        store8(c.D, dt, (t * 2 + 1) * c.pad + k, 8, true, u);
    }
}

// Parts of the sum's rows: as many as fill the chip once.
Call plan(const BackArgs& a) {
    Call c{};
    c.b = a;
    c.w_row = mx_code_bytes(a.d_in, GPTQ_MX_FP4);
    c.s_row = mx_scale_bytes(a.d_in);
    c.steps = (int)ceil_div(a.rows, KS);
    const int64_t tiles = ceil_div(a.d_in, BT) * ceil_div(a.n_tok, BT), all = (int64_t)c.steps * a.matrices;
    const int64_t want = std::max<int64_t>(1, std::min<int64_t>(512 / tiles, all / 8));
    c.per = (int)std::max<int64_t>(1, ceil_div(all, want));
    c.parts = (int)ceil_div(all, c.per);
    return c;
}

}  // namespace

size_t mx_backward_ws(gptq_dtype dt, int matrices, int64_t n_tok, int64_t d_in, int64_t rows) {
    BackArgs a{};
    a.dt = dt;
    a.matrices = matrices;
    a.n_tok = n_tok;
    a.d_in = d_in;
    a.rows = rows;
    const Call c = plan(a);
    return c.parts > 1 ? (size_t)c.parts * n_tok * d_in * sizeof(float) : 0;
}

gptq_status mx_backward_launch(const BackArgs& a, void* ws, hipStream_t s) {
    Call c = plan(a);
    const int size = a.dt == GPTQ_F32 ? 4 : 2, four = a.dx_dt == GPTQ_F32 ? 16 : 8;
    c.sums = (float*)ws;
    c.d_vec = ((uintptr_t)a.D | (uintptr_t)(a.ld * size) | (uintptr_t)(a.d2 * size)) % 16 == 0;
    c.out4 = ((uintptr_t)a.dX | (uintptr_t)(a.ld_dx * (four / 4))) % four == 0;
    if (c.parts > 0) {
        const dim3 grid((unsigned)ceil_div(a.d_in, BT), (unsigned)ceil_div(a.n_tok, BT), (unsigned)c.parts);
        switch (a.dt) {
            case GPTQ_BF16: mx_back_kernel<GPTQ_BF16><<<grid, 256, 0, s>>>(c); break;
            case GPTQ_F16: mx_back_kernel<GPTQ_F16><<<grid, 256, 0, s>>>(c); break;
            default: mx_back_kernel<GPTQ_F32><<<grid, 256, 0, s>>>(c); break;
        }
        GPTQ_LAUNCH_CHECK();
    }
    if (c.parts != 1) {
        for (int64_t t = 0; t < a.n_tok; t += 65535) {
            Call j = c;
            const int64_t n = std::min<int64_t>(65535, a.n_tok - t);
            j.b.dX = (char*)a.dX + t * a.ld_dx * (four / 4);
            if (j.sums) j.sums += t * a.d_in;
            if (a.exps) j.b.exps += t;
            mx_back_join_kernel<<<dim3((unsigned)ceil_div(a.d_in, 1024), (unsigned)n), 256, 0, s>>>(j);
            GPTQ_LAUNCH_CHECK();
        }
    }
    return GPTQ_OK;
}

namespace {

int64_t gates_pad(int64_t d_ff) { return ceil_div(d_ff, 64) * 64; }
size_t gates_bytes(gptq_dtype dt, int64_t n_tok, int64_t d_ff) {
    return align_up((size_t)n_tok * 2 * gates_pad(d_ff) * (dt == GPTQ_F32 ? 4 : 2) + (dt == GPTQ_F32 ? 0 : 4 * (size_t)n_tok), 256);
}

}  // namespace

size_t mx_gated_backward_ws(gptq_dtype dt, int64_t n_tok, int64_t d_in, int64_t d_ff) {
    return gates_bytes(dt, n_tok, d_ff) + mx_backward_ws(dt == GPTQ_F32 ? GPTQ_F32 : GPTQ_F16, 2, n_tok, d_in, d_ff);
}

gptq_status mx_gated_backward_launch(const GatedBackArgs& a, void* ws, hipStream_t s) {
    const bool wide = a.dt == GPTQ_F32;
    const int size = wide ? 4 : 2;
    const int64_t pad = gates_pad(a.d_ff);
    BackArgs b{};
    b.D = ws;
    b.dt = wide ? GPTQ_F32 : GPTQ_F16;
    b.n_tok = a.n_tok;
    b.ld = 2 * pad;
    b.d2 = pad;
    b.matrices = 2;
    b.rows = a.d_ff;
    b.d_in = a.d_in;
    b.dX = a.dX;
    b.dx_dt = a.dx_dt;
    b.ld_dx = a.ld_dx;
    for (int m = 0; m < 2; ++m) {
        b.codes[m] = a.codes[m];
        b.scales[m] = a.scales[m];
    }
    if (a.d_ff > 0) {
        Gates g{};
        g.a = a;
        g.D = ws;
        g.pad = pad;
        g.exps = wide ? nullptr : (int32_t*)((char*)ws + (size_t)a.n_tok * 2 * pad * size);
        const auto fits = [&](const void* p, int64_t ld) { return ((uintptr_t)p | (uintptr_t)(ld * size)) % 16 == 0; };
        g.vec = fits(a.dY, a.ld_dy) && fits(a.G, a.ld_gu) && fits(a.U, a.ld_gu);
        g.vec_out = a.dG && fits(a.dG, a.ld_dgu) && fits(a.dU, a.ld_dgu);
        mx_gates_kernel<<<(unsigned)a.n_tok, 256, 0, s>>>(g);
        GPTQ_LAUNCH_CHECK();
        b.exps = g.exps;
    }
    return mx_backward_launch(b, (char*)ws + gates_bytes(a.dt, a.n_tok, a.d_ff), s);
}

}  // namespace gptq
