// Norms around a block and their gradient (include/gptq.h, gptq_residual_norm
// and gptq_residual_norm_backward).
//
// A row is read once into registers, by one wave where it is short and by a
// workgroup otherwise, and everything about it is computed from there: no
// value is read twice but by rows of more than 16384 values (wide kernels).
// Sums over a row are float64: the squares of float32 values leave float32's
// range, and mean and variance come from one pass (sum and sum of squares)
// without the loss that float32 would have there.  They cost a few percent of
// what the row's bytes take.  All else is float32.
#include "norm.hpp"

#include <algorithm>
#include <type_traits>

namespace gptq {
namespace {

constexpr int MAX_WAVES = 16;

// ---------------------------------------------------------------------------
// Eight values of a row by a lane.  VEC (every row starts on 16 bytes, d a
// multiple of 8): eight in a row; else every T-th, so that neighbouring lanes
// read neighbouring values all the same.
// ---------------------------------------------------------------------------
struct Piece {
    uint32_t w[8];
};

template <bool VEC>
__device__ __forceinline__ int column(int v, int e, int T, int t) {
    return VEC ? (v * T + t) * 8 + e : (v * 8 + e) * T + t;
}

// Where a row starts: the same for all its lanes.
template <class P>
__device__ __forceinline__ P* row_at(P* p, gptq_dtype dt, int64_t elements) {
    using Byte = std::conditional_t<std::is_const_v<P>, const char, char>;
    return (P*)((Byte*)p + elements * (dt == GPTQ_F32 ? 4 : 2));
}

template <bool VEC>
__device__ __forceinline__ Piece load(const void* row, gptq_dtype dt, int v, int T, int t, int d) {
    Piece r;
#pragma unroll
    for (int e = 0; e < 8; ++e) r.w[e] = 0u;
    if constexpr (VEC) {
        const int c = column<true>(v, 0, T, t);
        if (c < d) {
            const uint4* q = (const uint4*)((const char*)row + (uint32_t)c * (dt == GPTQ_F32 ? 4u : 2u));
            const uint4 a = q[0];
            r.w[0] = a.x; r.w[1] = a.y; r.w[2] = a.z; r.w[3] = a.w;
            if (dt == GPTQ_F32) {
                const uint4 b = q[1];
                r.w[4] = b.x; r.w[5] = b.y; r.w[6] = b.z; r.w[7] = b.w;
            }
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int c = column<false>(v, e, T, t);
            if (c < d) r.w[e] = dt == GPTQ_F32 ? ((const uint32_t*)row)[c] : ((const uint16_t*)row)[c];
        }
    }
    return r;
}

template <bool VEC>
__device__ __forceinline__ void values(const Piece& r, gptq_dtype dt, float (&x)[8]) {
    const auto half = [&](int e) { return VEC ? r.w[e >> 1] >> (16 * (e & 1)) & 0xFFFFu : r.w[e]; };
    if (dt == GPTQ_F32) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = __uint_as_float(r.w[e]);
    } else if (dt == GPTQ_BF16) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = H16<true>::to_f32((uint16_t)half(e));
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = H16<false>::to_f32((uint16_t)half(e));
    }
}

template <bool VEC>
__device__ __forceinline__ void store(void* row, gptq_dtype dt, int v, int T, int t, int d, const float (&x)[8]) {
    if constexpr (VEC) {
        const int c = column<true>(v, 0, T, t);
        if (c >= d) return;
        char* p = (char*)row + (uint32_t)c * (dt == GPTQ_F32 ? 4u : 2u);
        if (dt == GPTQ_F32) {
            ((float4*)p)[0] = make_float4(x[0], x[1], x[2], x[3]);
            ((float4*)p)[1] = make_float4(x[4], x[5], x[6], x[7]);
        } else if (dt == GPTQ_BF16) {
            *(uint4*)p = make_uint4(H16<true>::pack(x[0], x[1]), H16<true>::pack(x[2], x[3]), H16<true>::pack(x[4], x[5]),
                                    H16<true>::pack(x[6], x[7]));
        } else {
            *(uint4*)p = make_uint4(H16<false>::pack(x[0], x[1]), H16<false>::pack(x[2], x[3]), H16<false>::pack(x[4], x[5]),
                                    H16<false>::pack(x[6], x[7]));
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int c = column<false>(v, e, T, t);
            if (c >= d) continue;
            if (dt == GPTQ_F32) ((float*)row)[c] = x[e];
            else ((uint16_t*)row)[c] = (uint16_t)(dt == GPTQ_BF16 ? H16<true>::pack(x[e], 0.f) : H16<false>::pack(x[e], 0.f));
        }
    }
}

// A vector of d values, or `none` of them.
template <bool VEC>
__device__ __forceinline__ void vector(const void* p, gptq_dtype dt, int v, int T, int t, int d, float none, float (&x)[8]) {
    if (p) {
        values<VEC>(load<VEC>(p, dt, v, T, t, d), dt, x);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = none;
    }
}

// ---------------------------------------------------------------------------
// Sums over a row's lanes, the same bits in all of them.
// ---------------------------------------------------------------------------
template <int CTRL>
__device__ __forceinline__ double moved(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, 0xF, 0xF, true);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, 0xF, 0xF, true);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double sum_of_16(double v) {
    v += moved<0xB1>(v);         // the neighbour's
    v += moved<0x4E>(v);         // the other pair's of four
    v += moved<0x141>(v);        // the other four's of eight
    v += moved<0x140>(v);        // the other eight's
    return v;
}
__device__ __forceinline__ double wave_sum(double v) {
    v = sum_of_16(v);
    v += __shfl_xor(v, 16, 64);
    v += __shfl_xor(v, 32, 64);
    return v;
}

template <int K>
using Sums = double[2][MAX_WAVES][K];

// Of K sums over the workgroup (over the wave where it has the row).  `turn`
// alternates, so that one barrier a sum is enough: who writes a half again has
// passed the barrier of the other in between, which nobody reaches before
// having read.  The barrier waits for LDS alone: rows asked for ahead and results
// on their way out stay under way (with __syncthreads() 8000 rows of 5120 took
// half as long again).
template <bool WAVE, int K, int KMAX>
__device__ __forceinline__ void row_sums(double (&v)[K], Sums<KMAX>& lds, int& turn) {
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = wave_sum(v[k]);
    if constexpr (!WAVE) {
        const int waves = blockDim.x >> 6;
        if (waves == 1) return;
        if ((threadIdx.x & 63) == 0) {
#pragma unroll
            for (int k = 0; k < K; ++k) lds[turn][threadIdx.x >> 6][k] = v[k];
        }
        meet();
        const int w = threadIdx.x & 15;
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] = w < waves ? lds[turn][w][k] : 0.0;
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] = sum_of_16(v[k]);
        turn ^= 1;
    }
}

// Mean (0 of an rms norm) and reciprocal deviation from a row's sum and sum of squares.
struct Stat {
    float mean, rstd;
};
__device__ __forceinline__ Stat stat(const NormArgs& a, double sum, double sq) {
    const double m = a.layer ? sum * a.inv_d : 0.0;
    const double var = sq * a.inv_d - m * m, x = (var < 0.0 ? 0.0 : var) + (double)a.eps;        // a NaN stays one
    // the hardware's estimate and one step of Newton's: far beyond float32
    const double r = __builtin_amdgcn_rsq(x);
    const bool inside = x > 0.0 && x < __builtin_inf();
    return Stat{(float)m, (float)(inside ? r * fma(-0.5 * x * r, r, 1.5) : r)};
}

// One piece of h = scale x + gate p, p the block's output (normalised).
template <bool VEC>
__device__ __forceinline__ void stream_value(const NormArgs& a, int64_t row, int v, int T, int t, Stat sb, const Piece& xr,
                                             const Piece& br, float (&h)[8]) {
    float p[8];
    values<VEC>(xr, a.x_dt, h);
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] *= a.scale;
    if (!a.B) return;
    values<VEC>(br, a.b_dt, p);
    if (a.post) {
        float w[8];
        vector<VEC>(a.post, a.v_dt, v, T, t, a.d, 1.0f, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) p[e] = (p[e] - sb.mean) * sb.rstd * w[e];
    }
    if (a.gate) {
        float g[8];
        values<VEC>(load<VEC>(row_at(a.gate, a.v_dt, row * a.ld_gate), a.v_dt, v, T, t, a.d), a.v_dt, g);
#pragma unroll
        for (int e = 0; e < 8; ++e) h[e] = fmaf(g[e], p[e], h[e]);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) h[e] += p[e];
    }
}

template <bool VEC>
__device__ __forceinline__ void write_y(const NormArgs& a, int64_t row, int v, int T, int t, Stat s, const float (&h)[8]) {
    float w[8], c[8];
    vector<VEC>(a.weight, a.v_dt, v, T, t, a.d, 1.0f, w);
    vector<VEC>(a.bias, a.v_dt, v, T, t, a.d, 0.0f, c);
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = fmaf((h[e] - s.mean) * s.rstd, w[e], c[e]);
    store<VEC>(row_at(a.Y, a.y_dt, row * a.ld_y), a.y_dt, v, T, t, a.d, w);
}

// A workgroup (a wave) takes every ROWS-th row and asks for the next one before it
// works on its own.  Lanes past the row's end hold zeros, which add nothing to
// sums.
template <int V, bool VEC, bool WAVE>
__global__ __launch_bounds__(WAVE ? 256 : 1024) void norm_kernel(NormArgs a) {
    __shared__ Sums<2> lds;
    const int T = WAVE ? 64 : blockDim.x, t = WAVE ? threadIdx.x & 63 : threadIdx.x;
    const int64_t first = WAVE ? (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)) : blockIdx.x;
    const int64_t rows = WAVE ? (int64_t)gridDim.x * 4 : gridDim.x;
    if (WAVE && first >= a.n_tok) return;
    Piece nx[V], nb[V];
    const auto ask = [&](int64_t row) {
#pragma unroll
        for (int v = 0; v < V; ++v) nx[v] = load<VEC>(row_at(a.X, a.x_dt, row * a.ld_x), a.x_dt, v, T, t, a.d);
        if (a.B) {
#pragma unroll
            for (int v = 0; v < V; ++v) nb[v] = load<VEC>(row_at(a.B, a.b_dt, row * a.ld_b), a.b_dt, v, T, t, a.d);
        }
    };
    ask(first);
    int turn = 0;
    for (int64_t row = first; row < a.n_tok; row += rows) {
        Piece x[V], b[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            x[v] = nx[v];
            b[v] = nb[v];
        }
        if (row + rows < a.n_tok) ask(row + rows);
        Stat sb{0.f, 0.f};
        if (a.post) {
            double s[2] = {0.0, 0.0};
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float p[8];
                values<VEC>(b[v], a.b_dt, p);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    s[0] += (double)p[e];
                    s[1] = fma((double)p[e], (double)p[e], s[1]);
                }
            }
            row_sums<WAVE, 2, 2>(s, lds, turn);
            sb = stat(a, s[0], s[1]);
        }
        float h[V][8];
        double s[2] = {0.0, 0.0};
#pragma unroll
        for (int v = 0; v < V; ++v) {
            stream_value<VEC>(a, row, v, T, t, sb, x[v], b[v], h[v]);
            if (a.H) store<VEC>(row_at(a.H, a.h_dt, row * a.ld_h), a.h_dt, v, T, t, a.d, h[v]);
            if (!a.Y) continue;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const bool is = column<VEC>(v, e, T, t) < a.d;   // a layer norm's p of a lane past the end is not 0
                const double q = is ? (double)h[v][e] : 0.0;
                s[0] += q;
                s[1] = fma(q, q, s[1]);
            }
        }
        if (!a.Y) continue;
        row_sums<WAVE, 2, 2>(s, lds, turn);
        const Stat sh = stat(a, s[0], s[1]);
#pragma unroll
        for (int v = 0; v < V; ++v) write_y<VEC>(a, row, v, T, t, sh, h[v]);
    }
}

// Rows that registers do not hold: sums in one pass over them, values in the next.
template <bool VEC>
__global__ __launch_bounds__(1024) void norm_wide_kernel(NormArgs a) {
    __shared__ Sums<2> lds;
    const int T = blockDim.x, t = threadIdx.x;
    const int64_t row = blockIdx.x;
    const int n = (int)((a.d + 8 * T - 1) / (8 * T));
    int turn = 0;
    Stat sb{0.f, 0.f};
    if (a.post) {
        double s[2] = {0.0, 0.0};
        for (int v = 0; v < n; ++v) {
            float p[8];
            values<VEC>(load<VEC>(row_at(a.B, a.b_dt, row * a.ld_b), a.b_dt, v, T, t, a.d), a.b_dt, p);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                s[0] += (double)p[e];
                s[1] = fma((double)p[e], (double)p[e], s[1]);
            }
        }
        row_sums<false, 2, 2>(s, lds, turn);
        sb = stat(a, s[0], s[1]);
    }
    const auto value = [&](int v, float (&h)[8]) {
        const Piece x = load<VEC>(row_at(a.X, a.x_dt, row * a.ld_x), a.x_dt, v, T, t, a.d);
        Piece b = x;
        if (a.B) b = load<VEC>(row_at(a.B, a.b_dt, row * a.ld_b), a.b_dt, v, T, t, a.d);
        stream_value<VEC>(a, row, v, T, t, sb, x, b, h);
    };
    Stat sh{0.f, 0.f};
    if (a.Y) {
        double s[2] = {0.0, 0.0};
        for (int v = 0; v < n; ++v) {
            float h[8];
            value(v, h);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const double q = column<VEC>(v, e, T, t) < a.d ? (double)h[e] : 0.0;
                s[0] += q;
                s[1] = fma(q, q, s[1]);
            }
        }
        row_sums<false, 2, 2>(s, lds, turn);
        sh = stat(a, s[0], s[1]);
    }
    for (int v = 0; v < n; ++v) {
        float h[8];
        value(v, h);
        if (a.H) store<VEC>(row_at(a.H, a.h_dt, row * a.ld_h), a.h_dt, v, T, t, a.d, h);      // may be X: its values are read
        if (a.Y) write_y<VEC>(a, row, v, T, t, sh, h);
    }
}

// ---------------------------------------------------------------------------
// The gradient.  With n the normalised row, r its reciprocal deviation and t
// the gradient for n,
//     r (t - n mean(t n) - mean(t))      (mean(t): layer norms only)
// is that for the row.  mean(t n) = r (sum(t h) - m sum(t)) / d, so that one
// round of sums (h, h^2, t, t h, and b, b^2 for the norm of the block's output)
// serves the stream's norm; the output's own gradient needs one more.
//
// Sums over tokens: a workgroup takes every PARTS-th row (a wave where it has
// the row), adds up its rows' terms in registers and leaves them as one part;
// a second kernel adds the parts in order, in float64.  No atomics: the same
// call gives the same bits.
// ---------------------------------------------------------------------------
enum Vec : int { V_WEIGHT = 0, V_BIAS, V_POST, V_GATE, N_VEC };

__device__ __forceinline__ float through(float t, float n, float r, float mt, float mtn) { return r * (t - mt - n * mtn); }

// What one row's first round of sums is taken over.
struct RowSums {
    Stat h, b;
    float mt, mtn;
};
__device__ __forceinline__ RowSums first_round(const NormGradArgs& a, const double (&s)[6]) {
    RowSums r;
    r.h = stat(a.f, s[0], s[1]);
    r.b = a.f.post ? stat(a.f, s[4], s[5]) : Stat{0.f, 0.f};
    r.mt = a.f.layer ? (float)(s[2] * a.f.inv_d) : 0.0f;
    r.mtn = (float)((s[3] - (double)r.h.mean * s[2]) * (double)r.h.rstd * a.f.inv_d);
    return r;
}

template <bool VEC>
__device__ __forceinline__ void first_sums(const NormGradArgs& a, const Piece& hr, const Piece& yr, const Piece& br, int v,
                                           int T, int t, double (&s)[6]) {
    float h[8], dy[8], w[8], b[8];
    values<VEC>(hr, a.h_dt, h);
    values<VEC>(yr, a.dy_dt, dy);
    vector<VEC>(a.f.weight, a.f.v_dt, v, T, t, a.f.d, 1.0f, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const double x = (double)h[e], g = (double)(dy[e] * w[e]);       // both 0 past the end
        s[0] += x;
        s[1] = fma(x, x, s[1]);
        s[2] += g;
        s[3] = fma(g, x, s[3]);
    }
    if (!a.f.post) return;
    values<VEC>(br, a.f.b_dt, b);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        s[4] += (double)b[e];
        s[5] = fma((double)b[e], (double)b[e], s[5]);
    }
}

// Of one piece: the gradient of the stream (also stored for x), the terms of
// the vectors' gradients, and what the output's gradient is before its norm
// (q), with the output's normalised values (nb).
template <bool VEC>
__device__ __forceinline__ void stream_gradient(const NormGradArgs& a, int64_t row, int v, int T, int t, const RowSums& r,
                                                const Piece& hr, const Piece& yr, const Piece& br, const Piece& ghr,
                                                float (&sum)[N_VEC][8], float (&q)[8], float (&nb)[8]) {
    float h[8], dy[8], w[8], D[8];
    values<VEC>(hr, a.h_dt, h);
    values<VEC>(yr, a.dy_dt, dy);
    vector<VEC>(a.f.weight, a.f.v_dt, v, T, t, a.f.d, 1.0f, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float n = (h[e] - r.h.mean) * r.h.rstd;
        D[e] = through(dy[e] * w[e], n, r.h.rstd, r.mt, r.mtn);
        sum[V_WEIGHT][e] = fmaf(dy[e], n, sum[V_WEIGHT][e]);
        sum[V_BIAS][e] += dy[e];
    }
    if (a.dH) {
        float g[8];
        values<VEC>(ghr, a.h_dt, g);
#pragma unroll
        for (int e = 0; e < 8; ++e) D[e] += g[e];
    }
    if (a.dX) {
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = D[e] * a.f.scale;
        store<VEC>(row_at(a.dX, a.h_dt, row * a.ld_dx), a.h_dt, v, T, t, a.f.d, x);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        q[e] = D[e];
        nb[e] = 0.0f;
    }
    if (!a.has_b) return;
    float p[8], pw[8];
    values<VEC>(br, a.f.b_dt, p);
    vector<VEC>(a.f.post, a.f.v_dt, v, T, t, a.f.d, 1.0f, pw);
#pragma unroll
    for (int e = 0; e < 8; ++e) nb[e] = a.f.post ? (p[e] - r.b.mean) * r.b.rstd : p[e];
    if (a.f.gate) {
        float g[8], each[8];
        values<VEC>(load<VEC>(row_at(a.f.gate, a.f.v_dt, row * a.f.ld_gate), a.f.v_dt, v, T, t, a.f.d), a.f.v_dt, g);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            each[e] = D[e] * (nb[e] * pw[e]);
            sum[V_GATE][e] += each[e];
            q[e] = D[e] * g[e];
        }
        if (a.d_gate_rows) store<VEC>(row_at(a.d_gate_rows, a.f.v_dt, row * a.ld_dgate), a.f.v_dt, v, T, t, a.f.d, each);
    }
    if (a.f.post) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            sum[V_POST][e] = fmaf(q[e], nb[e], sum[V_POST][e]);
            q[e] *= pw[e];
        }
    }
}

template <bool VEC>
__device__ __forceinline__ void second_sums(const NormGradArgs& a, int v, int T, int t, const float (&q)[8], const float (&nb)[8],
                                            double (&s)[2]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const bool is = column<VEC>(v, e, T, t) < a.f.d;
        const double x = is ? (double)q[e] : 0.0;
        s[0] += x;
        s[1] = fma(x, (double)nb[e], s[1]);
    }
}

template <bool VEC>
__device__ __forceinline__ void write_db(const NormGradArgs& a, int64_t row, int v, int T, int t, Stat sb, float mq, float mqn,
                                         float (&q)[8], const float (&nb)[8]) {
    if (a.f.post) {
#pragma unroll
        for (int e = 0; e < 8; ++e) q[e] = through(q[e], nb[e], sb.rstd, mq, mqn);
    }
    store<VEC>(row_at(a.dB, a.f.b_dt, row * a.ld_db), a.f.b_dt, v, T, t, a.f.d, q);
}

// One part's sums of vector k, if it is asked for.
template <bool VEC>
__device__ __forceinline__ void write_part(const NormGradArgs& a, int64_t part, int k, int v, int T, int t, const float (&x)[8]) {
    if (a.slot[k] < 0) return;
    store<VEC>(row_at(a.parts, GPTQ_F32, (part * a.n_slots + a.slot[k]) * a.ld_part), GPTQ_F32, v, T, t, a.f.d, x);
}

template <int V, bool VEC, bool WAVE>
__global__ __launch_bounds__(WAVE ? 256 : 512) void norm_grad_kernel(NormGradArgs a) {
    __shared__ Sums<6> lds;
    const int T = WAVE ? 64 : blockDim.x, t = WAVE ? threadIdx.x & 63 : threadIdx.x;
    const int64_t part = WAVE ? (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)) : blockIdx.x;
    const int64_t parts = WAVE ? (int64_t)gridDim.x * 4 : gridDim.x;
    float sum[V][N_VEC][8];
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int k = 0; k < N_VEC; ++k)
#pragma unroll
            for (int e = 0; e < 8; ++e) sum[v][k][e] = 0.0f;
    int turn = 0;
    Piece nh[V], ny[V], nb_[V], ng[V];
    const auto ask = [&](int64_t row) {          // the next row, before this one is worked on
#pragma unroll
        for (int v = 0; v < V; ++v) {
            nh[v] = load<VEC>(row_at(a.H, a.h_dt, row * a.ld_h), a.h_dt, v, T, t, a.f.d);
            ny[v] = load<VEC>(row_at(a.dY, a.dy_dt, row * a.ld_dy), a.dy_dt, v, T, t, a.f.d);
            if (a.has_b) nb_[v] = load<VEC>(row_at(a.f.B, a.f.b_dt, row * a.f.ld_b), a.f.b_dt, v, T, t, a.f.d);
            if (a.dH) ng[v] = load<VEC>(row_at(a.dH, a.h_dt, row * a.ld_dh), a.h_dt, v, T, t, a.f.d);
        }
    };
    if (part < a.f.n_tok) ask(part);
    for (int64_t row = part; row < a.f.n_tok; row += parts) {
        Piece h[V], y[V], b[V], g[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            h[v] = nh[v];
            y[v] = ny[v];
            b[v] = nb_[v];
            g[v] = ng[v];
        }
        if (row + parts < a.f.n_tok) ask(row + parts);
        double s[6] = {0.0, 0.0, 0.0, 0.0, 0.0, 0.0};
#pragma unroll
        for (int v = 0; v < V; ++v) first_sums<VEC>(a, h[v], y[v], b[v], v, T, t, s);
        row_sums<WAVE, 6, 6>(s, lds, turn);
        const RowSums r = first_round(a, s);
        float q[V][8], nb[V][8];
#pragma unroll
        for (int v = 0; v < V; ++v) stream_gradient<VEC>(a, row, v, T, t, r, h[v], y[v], b[v], g[v], sum[v], q[v], nb[v]);
        if (!a.dB) continue;
        float mq = 0.f, mqn = 0.f;
        if (a.f.post) {
            double u[2] = {0.0, 0.0};
#pragma unroll
            for (int v = 0; v < V; ++v) second_sums<VEC>(a, v, T, t, q[v], nb[v], u);
            row_sums<WAVE, 2, 6>(u, lds, turn);
            mq = a.f.layer ? (float)(u[0] * a.f.inv_d) : 0.0f;
            mqn = (float)(u[1] * a.f.inv_d);
        }
#pragma unroll
        for (int v = 0; v < V; ++v) write_db<VEC>(a, row, v, T, t, r.b, mq, mqn, q[v], nb[v]);
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int k = 0; k < N_VEC; ++k) write_part<VEC>(a, part, k, v, T, t, sum[v][k]);
}

// Rows that registers do not hold: each pass over them reads them again, and
// the vectors' sums live in the part itself (every value a lane's own).
template <bool VEC>
__global__ __launch_bounds__(512) void norm_grad_wide_kernel(NormGradArgs a) {
    __shared__ Sums<6> lds;
    const int T = blockDim.x, t = threadIdx.x;
    const int64_t part = blockIdx.x;
    const int n = (int)((a.f.d + 8 * T - 1) / (8 * T));
    int turn = 0;
    bool first = true;
    for (int64_t row = part; row < a.f.n_tok; row += gridDim.x) {
        Piece h, y, b, g;
        const auto read = [&](int v) {
            h = load<VEC>(row_at(a.H, a.h_dt, row * a.ld_h), a.h_dt, v, T, t, a.f.d);
            y = load<VEC>(row_at(a.dY, a.dy_dt, row * a.ld_dy), a.dy_dt, v, T, t, a.f.d);
            b = g = h;
            if (a.has_b) b = load<VEC>(row_at(a.f.B, a.f.b_dt, row * a.f.ld_b), a.f.b_dt, v, T, t, a.f.d);
            if (a.dH) g = load<VEC>(row_at(a.dH, a.h_dt, row * a.ld_dh), a.h_dt, v, T, t, a.f.d);
        };
        double s[6] = {0.0, 0.0, 0.0, 0.0, 0.0, 0.0};
        for (int v = 0; v < n; ++v) {
            read(v);
            first_sums<VEC>(a, h, y, b, v, T, t, s);
        }
        row_sums<false, 6, 6>(s, lds, turn);
        const RowSums r = first_round(a, s);
        double u[2] = {0.0, 0.0};
        float mq = 0.f, mqn = 0.f;
        // the output's gradient needs the stream's first: a pass that stores
        // nothing, where there is a norm to go through
        NormGradArgs quiet = a;
        quiet.dX = nullptr;
        quiet.d_gate_rows = nullptr;
        if (a.dB && a.f.post) {
            for (int v = 0; v < n; ++v) {
                float sum[N_VEC][8], q[8], nb[8];
#pragma unroll
                for (int k = 0; k < N_VEC; ++k)
#pragma unroll
                    for (int e = 0; e < 8; ++e) sum[k][e] = 0.0f;
                read(v);
                stream_gradient<VEC>(quiet, row, v, T, t, r, h, y, b, g, sum, q, nb);
                second_sums<VEC>(a, v, T, t, q, nb, u);
            }
            row_sums<false, 2, 6>(u, lds, turn);
            mq = a.f.layer ? (float)(u[0] * a.f.inv_d) : 0.0f;
            mqn = (float)(u[1] * a.f.inv_d);
        }
        for (int v = 0; v < n; ++v) {
            float sum[N_VEC][8], q[8], nb[8];
#pragma unroll
            for (int k = 0; k < N_VEC; ++k) {
#pragma unroll
                for (int e = 0; e < 8; ++e) sum[k][e] = 0.0f;
                if (!first && a.slot[k] >= 0)
                    values<VEC>(load<VEC>(row_at(a.parts, GPTQ_F32, (part * a.n_slots + a.slot[k]) * a.ld_part), GPTQ_F32, v, T, t, a.f.d), GPTQ_F32,
                                sum[k]);
            }
            read(v);
            stream_gradient<VEC>(a, row, v, T, t, r, h, y, b, g, sum, q, nb);
            if (a.dB) write_db<VEC>(a, row, v, T, t, r.b, mq, mqn, q, nb);
#pragma unroll
            for (int k = 0; k < N_VEC; ++k) write_part<VEC>(a, part, k, v, T, t, sum[k]);
        }
        first = false;
    }
}

// out[slot][c] = the parts' sums: 64 columns by 16 shares of the parts.
__global__ __launch_bounds__(1024) void norm_join_kernel(const float* parts, int64_t n_parts, int n_slots, int64_t ld, int64_t d,
                                                         float* o0, float* o1, float* o2, float* o3) {
    __shared__ double lds[16][64];
    const int lane = threadIdx.x & 63, share = threadIdx.x >> 6;
    const int64_t c = (int64_t)blockIdx.x * 64 + lane;
    const int slot = blockIdx.y;
    double s = 0.0;
    if (c < d) {
        const float* p = parts + slot * ld + c;
        const int64_t end = n_parts * (share + 1) / 16;
        int64_t i = n_parts * share / 16;
        for (; i + 8 <= end; i += 8) {           // eight on their way at once
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = p[(i + e) * n_slots * ld];
#pragma unroll
            for (int e = 0; e < 8; ++e) s += (double)v[e];
        }
        for (; i < end; ++i) s += (double)p[i * n_slots * ld];
    }
    lds[share][lane] = s;
    __syncthreads();
    if (share == 0 && c < d) {
#pragma unroll
        for (int k = 1; k < 16; ++k) s += lds[k][lane];
        float* o = slot == 0 ? o0 : slot == 1 ? o1 : slot == 2 ? o2 : o3;
        o[c] = (float)s;
    }
}

bool rows_on_16(const void* p, gptq_dtype dt, int64_t ld) {
    return !p || ((uintptr_t)p | (uintptr_t)(ld * (dt == GPTQ_F32 ? 4 : 2))) % 16 == 0;
}

// Threads of a workgroup for rows of d values, eight or sixteen or 32 a lane.
unsigned threads_for(int64_t d, int pieces) { return (unsigned)(ceil_div(ceil_div(d, 8 * pieces), 64) * 64); }

template <bool VEC>
void launch_norm(const NormArgs& a, hipStream_t s) {
    // as many workgroups as the chip holds at once (2048 threads a compute unit)
    const auto groups = [&](int64_t rows, unsigned threads) { return (unsigned)std::min<int64_t>(rows, 256 * (2048 / threads)); };
    const unsigned n = (unsigned)a.n_tok, four = groups(ceil_div(a.n_tok, 4), 256), t1 = threads_for(a.d, 1), t2 = threads_for(a.d, 2);
    if (a.d <= 512) norm_kernel<1, VEC, true><<<four, 256, 0, s>>>(a);
    else if (a.d <= 1024) norm_kernel<2, VEC, true><<<four, 256, 0, s>>>(a);
    else if (a.d <= 8192) norm_kernel<1, VEC, false><<<groups(n, t1), t1, 0, s>>>(a);
    else if (a.d <= 16384) norm_kernel<2, VEC, false><<<groups(n, t2), t2, 0, s>>>(a);
    else norm_wide_kernel<VEC><<<n, 1024, 0, s>>>(a);
}

// Parts of the sums over tokens, and with them workgroups of the gradient.
int64_t grad_parts(int64_t n_tok, int64_t d) {
    if (d <= 1024) return std::min<int64_t>(ceil_div(n_tok, 4), 1024) * 4;      // a wave's rows
    return std::min<int64_t>(n_tok, 512);
}

template <bool VEC>
void launch_grad(const NormGradArgs& a, hipStream_t s) {
    const int64_t d = a.f.d;
    const unsigned n = (unsigned)grad_parts(a.f.n_tok, d);
    if (d <= 512) norm_grad_kernel<1, VEC, true><<<n / 4, 256, 0, s>>>(a);
    else if (d <= 1024) norm_grad_kernel<2, VEC, true><<<n / 4, 256, 0, s>>>(a);
    else if (d <= 4096) norm_grad_kernel<1, VEC, false><<<n, threads_for(d, 1), 0, s>>>(a);
    else if (d <= 8192) norm_grad_kernel<2, VEC, false><<<n, threads_for(d, 2), 0, s>>>(a);
    else if (d <= 16384) norm_grad_kernel<4, VEC, false><<<n, threads_for(d, 4), 0, s>>>(a);
    else norm_grad_wide_kernel<VEC><<<n, 512, 0, s>>>(a);
}

}  // namespace

gptq_status norm_launch(const NormArgs& a, hipStream_t s) {
    const bool vec = a.d % 8 == 0 && rows_on_16(a.X, a.x_dt, a.ld_x) && rows_on_16(a.B, a.b_dt, a.ld_b) &&
                     rows_on_16(a.H, a.h_dt, a.ld_h) && rows_on_16(a.Y, a.y_dt, a.ld_y) && rows_on_16(a.weight, a.v_dt, 0) &&
                     rows_on_16(a.bias, a.v_dt, 0) && rows_on_16(a.post, a.v_dt, 0) && rows_on_16(a.gate, a.v_dt, a.ld_gate);
    if (vec) launch_norm<true>(a, s);
    else launch_norm<false>(a, s);
    GPTQ_LAUNCH_CHECK();
    return GPTQ_OK;
}

size_t norm_grad_ws(int64_t n_tok, int64_t d) {
    return (size_t)grad_parts(n_tok, d) * N_VEC * (size_t)(ceil_div(d, 8) * 8) * sizeof(float);
}

gptq_status norm_grad_launch(NormGradArgs a, float* d_weight, float* d_bias, float* d_post, float* d_gate, hipStream_t s) {
    const int64_t d = a.f.d;
    const bool vec = d % 8 == 0 && rows_on_16(a.dY, a.dy_dt, a.ld_dy) && rows_on_16(a.H, a.h_dt, a.ld_h) &&
                     rows_on_16(a.f.B, a.f.b_dt, a.f.ld_b) && rows_on_16(a.dH, a.h_dt, a.ld_dh) &&
                     rows_on_16(a.dX, a.h_dt, a.ld_dx) && rows_on_16(a.dB, a.f.b_dt, a.ld_db) &&
                     rows_on_16(a.f.weight, a.f.v_dt, 0) && rows_on_16(a.f.post, a.f.v_dt, 0) &&
                     rows_on_16(a.f.gate, a.f.v_dt, a.f.ld_gate) && rows_on_16(a.d_gate_rows, a.f.v_dt, a.ld_dgate);
    float* outs[N_VEC] = {d_weight, d_bias, d_post, d_gate};
    float* o[N_VEC] = {nullptr, nullptr, nullptr, nullptr};
    a.n_slots = 0;
    a.ld_part = ceil_div(d, 8) * 8;
    for (int k = 0; k < N_VEC; ++k) {
        a.slot[k] = outs[k] ? a.n_slots : -1;
        if (outs[k]) o[a.n_slots++] = outs[k];
    }
    if (a.f.n_tok > 0) {
        if (vec) launch_grad<true>(a, s);
        else launch_grad<false>(a, s);
        GPTQ_LAUNCH_CHECK();
    }
    if (a.n_slots) {       // without tokens: zeros
        norm_join_kernel<<<dim3((unsigned)ceil_div(d, 64), (unsigned)a.n_slots), 1024, 0, s>>>(
            a.parts, grad_parts(a.f.n_tok, d), a.n_slots, a.ld_part, d, o[0], o[1], o[2], o[3]);
        GPTQ_LAUNCH_CHECK();
    }
    return GPTQ_OK;
}

}  // namespace gptq
