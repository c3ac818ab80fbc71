// Norms around a block and their gradient (include/gptq.h, gptq_residual_norm
// and gptq_residual_norm_backward).
//
// A row is read once into registers, by one wave where it is short and by a
// workgroup otherwise, and everything about it is computed from there: no
// value is read twice but by rows of more than 16384 values, with float32 ones and of
// gradients 8192 (wide kernels).
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
// Eight neighbouring values of a row by a lane, wherever the row starts (wide
// accesses need no alignment here).  Of rows of EIGHTS every lane has its own; of
// others the last lane has the row's last eight, of which it leaves the first
// (`twice`), the lane before's too, out of sums and out of what it stores: 8000 rows
// of 5118 bf16 101 us (5120: 74), 30 of 15101 14 (70 with single elements in every
// lane).  TINY: fewer than eight, one by one.
// ---------------------------------------------------------------------------
enum Width { EIGHTS, OTHER, TINY };
template <bool NARROW = false>
struct Raw8 {
    uint32_t w[NARROW ? 4 : 8];           // NARROW: eight values of 16 bits in a row
};
using Piece = Raw8<>;

__device__ __forceinline__ int column(int v, int T, int t) { return (v * T + t) * 8; }
// Where a lane's eight start, and how many of them are the lane before's.
template <Width D>
__device__ __forceinline__ int start(int c, int d) { return D == OTHER ? min(c, d - 8) : c; }
template <Width D>
__device__ __forceinline__ int twice(int v, int T, int t, int d) {
    const int c = column(v, T, t);
    return c < d ? c - start<D>(c, d) : 0;
}

// Where a row starts: the same for all its lanes.
template <class P>
__device__ __forceinline__ P* row_at(P* p, gptq_dtype dt, int64_t elements) {
    using Byte = std::conditional_t<std::is_const_v<P>, const char, char>;
    return (P*)((Byte*)p + elements * (dt == GPTQ_F32 ? 4 : 2));
}

template <Width D, bool NARROW>
__device__ __forceinline__ Raw8<NARROW> load_as(const void* row, gptq_dtype dt, int v, int T, int t, int d) {
    const bool wide = !NARROW && dt == GPTQ_F32;
    Raw8<NARROW> r;
#pragma unroll
    for (int e = 0; e < (NARROW ? 4 : 8); ++e) r.w[e] = 0u;
    const int c = column(v, T, t);
    if (c >= d) return r;
    if constexpr (D == TINY) {
#pragma unroll
        for (int e = 0; e < 7; ++e) {
            if (e >= d) continue;
            if (!wide) r.w[e >> 1] |= (uint32_t)((const uint16_t*)row)[e] << 16 * (e & 1);
            else if constexpr (!NARROW) r.w[e] = ((const uint32_t*)row)[e];
        }
    } else {
        const u32x4_any_t* q = (const u32x4_any_t*)((const char*)row + (uint32_t)start<D>(c, d) * (wide ? 4u : 2u));
        const u32x4_any_t a = q[0];
        r.w[0] = a.x; r.w[1] = a.y; r.w[2] = a.z; r.w[3] = a.w;
        if constexpr (!NARROW) {
            if (wide) {
                const u32x4_any_t b = q[1];
                r.w[4] = b.x; r.w[5] = b.y; r.w[6] = b.z; r.w[7] = b.w;
            }
        }
    }
    return r;
}
template <Width D>
__device__ __forceinline__ Piece load(const void* row, gptq_dtype dt, int v, int T, int t, int d) {
    return load_as<D, false>(row, dt, v, T, t, d);
}

template <bool NARROW>
__device__ __forceinline__ void values(const Raw8<NARROW>& r, gptq_dtype dt, float (&x)[8]) {
    const auto half = [&](int e) { return r.w[e >> 1] >> (16 * (e & 1)) & 0xFFFFu; };
    if constexpr (!NARROW) {
        if (dt == GPTQ_F32) {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = __uint_as_float(r.w[e]);
            return;
        }
    }
    if (dt == GPTQ_BF16) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = H16<true>::to_f32((uint16_t)half(e));
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = H16<false>::to_f32((uint16_t)half(e));
    }
}

// The last n (1 .. 7) of eight words or halves of words: four, two and one of them.
template <class E, class E2, class E4, class W>
__device__ __forceinline__ void store_last(E* p, int n, const W& at) {
    if (n & 4) *(E4*)(p + 4) = at.four();
    const int to = n & 4 ? 0 : 4;
    if (n & 2) *(E2*)(p + to + 2) = at.two(to);
    if (n & 1) p[to + (n & 2 ? 1 : 3)] = at.one(to, n & 2);
}
struct Words {
    f32x4_t lo, hi;                       // by value: selected addresses would put the eight into scratch
    __device__ f32x4_any_t four() const { return hi; }
    __device__ f32x2_any_t two(int to) const { const f32x4_t q = to ? hi : lo; return f32x2_any_t{q.z, q.w}; }
    __device__ float one(int to, int two) const { const f32x4_t q = to ? hi : lo; return two ? q.y : q.w; }
};
struct Halves {
    u32x4_t w;
    __device__ u32x2_any_t four() const { return u32x2_any_t{w.z, w.w}; }
    __device__ u32_any_t two(int to) const { return to ? w.w : w.y; }
    __device__ uint16_t one(int to, int two) const { return (uint16_t)((to ? (two ? w.z : w.w) : (two ? w.x : w.y)) >> 16); }
};

// The lane's own of eight values.
template <Width D>
__device__ __forceinline__ void store(void* row, gptq_dtype dt, int v, int T, int t, int d, const float (&x)[8]) {
    const int c = column(v, T, t);
    if (c >= d) return;
    if constexpr (D == TINY) {
#pragma unroll
        for (int e = 0; e < 7; ++e) {
            if (e >= d) continue;
            if (dt == GPTQ_F32) ((float*)row)[e] = x[e];
            else ((uint16_t*)row)[e] = (uint16_t)(dt == GPTQ_BF16 ? H16<true>::pack(x[e], 0.f) : H16<false>::pack(x[e], 0.f));
        }
        return;
    }
    const int n = 8 - twice<D>(v, T, t, d);
    char* p = (char*)row + (uint32_t)start<D>(c, d) * (dt == GPTQ_F32 ? 4u : 2u);
    if (dt == GPTQ_F32) {
        if (D != OTHER || n == 8) {
            ((f32x4_any_t*)p)[0] = f32x4_any_t{x[0], x[1], x[2], x[3]};
            ((f32x4_any_t*)p)[1] = f32x4_any_t{x[4], x[5], x[6], x[7]};
        } else {
            store_last<float, f32x2_any_t, f32x4_any_t>((float*)p, n, Words{{x[0], x[1], x[2], x[3]}, {x[4], x[5], x[6], x[7]}});
        }
        return;
    }
    u32x4_t w;
    if (dt == GPTQ_BF16)
        w = u32x4_t{H16<true>::pack(x[0], x[1]), H16<true>::pack(x[2], x[3]), H16<true>::pack(x[4], x[5]), H16<true>::pack(x[6], x[7])};
    else
        w = u32x4_t{H16<false>::pack(x[0], x[1]), H16<false>::pack(x[2], x[3]), H16<false>::pack(x[4], x[5]), H16<false>::pack(x[6], x[7])};
    if (D != OTHER || n == 8) *(u32x4_any_t*)p = w;
    else store_last<uint16_t, u32_any_t, u32x2_any_t>((uint16_t*)p, n, Halves{w});
}

// A vector of d values, or `none` of them.
template <Width D>
__device__ __forceinline__ void vector(const void* p, gptq_dtype dt, int v, int T, int t, int d, float none, float (&x)[8]) {
    if (p) {
        values(load<D>(p, dt, v, T, t, d), dt, x);
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

// A row's sum of squares and, for a layer norm, its sum.
template <bool LAYER>
constexpr int STATS = LAYER ? 2 : 1;
template <Width D, bool LAYER>
__device__ __forceinline__ void add_stats(const float (&x)[8], int twice, double (&s)[STATS<LAYER>]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const double q = (double)(D != OTHER || e >= twice ? x[e] : 0.0f);
        s[0] = fma(q, q, s[0]);
        if constexpr (LAYER) s[1] += q;
    }
}
// Mean (0 of an rms norm) and reciprocal deviation from a row's sum and sum of squares.
struct Stat {
    float mean, rstd;
};
template <bool LAYER>
__device__ __forceinline__ Stat stat(const NormArgs& a, double sq, double sum) {
    const double m = LAYER ? sum * a.inv_d : 0.0;
    const double var = sq * a.inv_d - m * m, x = (var < 0.0 ? 0.0 : var) + (double)a.eps;        // a NaN stays one
    // the hardware's estimate and one step of Newton's: far beyond float32
    const double r = __builtin_amdgcn_rsq(x);
    const bool inside = x > 0.0 && x < __builtin_inf();
    return Stat{(float)m, (float)(inside ? r * fma(-0.5 * x * r, r, 1.5) : r)};
}

// One piece of h = scale x + gate p from x in h, p the block's output (here to be
// normalised).
template <Width D>
__device__ __forceinline__ void stream_value(const NormArgs& a, int64_t row, int v, int T, int t, Stat sb, float (&p)[8],
                                             float (&h)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] *= a.scale;
    if (!a.B) return;
    if (a.post) {
        float w[8];
        vector<D>(a.post, a.v_dt, v, T, t, a.d, 1.0f, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) p[e] = (p[e] - sb.mean) * sb.rstd * w[e];
    }
    if (a.gate) {
        float g[8];
        values(load<D>(row_at(a.gate, a.v_dt, row * a.ld_gate), a.v_dt, v, T, t, a.d), a.v_dt, g);
#pragma unroll
        for (int e = 0; e < 8; ++e) h[e] = fmaf(g[e], p[e], h[e]);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) h[e] += p[e];
    }
}

template <Width D>
__device__ __forceinline__ void write_y(const NormArgs& a, int64_t row, int v, int T, int t, Stat s, const float (&h)[8]) {
    float w[8], c[8];
    vector<D>(a.weight, a.v_dt, v, T, t, a.d, 1.0f, w);
    vector<D>(a.bias, a.v_dt, v, T, t, a.d, 0.0f, c);
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = fmaf((h[e] - s.mean) * s.rstd, w[e], c[e]);
    store<D>(row_at(a.Y, a.y_dt, row * a.ld_y), a.y_dt, v, T, t, a.d, w);
}

// A workgroup (a wave) takes every ROWS-th row and asks for the next one before it
// works on its own.  Bound by memory: 8000 rows of 5120 bf16, two norms, stream and
// norm written, 76 us (4.3 TB/s; a copy has 5.1), with a float32 stream and output of
// the block 116 (4.9); one token 2.9, a launch.  Lanes past the row's end read zeros,
// weights too, so that their values are zeros throughout and add nothing to sums.
template <int V, Width D, bool WAVE, bool LAYER, bool NARROW = false>
__global__ __launch_bounds__(WAVE ? 256 : V == 1 ? 1024 : 512) void norm_kernel(NormArgs a) {
    constexpr int K = STATS<LAYER>;
    __shared__ Sums<2> lds;
    const int T = WAVE ? 64 : blockDim.x, t = WAVE ? threadIdx.x & 63 : threadIdx.x;
    const int64_t first = WAVE ? (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)) : blockIdx.x;
    const int64_t rows = WAVE ? (int64_t)gridDim.x * 4 : gridDim.x;
    if (WAVE && first >= a.n_tok) return;
    Raw8<NARROW> x[V], b[V];
    const auto ask = [&](int64_t row) {
        const void *xr = row_at(a.X, a.x_dt, row * a.ld_x), *br = row_at(a.B, a.b_dt, row * a.ld_b);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if constexpr (NARROW) {
                x[v] = load_as<D, true>(xr, a.x_dt, v, T, t, a.d);
                if (a.B) b[v] = load_as<D, true>(br, a.b_dt, v, T, t, a.d);
            } else {
                x[v] = load<D>(xr, a.x_dt, v, T, t, a.d);
                if (a.B) b[v] = load<D>(br, a.b_dt, v, T, t, a.d);
            }
        }
    };
    ask(first);
    int turn = 0;
    for (int64_t row = first; row < a.n_tok; row += rows) {
        float h[V][8], p[V][8];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if (a.B) values(b[v], a.b_dt, p[v]);
            values(x[v], a.x_dt, h[v]);
        }
        if (row + rows < a.n_tok) ask(row + rows);
        Stat sb{0.f, 0.f};
        if (a.post) {
            double s[K] = {};
#pragma unroll
            for (int v = 0; v < V; ++v) add_stats<D, LAYER>(p[v], twice<D>(v, T, t, a.d), s);
            row_sums<WAVE, K, 2>(s, lds, turn);
            sb = stat<LAYER>(a, s[0], s[K - 1]);
        }
        double s[K] = {};
#pragma unroll
        for (int v = 0; v < V; ++v) {
            stream_value<D>(a, row, v, T, t, sb, p[v], h[v]);
            if (a.H) store<D>(row_at(a.H, a.h_dt, row * a.ld_h), a.h_dt, v, T, t, a.d, h[v]);
            add_stats<D, LAYER>(h[v], twice<D>(v, T, t, a.d), s);
        }
        if (!a.Y) continue;
        row_sums<WAVE, K, 2>(s, lds, turn);
        const Stat sh = stat<LAYER>(a, s[0], s[K - 1]);
#pragma unroll
        for (int v = 0; v < V; ++v) write_y<D>(a, row, v, T, t, sh, h[v]);
    }
}

// Rows that registers do not hold: sums in one pass over them, values in the next
// (from the caches: 2048 x 20000 bf16 112 us, 2.9 TB/s of the bytes that it must move,
// with a float32 stream and output of the block 165, 3.5 TB/s).
template <Width D, bool LAYER>
__global__ __launch_bounds__(1024) void norm_wide_kernel(NormArgs a) {
    constexpr int K = STATS<LAYER>;
    __shared__ Sums<2> lds;
    const int T = blockDim.x, t = threadIdx.x;
    const int64_t row = blockIdx.x;
    const int n = (int)((a.d + 8 * T - 1) / (8 * T));
    int turn = 0;
    Stat sb{0.f, 0.f};
    if (a.post) {
        double s[K] = {};
        for (int v = 0; v < n; ++v) {
            float p[8];
            values(load<D>(row_at(a.B, a.b_dt, row * a.ld_b), a.b_dt, v, T, t, a.d), a.b_dt, p);
            add_stats<D, LAYER>(p, twice<D>(v, T, t, a.d), s);
        }
        row_sums<false, K, 2>(s, lds, turn);
        sb = stat<LAYER>(a, s[0], s[K - 1]);
    }
    const auto value = [&](int v, float (&h)[8]) {
        float p[8];
        values(load<D>(row_at(a.X, a.x_dt, row * a.ld_x), a.x_dt, v, T, t, a.d), a.x_dt, h);
        if (a.B) values(load<D>(row_at(a.B, a.b_dt, row * a.ld_b), a.b_dt, v, T, t, a.d), a.b_dt, p);
        stream_value<D>(a, row, v, T, t, sb, p, h);
    };
    Stat sh{0.f, 0.f};
    if (a.Y) {
        double s[K] = {};
        for (int v = 0; v < n; ++v) {
            float h[8];
            value(v, h);
            add_stats<D, LAYER>(h, twice<D>(v, T, t, a.d), s);
        }
        row_sums<false, K, 2>(s, lds, turn);
        sh = stat<LAYER>(a, s[0], s[K - 1]);
    }
    for (int v = 0; v < n; ++v) {
        float h[8];
        value(v, h);
        if (a.H) store<D>(row_at(a.H, a.h_dt, row * a.ld_h), a.h_dt, v, T, t, a.d, h);      // may be X: its values are read
        if (a.Y) write_y<D>(a, row, v, T, t, sh, h);
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
// call gives the same bits.  The sums' registers leave a compute unit eight waves,
// which bound it: 8192 x 4096 with a float32 stream 165 us (3.7 TB/s), 16 bits 115;
// 500 x 768 8.9 and 6 for the parts.
// ---------------------------------------------------------------------------
enum Vec : int { V_WEIGHT = 0, V_BIAS, V_POST, V_GATE, N_VEC };

__device__ __forceinline__ float through(float t, float n, float r, float mt, float mtn) { return r * (t - mt - n * mtn); }

// What one row's first round of sums is taken over.
struct RowSums {
    Stat h, b;
    float mt, mtn;
};
// of h^2, t h, b^2, and for layer norms of h, t, b
template <bool LAYER>
constexpr int FIRST = LAYER ? 6 : 3;
template <bool LAYER>
__device__ __forceinline__ RowSums first_round(const NormGradArgs& a, const double (&s)[FIRST<LAYER>]) {
    constexpr int L = LAYER ? 3 : 0;
    RowSums r;
    r.h = stat<LAYER>(a.f, s[0], s[L]);
    r.b = a.f.post ? stat<LAYER>(a.f, s[2], s[L + 2]) : Stat{0.f, 0.f};
    r.mt = LAYER ? (float)(s[L + 1] * a.f.inv_d) : 0.0f;
    r.mtn = (float)((LAYER ? s[1] - (double)r.h.mean * s[L + 1] : s[1]) * (double)r.h.rstd * a.f.inv_d);
    return r;
}

template <Width D, bool LAYER>
__device__ __forceinline__ void first_sums(const NormGradArgs& a, const float (&h)[8], const float (&dy)[8], const float (&b)[8],
                                           int v, int T, int t, double (&s)[FIRST<LAYER>]) {
    float w[8];
    vector<D>(a.f.weight, a.f.v_dt, v, T, t, a.f.d, 1.0f, w);
    const int skip = twice<D>(v, T, t, a.f.d);
    const auto own = [&](int e, float q) { return (double)(D != OTHER || e >= skip ? q : 0.0f); };
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const double x = own(e, h[e]), g = own(e, dy[e] * w[e]);       // both 0 past the end
        s[0] = fma(x, x, s[0]);
        s[1] = fma(g, x, s[1]);
        if constexpr (LAYER) {
            s[3] += x;
            s[4] += g;
        }
    }
    if (!a.f.post) return;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const double x = own(e, b[e]);
        s[2] = fma(x, x, s[2]);
        if constexpr (LAYER) s[5] += x;
    }
}

// Of one piece: the gradient of the stream (also stored for x), the terms of
// the vectors' gradients, and what the output's gradient is before its norm,
// with the output's normalised values.  In: h, dy, b, dH; out: q in g and nb in b.
template <Width D>
__device__ __forceinline__ void stream_gradient(const NormGradArgs& a, int64_t row, int v, int T, int t, const RowSums& r,
                                                const float (&h)[8], const float (&dy)[8], float (&b)[8], float (&g)[8],
                                                float (&sum)[N_VEC][8]) {
    float w[8];
    vector<D>(a.f.weight, a.f.v_dt, v, T, t, a.f.d, 1.0f, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float n = (h[e] - r.h.mean) * r.h.rstd;
        const float back = through(dy[e] * w[e], n, r.h.rstd, r.mt, r.mtn);
        sum[V_WEIGHT][e] = fmaf(dy[e], n, sum[V_WEIGHT][e]);
        sum[V_BIAS][e] += dy[e];
        g[e] = a.dH ? back + g[e] : back;
    }
    if (a.dX) {
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = g[e] * a.f.scale;
        store<D>(row_at(a.dX, a.h_dt, row * a.ld_dx), a.h_dt, v, T, t, a.f.d, w);
    }
    if (!a.has_b) return;
    vector<D>(a.f.post, a.f.v_dt, v, T, t, a.f.d, 1.0f, w);
    if (a.f.post) {
#pragma unroll
        for (int e = 0; e < 8; ++e) b[e] = (b[e] - r.b.mean) * r.b.rstd;
    }
    if (a.f.gate) {
        float gate[8], each[8];
        values(load<D>(row_at(a.f.gate, a.f.v_dt, row * a.f.ld_gate), a.f.v_dt, v, T, t, a.f.d), a.f.v_dt, gate);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            each[e] = g[e] * (b[e] * w[e]);
            sum[V_GATE][e] += each[e];
            g[e] *= gate[e];
        }
        if (a.d_gate_rows) store<D>(row_at(a.d_gate_rows, a.f.v_dt, row * a.ld_dgate), a.f.v_dt, v, T, t, a.f.d, each);
    }
    if (a.f.post) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            sum[V_POST][e] = fmaf(g[e], b[e], sum[V_POST][e]);
            g[e] *= w[e];
        }
    }
}

// of q nb and, for layer norms, q (0 past the end, where post_weight reads as 0)
template <Width D, bool LAYER>
__device__ __forceinline__ void second_sums(const float (&q)[8], const float (&nb)[8], int twice, double (&s)[STATS<LAYER>]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const bool own = D != OTHER || e >= twice;
        const double x = (double)(own ? q[e] : 0.0f);
        s[0] = fma(x, (double)(own ? nb[e] : 0.0f), s[0]);
        if constexpr (LAYER) s[1] += x;
    }
}

template <Width D>
__device__ __forceinline__ void write_db(const NormGradArgs& a, int64_t row, int v, int T, int t, Stat sb, float mq, float mqn,
                                         float (&q)[8], const float (&nb)[8]) {
    if (a.f.post) {
#pragma unroll
        for (int e = 0; e < 8; ++e) q[e] = through(q[e], nb[e], sb.rstd, mq, mqn);
    }
    store<D>(row_at(a.dB, a.f.b_dt, row * a.ld_db), a.f.b_dt, v, T, t, a.f.d, q);
}

// One part's sums of vector k, if it is asked for.
template <Width D>
__device__ __forceinline__ void write_part(const NormGradArgs& a, int64_t part, int k, int v, int T, int t, const float (&x)[8]) {
    if (a.slot[k] < 0) return;
    store<D>(row_at(a.parts, GPTQ_F32, (part * a.n_slots + a.slot[k]) * a.ld_part), GPTQ_F32, v, T, t, a.f.d, x);
}

template <int V, Width D, bool WAVE, bool LAYER, bool NARROW>
__global__ __launch_bounds__(WAVE ? 256 : 512) void norm_grad_kernel(NormGradArgs a) {
    constexpr int F = FIRST<LAYER>, K = STATS<LAYER>;
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
    Raw8<NARROW> hr[V], yr[V], br[V], gr[V];
    const auto ask = [&](int64_t row) {          // the next row, before this one is worked on
#pragma unroll
        for (int v = 0; v < V; ++v) {
            hr[v] = load_as<D, NARROW>(row_at(a.H, a.h_dt, row * a.ld_h), a.h_dt, v, T, t, a.f.d);
            yr[v] = load_as<D, NARROW>(row_at(a.dY, a.dy_dt, row * a.ld_dy), a.dy_dt, v, T, t, a.f.d);
            if (a.has_b) br[v] = load_as<D, NARROW>(row_at(a.f.B, a.f.b_dt, row * a.f.ld_b), a.f.b_dt, v, T, t, a.f.d);
            if (a.dH) gr[v] = load_as<D, NARROW>(row_at(a.dH, a.h_dt, row * a.ld_dh), a.h_dt, v, T, t, a.f.d);
        }
    };
    if (part < a.f.n_tok) ask(part);
    for (int64_t row = part; row < a.f.n_tok; row += parts) {
        float h[V][8], y[V][8], b[V][8], g[V][8];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            values(hr[v], a.h_dt, h[v]);
            values(yr[v], a.dy_dt, y[v]);
            if (a.has_b) values(br[v], a.f.b_dt, b[v]);
            if (a.dH) values(gr[v], a.h_dt, g[v]);
        }
        if (row + parts < a.f.n_tok) ask(row + parts);
        double s[F] = {};
#pragma unroll
        for (int v = 0; v < V; ++v) first_sums<D, LAYER>(a, h[v], y[v], b[v], v, T, t, s);
        row_sums<WAVE, F, 6>(s, lds, turn);
        const RowSums r = first_round<LAYER>(a, s);
#pragma unroll
        for (int v = 0; v < V; ++v) stream_gradient<D>(a, row, v, T, t, r, h[v], y[v], b[v], g[v], sum[v]);
        if (!a.dB) continue;
        float mq = 0.f, mqn = 0.f;
        if (a.f.post) {
            double u[K] = {};
#pragma unroll
            for (int v = 0; v < V; ++v) second_sums<D, LAYER>(g[v], b[v], twice<D>(v, T, t, a.f.d), u);
            row_sums<WAVE, K, 6>(u, lds, turn);
            mq = LAYER ? (float)(u[K - 1] * a.f.inv_d) : 0.0f;
            mqn = (float)(u[0] * a.f.inv_d);
        }
#pragma unroll
        for (int v = 0; v < V; ++v) write_db<D>(a, row, v, T, t, r.b, mq, mqn, g[v], b[v]);
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int k = 0; k < N_VEC; ++k) write_part<D>(a, part, k, v, T, t, sum[v][k]);
}

// Rows that registers do not hold: each pass over them reads them again, and
// the vectors' sums live in the part itself (every value a lane's own).  2048 x
// 12288 bf16 177 us; in registers, of which half went to scratch, 397.
template <Width D, bool LAYER>
__global__ __launch_bounds__(512) void norm_grad_wide_kernel(NormGradArgs a) {
    constexpr int F = FIRST<LAYER>, K = STATS<LAYER>;
    __shared__ Sums<6> lds;
    const int T = blockDim.x, t = threadIdx.x;
    const int64_t part = blockIdx.x;
    const int n = (int)((a.f.d + 8 * T - 1) / (8 * T));
    int turn = 0;
    bool first = true;
    for (int64_t row = part; row < a.f.n_tok; row += gridDim.x) {
        float h[8], y[8], b[8], g[8];
        const auto read = [&](int v) {
            values(load<D>(row_at(a.H, a.h_dt, row * a.ld_h), a.h_dt, v, T, t, a.f.d), a.h_dt, h);
            values(load<D>(row_at(a.dY, a.dy_dt, row * a.ld_dy), a.dy_dt, v, T, t, a.f.d), a.dy_dt, y);
            if (a.has_b) values(load<D>(row_at(a.f.B, a.f.b_dt, row * a.f.ld_b), a.f.b_dt, v, T, t, a.f.d), a.f.b_dt, b);
            if (a.dH) values(load<D>(row_at(a.dH, a.h_dt, row * a.ld_dh), a.h_dt, v, T, t, a.f.d), a.h_dt, g);
        };
        double s[F] = {};
        for (int v = 0; v < n; ++v) {
            read(v);
            first_sums<D, LAYER>(a, h, y, b, v, T, t, s);
        }
        row_sums<false, F, 6>(s, lds, turn);
        const RowSums r = first_round<LAYER>(a, s);
        double u[K] = {};
        float mq = 0.f, mqn = 0.f;
        // the output's gradient needs the stream's first: a pass that stores
        // nothing, where there is a norm to go through
        NormGradArgs quiet = a;
        quiet.dX = nullptr;
        quiet.d_gate_rows = nullptr;
        if (a.dB && a.f.post) {
            for (int v = 0; v < n; ++v) {
                float sum[N_VEC][8];
#pragma unroll
                for (int k = 0; k < N_VEC; ++k)
#pragma unroll
                    for (int e = 0; e < 8; ++e) sum[k][e] = 0.0f;
                read(v);
                stream_gradient<D>(quiet, row, v, T, t, r, h, y, b, g, sum);
                second_sums<D, LAYER>(g, b, twice<D>(v, T, t, a.f.d), u);
            }
            row_sums<false, K, 6>(u, lds, turn);
            mq = LAYER ? (float)(u[K - 1] * a.f.inv_d) : 0.0f;
            mqn = (float)(u[0] * a.f.inv_d);
        }
        for (int v = 0; v < n; ++v) {
            float sum[N_VEC][8];
#pragma unroll
            for (int k = 0; k < N_VEC; ++k) {
#pragma unroll
                for (int e = 0; e < 8; ++e) sum[k][e] = 0.0f;
                if (!first && a.slot[k] >= 0)
                    values(load<D>(row_at(a.parts, GPTQ_F32, (part * a.n_slots + a.slot[k]) * a.ld_part), GPTQ_F32, v, T, t, a.f.d), GPTQ_F32, sum[k]);
            }
            read(v);
            stream_gradient<D>(a, row, v, T, t, r, h, y, b, g, sum);
            if (a.dB) write_db<D>(a, row, v, T, t, r.b, mq, mqn, g, b);
#pragma unroll
            for (int k = 0; k < N_VEC; ++k) write_part<D>(a, part, k, v, T, t, sum[k]);
        }
        first = false;
    }
}

// out[slot][c] = the parts' sums: C columns by 1024 / C shares of the parts, of
// which a thread asks for eight at once.  With many parts (4096 of 89 columns: 15
// us by 64 columns, 10 by 16) a workgroup takes fewer columns.
template <int C>
__global__ __launch_bounds__(1024) void norm_join_kernel(const float* parts, int64_t n_parts, int n_slots, int64_t ld, int64_t d,
                                                         float* o0, float* o1, float* o2, float* o3) {
    constexpr int S = 1024 / C;
    __shared__ double lds[S][C];
    const int lane = threadIdx.x % C, share = threadIdx.x / C;
    const int64_t c = (int64_t)blockIdx.x * C + lane;
    const int slot = blockIdx.y;
    double s = 0.0;
    if (c < d) {
        const float* p = parts + slot * ld + c;
        const int64_t end = n_parts * (share + 1) / S;
        for (int64_t i = n_parts * share / S; i < end; i += 8) {
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = p[min(i + e, end - 1) * n_slots * ld];
#pragma unroll
            for (int e = 0; e < 8; ++e) s += i + e < end ? (double)v[e] : 0.0;
        }
    }
    lds[share][lane] = s;
    __syncthreads();
    if (share == 0 && c < d) {
#pragma unroll 8
        for (int k = 1; k < S; ++k) s += lds[k][lane];
        float* o = slot == 0 ? o0 : slot == 1 ? o1 : slot == 2 ? o2 : o3;
        o[c] = (float)s;
    }
}

// Threads of a workgroup for rows of d values, eight or sixteen or 32 a lane.
unsigned threads_for(int64_t d, int pieces) { return (unsigned)(ceil_div(ceil_div(d, 8 * pieces), 64) * 64); }

// Rows of 8193 to 16384 values in registers, 32 a lane, where all are of 16 bits
// (4096 rows with two norms, of 8200 97 us against 105 in passes, of 11008 112 and 135,
// of 16384 137 and 150); float32 ones leave the registers (4096 x 8200 float32 stream
// 145 against 106 in passes, x 16384 219 and 179).
template <Width D, bool LAYER, bool NARROW>
void launch_norm(const NormArgs& a, hipStream_t s) {
    // as many workgroups as the chip holds at once (six waves a SIMD, by their registers)
    const auto groups = [&](int64_t rows, unsigned threads) { return (unsigned)std::min<int64_t>(rows, 256 * (1536 / threads)); };
    const unsigned four = groups(ceil_div(a.n_tok, 4), 256), t1 = threads_for(a.d, 1), t4 = threads_for(a.d, 4);
    if (D == TINY || a.d <= 512) norm_kernel<1, D, true, LAYER, NARROW><<<four, 256, 0, s>>>(a);
    else if constexpr (D == TINY) return;
    else if (a.d <= 1024) norm_kernel<2, D, true, LAYER, NARROW><<<four, 256, 0, s>>>(a);
    else if (a.d <= 8192) norm_kernel<1, D, false, LAYER, NARROW><<<groups(a.n_tok, t1), t1, 0, s>>>(a);
    else if (!NARROW || a.d > 16384) norm_wide_kernel<D, LAYER><<<(unsigned)a.n_tok, 1024, 0, s>>>(a);
    else if constexpr (NARROW) norm_kernel<4, D, false, LAYER, true><<<groups(a.n_tok, t4), t4, 0, s>>>(a);
}

// Parts of the sums over tokens, and with them workgroups of the gradient.
int64_t grad_parts(int64_t n_tok, int64_t d) {
    if (d <= 1024) return std::min<int64_t>(ceil_div(n_tok, 4), 1024) * 4;      // a wave's rows
    return std::min<int64_t>(n_tok, 512);
}

// Sixteen values a lane where registers hold them (16-bit rows: two workgroups of
// four waves a compute unit do better than one of eight, 8192 x 4096 115 us against
// 127).  With float32 rows they do not, and some go to memory: eight a lane are better
// as long as a workgroup has them (8192 x 4096 167 us, sixteen 237), and past that
// sixteen are still better than passes (4096 x 5120 float32 stream 198 against 251,
// x 8192 233 and 338).
template <Width D, bool LAYER, bool NARROW>
void launch_grad(const NormGradArgs& a, hipStream_t s) {
    const int64_t d = a.f.d;
    const unsigned n = (unsigned)grad_parts(a.f.n_tok, d);
    if (D == TINY || d <= 512) norm_grad_kernel<1, D, true, LAYER, NARROW><<<n / 4, 256, 0, s>>>(a);
    else if constexpr (D == TINY) return;
    else if (d <= 1024) norm_grad_kernel<2, D, true, LAYER, NARROW><<<n / 4, 256, 0, s>>>(a);
    else if (d <= (NARROW ? 2048 : 4096)) norm_grad_kernel<1, D, false, LAYER, NARROW><<<n, threads_for(d, 1), 0, s>>>(a);
    else if (d <= 8192) norm_grad_kernel<2, D, false, LAYER, NARROW><<<n, threads_for(d, 2), 0, s>>>(a);
    else norm_grad_wide_kernel<D, LAYER><<<n, 512, 0, s>>>(a);
}

}  // namespace

gptq_status norm_launch(const NormArgs& a, hipStream_t s) {
    const bool narrow = a.x_dt != GPTQ_F32 && (!a.B || a.b_dt != GPTQ_F32);
    const auto go = [&](auto layer) {
        constexpr bool L = decltype(layer)::value;
        if (a.d < 8) launch_norm<TINY, L, false>(a, s);
        else if (a.d % 8 == 0) narrow ? launch_norm<EIGHTS, L, true>(a, s) : launch_norm<EIGHTS, L, false>(a, s);
        else narrow ? launch_norm<OTHER, L, true>(a, s) : launch_norm<OTHER, L, false>(a, s);
    };
    a.layer ? go(std::true_type{}) : go(std::false_type{});
    GPTQ_LAUNCH_CHECK();
    return GPTQ_OK;
}

size_t norm_grad_ws(int64_t n_tok, int64_t d) {
    return (size_t)grad_parts(n_tok, d) * N_VEC * (size_t)(ceil_div(d, 8) * 8) * sizeof(float);
}

gptq_status norm_grad_launch(NormGradArgs a, float* d_weight, float* d_bias, float* d_post, float* d_gate, hipStream_t s) {
    const int64_t d = a.f.d;
    float* outs[N_VEC] = {d_weight, d_bias, d_post, d_gate};
    float* o[N_VEC] = {nullptr, nullptr, nullptr, nullptr};
    a.n_slots = 0;
    a.ld_part = ceil_div(d, 8) * 8;
    for (int k = 0; k < N_VEC; ++k) {
        a.slot[k] = outs[k] ? a.n_slots : -1;
        if (outs[k]) o[a.n_slots++] = outs[k];
    }
    if (a.f.n_tok > 0) {
        const bool narrow = a.h_dt != GPTQ_F32 && a.dy_dt != GPTQ_F32 && (!a.has_b || a.f.b_dt != GPTQ_F32);
        const auto go = [&](auto layer) {
            constexpr bool L = decltype(layer)::value;
            if (d < 8) launch_grad<TINY, L, false>(a, s);
            else if (d % 8 == 0) narrow ? launch_grad<EIGHTS, L, true>(a, s) : launch_grad<EIGHTS, L, false>(a, s);
            else narrow ? launch_grad<OTHER, L, true>(a, s) : launch_grad<OTHER, L, false>(a, s);
        };
        a.f.layer ? go(std::true_type{}) : go(std::false_type{});
        GPTQ_LAUNCH_CHECK();
    }
    if (a.n_slots) {       // without tokens: zeros
        const int64_t n = grad_parts(a.f.n_tok, d);
        const auto join = [&](auto columns) {
            constexpr int C = decltype(columns)::value;
            norm_join_kernel<C><<<dim3((unsigned)ceil_div(d, C), (unsigned)a.n_slots), 1024, 0, s>>>(a.parts, n, a.n_slots, a.ld_part,
                                                                                                     d, o[0], o[1], o[2], o[3]);
        };
        n > 512 ? join(std::integral_constant<int, 16>{}) : join(std::integral_constant<int, 64>{});
        GPTQ_LAUNCH_CHECK();
    }
    return GPTQ_OK;
}

}  // namespace gptq
