// Products with e2m1 weights: Y = X W^T (include/gptq.h, gptq_mx_matmul and
// gptq_mx_matmul_quantized).
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "mx.hpp"

namespace gptq {
namespace {

// Kinds of activations.
enum Act : int { ACT_F32 = GPTQ_F32, ACT_F16 = GPTQ_F16, ACT_BF16 = GPTQ_BF16, ACT_FP8, ACT_FP4 };

struct MatArgs {
    const void* X;         // values, or codes
    const uint8_t* XS;     // scale bytes of the codes
    int64_t n_tok, d_in, ld_x;
    bool aligned;          // X rows start on 16 bytes
    const uint8_t* W;      // codes
    const uint8_t* S;      // scale bytes
    int64_t w_row, s_row;  // bytes per row
    int steps;             // padded 128-column steps
    int full;              // the first of them whose activations are read in whole 16-byte pieces
    int64_t d_out, ld_y;
    float* Y;
    bool y_aligned;        // Y rows start on 16 bytes
};

// ---------------------------------------------------------------------------
// Activations as bfloat16 parts.  A float32 is the sum of three bfloat16 cut
// off its top (8 + 8 + 8 of its 24 bits), a float16 of two: no rounding, and
// no overflow, down to bfloat16's smallest step, 2^-133 (float32 values below
// 2^-110 lose what is under it).  The parts below an infinity or NaN are 0.  A
// microscaled value is a bfloat16 as it is (e4m3 from scale byte 3 on).
// (v_mfma_scale_f32_32x32x64_f8f6f4 would take e4m3 codes directly, at twice
// the rate, but with an e4m3 operand it cuts products off some 16 bits below the
// largest one of an instruction: an error of 1e-5 of sum |x w| and more,
// measured, where these sums keep 1e-7.)
//
// Float16 activations enter as they are, with weights as float16, for blocks
// whose scale leaves them in float16's range (byte 104 .. 140: 2^-24 ..
// 6 * 2^13), which those of trained weights do.  A wave that met another block
// (that counted as zeros till then) drops its sums and takes them again from
// the start with activations in two parts.  (Adding the missing blocks alone
// would not do: an infinite activation times the zeros is NaN.)
// ---------------------------------------------------------------------------
template <Act DT>
constexpr int parts_of() { return DT == ACT_F16 ? 2 : DT == ACT_F32 ? 3 : 1; }

__device__ __forceinline__ bool scale_fits_f16(uint32_t byte) { return byte - 104u <= 36u; }
// codes if `keep`, else zeros
__device__ __forceinline__ u32x4_t codes_if(bool keep, u32x4_t w) {
    const uint32_t m = keep ? 0xFFFFFFFFu : 0u;
    return w & u32x4_t{m, m, m, m};
}
// codes that are not all zero
__device__ __forceinline__ bool some(u32x4_t w) { return (w.x | w.y | w.z | w.w) != 0u; }

// Some consecutive activations of a token as they are in memory: N groups of
// eight (N = 4, a block, for e2m1).
template <Act DT, int N = 4>
struct Raw {
    static constexpr int W = DT == ACT_F32 ? 2 * N : DT == ACT_FP8 ? (N + 1) / 2 : DT == ACT_FP4 ? 1 : N;
    u32x4_t w[W];
    uint32_t s;

    // whole: aligned, and every column exists
    template <bool WHOLE>
    __device__ __forceinline__ void load(const MatArgs& a, int64_t t, int64_t k) {
        if constexpr (DT == ACT_FP4) {
            static_assert(N == 4, "whole blocks");
            w[0] = *(const u32x4_t*)((const uint8_t*)a.X + t * a.ld_x + (k >> 1));
            s = a.XS[t * a.s_row + (k >> 5)];
        } else if constexpr (DT == ACT_FP8) {
            const uint8_t* p = (const uint8_t*)a.X + t * a.ld_x + k;
            if constexpr (N == 4) {
                w[0] = *(const u32x4_t*)p;
                w[1] = *(const u32x4_t*)(p + 16);
            } else {
                const u32x2_t v = *(const u32x2_t*)p;
                w[0].x = v.x;
                w[0].y = v.y;
            }
            s = a.XS[t * a.s_row + (k >> 5)];
        } else if constexpr (WHOLE) {
            const u32x4_t* p = (const u32x4_t*)((const char*)a.X + (t * a.ld_x + k) * (DT == ACT_F32 ? 4 : 2));
#pragma unroll
            for (int i = 0; i < W; ++i) w[i] = p[i];
        } else {
            const int n = (int)max((int64_t)0, min((int64_t)(8 * N), a.d_in - k));
            if constexpr (DT == ACT_F32) {
                const uint32_t* p = (const uint32_t*)a.X + t * a.ld_x + k;
#pragma unroll
                for (int i = 0; i < 8 * N; ++i) w[i >> 2][i & 3] = i < n ? p[i] : 0u;
            } else {
                const uint16_t* p = (const uint16_t*)a.X + t * a.ld_x + k;
#pragma unroll
                for (int i = 0; i < 4 * N; ++i) {
                    const uint32_t lo = 2 * i < n ? p[2 * i] : 0, hi = 2 * i + 1 < n ? p[2 * i + 1] : 0;
                    w[i >> 2][i & 3] = lo | hi << 16;
                }
            }
        }
    }

    // Group c as 16-bit values (not for float32).
    __device__ __forceinline__ u32x4_t eight(int c) const {
        if constexpr (DT == ACT_FP4) return fp4x8<true>(w[0][c], mx_scale(s));
        else if constexpr (DT == ACT_FP8) return fp8x8<true>(w[c >> 1][2 * (c & 1)], w[c >> 1][2 * (c & 1) + 1], mx_scale(s));
        else return w[c];
    }
};

// bfloat16 parts of eight float32 values: the top half of each, then that of
// what is left; below an infinity or NaN 0 (ODD: where there may be some, which
// the first part sees: all others are of finite values).
template <int NP, bool ODD>
__device__ __forceinline__ void split(float (&v)[8], u32x4_t (&p)[NP]) {
#pragma unroll
    for (int j = 0; j < NP; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t w[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float& x = v[2 * i + k];
                w[k] = __float_as_uint(x);
                const bool fin = !ODD || j > 0 || (w[k] & 0x7F800000u) != 0x7F800000u;
                x = fin ? x - __uint_as_float(w[k] & 0xFFFF0000u) : 0.0f;
                // a NaN whose top bits are an infinity's keeps a quiet bit
                if (ODD && j == 0 && (w[k] & 0x7FFFFFFFu) > 0x7F800000u) w[k] |= 0x00400000u;
            }
            p[j][i] = __builtin_amdgcn_perm(w[1], w[0], 0x07060302u);
        }
}
// The same of eight float16.
__device__ __forceinline__ void split_f16(u32x4_t h, u32x4_t (&p)[2]) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = H16<false>::to_f32((uint16_t)h[i]);
        v[2 * i + 1] = H16<false>::to_f32((uint16_t)(h[i] >> 16));
    }
    split<2, true>(v, p);
}
// An infinity or NaN among float32 values.
template <int N>
__device__ __forceinline__ bool odd(const Raw<ACT_F32, N>& x) {
    bool any = false;
#pragma unroll
    for (int i = 0; i < 8 * N; ++i) any |= !__builtin_isfinite(__uint_as_float(x.w[i >> 2][i & 3]));
    return any;
}
// ODD: whether float32 values may be infinite or NaN
template <bool ODD, Act DT, int N>
__device__ __forceinline__ void parts(const Raw<DT, N>& x, int c, u32x4_t (&p)[parts_of<DT>()]) {
    if constexpr (DT == ACT_F32) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(x.w[2 * c + (i >> 2)][i & 3]);
        split<3, ODD>(v, p);
    } else if constexpr (DT == ACT_F16) {
        split_f16(x.w[c], p);
    } else {
        p[0] = x.eight(c);
    }
}

// Four neighbouring outputs of a token.
__device__ __forceinline__ void store4(const MatArgs& a, int64_t t, int64_t r, float v0, float v1, float v2, float v3) {
    float* y = a.Y + t * a.ld_y + r;
    if (a.y_aligned && r + 4 <= a.d_out) {
        *(f32x4_t*)y = f32x4_t{v0, v1, v2, v3};
    } else {
        if (r < a.d_out) y[0] = v0;
        if (r + 1 < a.d_out) y[1] = v1;
        if (r + 2 < a.d_out) y[2] = v2;
        if (r + 3 < a.d_out) y[3] = v3;
    }
}

// ---------------------------------------------------------------------------
// Few tokens: a workgroup computes 16 RT weight rows x 16 TT tokens; its waves
// take a share of the 128-column steps each, and their sums meet in LDS.
//
// Such a product is bound by how many bytes are on their way at once, and by
// how they are asked for: a lane's own load of 16 bytes is a request to the
// cache by itself unless its neighbours' continue it, and with a matrix
// instruction's rows on neighbouring lanes none does (13 x 11008 -> 4096
// float16: 43000 requests per compute unit, 19 us).  So each wave brings its
// steps into a ring of LDS slots of its own, four lanes to 64 bytes in a row,
// RING steps ahead, without registers and without a barrier.  Rows there are
// whole (64 bytes of codes, 64 .. 512 of activations), with 16-byte chunk c at
// slot c ^ swizzle(row), so that reads of one chunk of eight rows hit all
// banks.  Reads of tokens and steps past the end fall outside their buffer,
// make no request and give zeros; rows past the end repeat the last one.
//
// v_mfma_f32_16x16x32 with a lane's four k-groups of eight chosen as one block
// of 32 columns: lane l holds row l % 16, block l / 16 of the step (16 bytes
// of codes, one scale), and activations of token l % 16 in the same columns.
// Columns after the last whole 128 (all, where activations do not start on 16
// bytes) come from memory directly.
//
// Measured: one bf16 token, 4096 -> 4096, 4.9 us (an empty launch is 2.6; the
// codes 1.7 at the rate of a copy); 13 float16 tokens, 11008 -> 4096, 9.8 us
// (2.5 TB/s; every compute unit reads all 286 KB of activations, which L2
// hands out at some 20 bytes a clock); 64 bf16 tokens, 4096 -> 4096, 8.1 us.
// ---------------------------------------------------------------------------
constexpr int LDS_BYTES = 160 * 1024;      // of a compute unit

template <Act DT, int RT, int TT>
struct FewTile {
    static constexpr int X_ROW = DT == ACT_F32 ? 512 : DT == ACT_FP8 ? 128 : DT == ACT_FP4 ? 64 : 256;   // bytes of a token
    static constexpr int XS = DT == ACT_FP8 || DT == ACT_FP4 ? TT : 0;                       // 16-row groups of X scales
    static constexpr int W_DMA = RT, X_DMA = TT * X_ROW / 64, DMA = W_DMA + X_DMA + RT + XS;
    static constexpr int S_AT = 1024 * (W_DMA + X_DMA), STAGE = S_AT + 256 * (RT + XS);
    static constexpr int WAVES = 2 * 8 * STAGE <= LDS_BYTES ? 8 : 4;
    static constexpr int RING = LDS_BYTES / (WAVES * STAGE) < 4 ? LDS_BYTES / (WAVES * STAGE) : 4;
    static constexpr int AT = RT * TT < 4 ? RT * TT : 4;                                      // tiles joined at a time
    static constexpr int BYTES = WAVES * (RING * STAGE > 1024 * AT ? RING * STAGE : 1024 * AT);
    static constexpr bool FITS = RING >= 2 && (RING - 1) * DMA < 64;
};
constexpr uint32_t NOWHERE = 1u << 30;     // an offset past every tile's buffer, also with another added

template <Act DT, int RT, int TT, int THREADS = 64 * FewTile<DT, RT, TT>::WAVES>
__global__ __launch_bounds__(THREADS) void mx_few_kernel(MatArgs a) {
    using T = FewTile<DT, RT, TT>;
    constexpr int NP = parts_of<DT>(), CH = T::X_ROW / 16, PER = CH < 16 ? 16 / CH : 1, LOW = CH < 16 ? CH - 1 : 15;
    using Half = std::bool_constant<DT == ACT_F16>;
    extern __shared__ __attribute__((aligned(16))) char lds[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int i16 = lane & 15, g = lane >> 4;
    const int64_t r0 = (int64_t)blockIdx.x * (16 * RT), t0 = (int64_t)blockIdx.y * (16 * TT);
    const int64_t wn = min((int64_t)(16 * RT), a.d_out - r0), xn = min((int64_t)(16 * TT), a.n_tok - t0);
    f32x4_t acc[RT][TT];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < TT; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    struct Step {
        u32x4_t w[RT];
        uint32_t s[RT];
        Raw<DT> x[TT];
    };
    bool left = false;       // float16: a block was left out
    const auto multiply_as = [&](const Step& d, auto half, auto may) {
        constexpr bool HALF = decltype(half)::value, ODD = decltype(may)::value;
        u32x4_t codes[RT];
        uint32_t sc[RT];
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            codes[i] = d.w[i];
            sc[i] = d.s[i];
            if constexpr (HALF) {
                const bool fits = scale_fits_f16(sc[i]);
                left |= !fits && (some(codes[i]) || sc[i] == 255u);
                codes[i] = codes_if(fits, codes[i]);
                if (!fits) sc[i] = 127u;
            }
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            u32x4_t w[RT];
#pragma unroll
            for (int i = 0; i < RT; ++i) w[i] = fp4x8<!HALF>(codes[i][c], mx_scale(sc[i]));
#pragma unroll
            for (int j = 0; j < TT; ++j) {
                if constexpr (HALF) {
#pragma unroll
                    for (int i = 0; i < RT; ++i) acc[i][j] = H16<false>::mfma16(w[i], d.x[j].eight(c), acc[i][j]);
                } else {
                    u32x4_t p[NP];
                    parts<ODD>(d.x[j], c, p);
#pragma unroll
                    for (int q = 0; q < NP; ++q)
#pragma unroll
                        for (int i = 0; i < RT; ++i) acc[i][j] = H16<true>::mfma16(w[i], p[q], acc[i][j]);
                }
            }
        }
    };

    // Float32: one look at a step's values leaves half of the work on their parts
    // (13 tokens 4096 -> 4096 9.3 us, 14.6 with every part looking for itself).
    const auto multiply = [&](const Step& d, auto half) {
        if constexpr (DT == ACT_F32) {
            bool any = false;
#pragma unroll
            for (int j = 0; j < TT; ++j) any |= odd(d.x[j]);
            if (__any(any)) multiply_as(d, half, std::true_type{});
            else multiply_as(d, half, std::false_type{});
        } else {
            multiply_as(d, half, std::true_type{});
        }
    };

    // this wave's whole steps, in a row
    const int first = a.full * wave / T::WAVES, end = a.full * (wave + 1) / T::WAVES;
    if (first < end) {
        constexpr int XB = T::XS ? 1 : DT == ACT_F32 ? 4 : 2;                    // bytes per element of ld_x
        const u32x4_t wb = buffer_of(a.W + r0 * a.w_row, wn * a.w_row), wsb = buffer_of(a.S + r0 * a.s_row, wn * a.s_row);
        const u32x4_t xb = buffer_of((const char*)a.X + t0 * a.ld_x * XB, ((xn - 1) * a.ld_x + (T::XS ? a.ld_x : a.d_in)) * XB);
        const u32x4_t xsb = T::XS ? buffer_of(a.XS + t0 * a.s_row, xn * a.s_row) : wsb;
        uint32_t woff[T::W_DMA], xoff[T::X_DMA], wsoff[RT], xsoff[T::XS ? T::XS : 1];
#pragma unroll
        for (int k = 0; k < RT; ++k) {
            const int r = 16 * k + (lane >> 2);
            woff[k] = (uint32_t)(min((int64_t)r, wn - 1) * a.w_row + 16 * ((lane & 3) ^ (r >> 2 & 3)));
            wsoff[k] = lane < 16 ? (uint32_t)(min((int64_t)(16 * k + lane), wn - 1) * a.s_row) : NOWHERE;
        }
#pragma unroll
        for (int k = 0; k < T::X_DMA; ++k) {
            const int at = 64 * k + lane, t = at / CH, c = at % CH ^ (t / PER & LOW);
            xoff[k] = t < xn ? (uint32_t)(t * a.ld_x * XB + 16 * c) : NOWHERE;
        }
#pragma unroll
        for (int k = 0; k < T::XS; ++k) xsoff[k] = lane < 16 && 16 * k + lane < xn ? (uint32_t)((16 * k + lane) * a.s_row) : NOWHERE;
        const uint32_t base = (uint32_t)(uintptr_t)lds + wave * (T::RING * T::STAGE);
        const auto fetch = [&](int st, int slot) {
            const uint32_t at = base + slot * T::STAGE;
            const bool is = st < end;
            const uint32_t wo = is ? 64u * st : NOWHERE, xo = is ? (uint32_t)T::X_ROW * st : NOWHERE, so = is ? 4u * st : NOWHERE;
#pragma unroll
            for (int k = 0; k < RT; ++k) dma_16(at + 1024 * k, woff[k] + wo, wb);
#pragma unroll
            for (int k = 0; k < T::X_DMA; ++k) dma_16(at + 1024 * (RT + k), xoff[k] + xo, xb);
#pragma unroll
            for (int k = 0; k < RT; ++k) dma_4(at + T::S_AT + 256 * k, wsoff[k] + so, wsb);
#pragma unroll
            for (int k = 0; k < T::XS; ++k) dma_4(at + T::S_AT + 256 * (RT + k), xsoff[k] + so, xsb);
        };
#pragma unroll
        for (int i = 0; i < T::RING; ++i) fetch(first + i, i);
        for (int s0 = first; s0 < end; s0 += T::RING) {
#pragma unroll
            for (int i = 0; i < T::RING; ++i) {
                if (s0 + i < end) {
                    wait_vmem<(T::RING - 1) * T::DMA>();
                    const char* p = lds + wave * (T::RING * T::STAGE) + i * T::STAGE;
                    Step d;
#pragma unroll
                    for (int k = 0; k < RT; ++k) {
                        d.w[k] = *(const u32x4_t*)(p + 1024 * k + 64 * i16 + 16 * (g ^ (i16 >> 2)));
                        d.s[k] = *(const uint8_t*)(p + T::S_AT + 256 * k + 4 * i16 + g);
                    }
#pragma unroll
                    for (int j = 0; j < TT; ++j) {
#pragma unroll
                        for (int e = 0; e < CH / 4; ++e)
                            d.x[j].w[e] = *(const u32x4_t*)(p + 1024 * RT + (16 * j + i16) * T::X_ROW +
                                                            16 * ((CH / 4 * g + e) ^ (i16 / PER & LOW)));
                        if constexpr (T::XS > 0) d.x[j].s = *(const uint8_t*)(p + T::S_AT + 256 * (RT + j) + 4 * i16 + g);
                    }
                    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");       // read before the slot is filled again
                    fetch(s0 + i + T::RING, i);
                    multiply(d, Half{});
                }
            }
        }
        wait_vmem<0>();
    }

    // steps whose columns come from memory directly
    const auto direct = [&](int st, auto half) {
        Step d;
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            const int64_t row = min(r0 + 16 * i + i16, a.d_out - 1);
            d.w[i] = *(const u32x4_t*)(a.W + row * a.w_row + 64 * (int64_t)st + 16 * g);
            d.s[i] = a.S[row * a.s_row + 4 * (int64_t)st + g];
        }
#pragma unroll
        for (int j = 0; j < TT; ++j)
            d.x[j].template load<false>(a, min(t0 + 16 * j + i16, a.n_tok - 1), 128 * (int64_t)st + 32 * g);
        multiply(d, half);
    };
    for (int st = a.full + wave; st < a.steps; st += T::WAVES) direct(st, Half{});
    if constexpr (DT == ACT_F16) {
        const bool again = __any(left);
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int j = 0; j < TT; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][j][e] = again ? 0.f : acc[i][j][e];
        if (again) {
            for (int st = first; st < end; ++st) direct(st, std::false_type{});
            for (int st = a.full + wave; st < a.steps; st += T::WAVES) direct(st, std::false_type{});
        }
    }

    // the waves' sums, in the order of the waves, AT tiles at a time
    constexpr int AT = T::AT;
    f32x4_t* part = (f32x4_t*)lds;
#pragma unroll
    for (int b = 0; b < RT * TT; b += AT) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < AT; ++e) part[(wave * AT + e) * 64 + lane] = acc[(b + e) / TT][(b + e) % TT];
        __syncthreads();
        for (int e = threadIdx.x; e < AT * 64; e += 64 * T::WAVES) {
            const int tile = b + (e >> 6), l = e & 63;
            f32x4_t v = part[e];
#pragma unroll
            for (int q = 1; q < T::WAVES; ++q) v += part[q * AT * 64 + e];
            const int64_t t = t0 + 16 * (tile % TT) + (l & 15), r = r0 + 16 * (tile / TT) + 4 * (l >> 4);
            if (t < a.n_tok) store4(a, t, r, v[0], v[1], v[2], v[3]);
        }
    }
}

// ---------------------------------------------------------------------------
// Many tokens, any activations: 128 weight rows x 128 tokens per workgroup of
// 2 x 2 waves, each 64 x 64 in v_mfma_f32_32x32x16.  Activations go through two LDS
// buffers of 64 columns (float32 ones as their three parts), weights straight
// from memory into the lanes that multiply them: lane l holds row l % 32 and,
// of every 64 columns, block l / 32.  Both are fetched a step ahead.  Bound by
// the conversions (float32: three products for one as well).  Measured: 2048 x
// 4096 -> 4096 with e4m3 activations 99 us (695 TFLOP/s), with float32 ones
// 257 us (267 TFLOP/s); 16-bit ones whose rows do not start on 16 bytes 306 us.
// ---------------------------------------------------------------------------
constexpr int MT = 128, MK = 64, X_ROW = MK * 2 + 16;   // 16 bytes further in the banks with each row

template <Act DT>
__global__ __launch_bounds__(256, 2) void mx_many_kernel(MatArgs a) {
    constexpr int RW = 2;
    constexpr int NP = DT == ACT_F32 ? 3 : 1;           // planes in LDS
    constexpr int BUF = NP * MT * X_ROW;
    extern __shared__ __attribute__((aligned(16))) char xs[];   // two buffers
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int i32 = lane & 31, h = lane >> 5;
    // consecutive workgroups go to different dies: give each die a run of
    // tiles that share weight rows
    const uint32_t nt = (uint32_t)((a.n_tok + MT - 1) / MT), n = gridDim.x, per = n / 8;
    const uint32_t id = blockIdx.x < per * 8 ? (blockIdx.x % 8) * per + blockIdx.x / 8 : blockIdx.x;
    const int64_t r0 = (int64_t)(id / nt) * (64 * RW) + 32 * RW * (wave >> 1), t0 = (int64_t)(id % nt) * MT;
    const int tw = 64 * (wave & 1);
    const uint8_t *wp[RW], *sp[RW];
#pragma unroll
    for (int i = 0; i < RW; ++i) {
        const int64_t row = min(r0 + 32 * i + i32, a.d_out - 1);
        wp[i] = a.W + row * a.w_row + 16 * h;
        sp[i] = a.S + row * a.s_row + h;
    }
    f16_t acc[RW][2];
#pragma unroll
    for (int i = 0; i < RW; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;

    // this thread's four pieces of eight columns
    Raw<DT, 1> x[4];
    const auto load_x = [&](int st) {
        if (st < 2 * a.full) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int e = threadIdx.x + 256 * q;
                x[q].template load<true>(a, min(t0 + (e >> 3), a.n_tok - 1), (int64_t)MK * st + 8 * (e & 7));
            }
        } else {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int e = threadIdx.x + 256 * q;
                x[q].template load<false>(a, min(t0 + (e >> 3), a.n_tok - 1), (int64_t)MK * st + 8 * (e & 7));
            }
        }
    };
    const auto store_x = [&](int b) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int e = threadIdx.x + 256 * q;
            char* p = xs + b * BUF + (e >> 3) * X_ROW + 16 * (e & 7);
            if constexpr (DT == ACT_F32) {
                u32x4_t v[3];
                parts<true>(x[q], 0, v);
#pragma unroll
                for (int j = 0; j < 3; ++j) *(u32x4_t*)(p + j * MT * X_ROW) = v[j];
            } else {
                *(u32x4_t*)p = x[q].eight(0);
            }
        }
    };
    bool left = false;       // float16: a block was left out
    u32x4_t w[RW];
    uint32_t sc[RW];
    const auto load_w = [&](int st) {
#pragma unroll
        for (int i = 0; i < RW; ++i) {
            w[i] = *(const u32x4_t*)(wp[i] + 32 * (int64_t)st);
            sc[i] = sp[i][2 * (int64_t)st];
        }
    };
    const int last = 2 * a.steps - 1;
    load_x(0);
    load_w(0);
    store_x(0);
    __syncthreads();
    for (int st = 0; st <= last; ++st) {
        const char* xb = xs + (st & 1) * BUF + (tw + i32) * X_ROW + 64 * h;
        u32x4_t cw[RW];
        uint32_t cs[RW];
#pragma unroll
        for (int i = 0; i < RW; ++i) {
            cw[i] = w[i];
            cs[i] = sc[i];
        }
        const int nx = min(st + 1, last);
        load_x(nx);
        load_w(nx);
        if constexpr (DT == ACT_F16) {
#pragma unroll
            for (int i = 0; i < RW; ++i) {
                const bool fits = scale_fits_f16(cs[i]);
                left |= !fits && (some(cw[i]) || cs[i] == 255u);
                cw[i] = codes_if(fits, cw[i]);
                if (!fits) cs[i] = 127u;
            }
        }
        constexpr bool HALF = DT == ACT_F16;
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int p = 0; p < NP; ++p) {
                u32x4_t b[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) b[j] = *(const u32x4_t*)(xb + (p * MT + 32 * j) * X_ROW + 16 * c);
#pragma unroll
                for (int i = 0; i < RW; ++i) {
                    const u32x4_t v = fp4x8<!HALF>(cw[i][c], mx_scale(cs[i]));
#pragma unroll
                    for (int j = 0; j < 2; ++j) acc[i][j] = H16<!HALF>::mfma32(v, b[j], acc[i][j]);
                }
            }
        store_x((st & 1) ^ 1);
        __syncthreads();
    }
    if constexpr (DT == ACT_F16) {
        const bool again = __any(left);
#pragma unroll
        for (int i = 0; i < RW; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int e = 0; e < 16; ++e) acc[i][j][e] = again ? 0.f : acc[i][j][e];
        for (int st = again ? 0 : last + 1; st <= last; ++st) {
            load_w(st);
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    Raw<DT, 1> y;
                    y.template load<false>(a, min(t0 + tw + 32 * j + i32, a.n_tok - 1), (int64_t)MK * st + 32 * h + 8 * c);
                    u32x4_t p[2];
                    split_f16(y.w[0], p);
#pragma unroll
                    for (int i = 0; i < RW; ++i) {
                        const u32x4_t v = fp4x8<true>(w[i][c], mx_scale(sc[i]));
                        acc[i][j] = H16<true>::mfma32(v, p[0], acc[i][j]);
                        acc[i][j] = H16<true>::mfma32(v, p[1], acc[i][j]);
                    }
                }
        }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int64_t t = t0 + tw + 32 * j + i32;
        if (t >= a.n_tok) continue;
#pragma unroll
        for (int i = 0; i < RW; ++i)
#pragma unroll
            for (int e = 0; e < 16; e += 4)
                store4(a, t, r0 + 32 * i + 2 * e + 4 * h, acc[i][j][e], acc[i][j][e + 1], acc[i][j][e + 2], acc[i][j][e + 3]);
    }
}

// ---------------------------------------------------------------------------
// Many tokens of 16 bits whose rows start on 16 bytes: 64 RG weight rows x 128
// tokens per workgroup of RG x 2 waves of 64 x 64, with both operands
// brought from memory to a ring of three LDS slots of 128 columns, two stages
// ahead and without registers.  16-byte chunk c of a row sits at slot c ^
// (row % 16) (activations: 16 chunks) or c ^ (row / 4 % 4) (codes: 4), so that
// sixteen rows' reads of one chunk hit all banks.  Scales are fetched for four
// stages at once, a quarter of the rows with each stage (four lanes to the 16
// bytes of a row), and held in registers from there.  Columns after the last
// whole 128 come from memory directly, at the end.  Bound by the matrix
// instructions (the matrix cores are busy for 69 % of the time) and, beside
// them, the conversions of the codes (four per eight products): 2048 x 4096 ->
// 11008 bf16 163 to 177 us by card (1043 to 1136 TFLOP/s, where a large library
// product of two bf16 matrices reaches 1600); through registers and one LDS
// buffer per operand it took 258 us.
// ---------------------------------------------------------------------------
template <int RG>
struct WideTile {
    static constexpr int WAVES = 2 * RG, WR = 64 * RG;
    static constexpr int W_BYTES = 64 * WR, X_BYTES = 256 * MT, STAGE = W_BYTES + X_BYTES, RING = 3, SCALES = 16 * WR;
    static constexpr int W_DMA = WR / 16 / WAVES, X_DMA = MT / 4 / WAVES;   // per wave and stage: 16 rows of codes, 4 tokens
    static constexpr int LDS = RING * STAGE + 2 * SCALES;
};

template <Act DT, int RG>
__global__ __launch_bounds__(128 * RG, 2) void mx_wide_kernel(MatArgs a) {
    using T = WideTile<RG>;
    constexpr int RW = 2, NW = T::WAVES;
    constexpr int DMA = T::W_DMA + T::X_DMA + 1;
    constexpr bool HALF = DT == ACT_F16;
    extern __shared__ __attribute__((aligned(16))) char lds[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int i32 = lane & 31, h = lane >> 5;
    const uint32_t nt = (uint32_t)((a.n_tok + MT - 1) / MT), n = gridDim.x, per = n / 8;
    const uint32_t id = blockIdx.x < per * 8 ? (blockIdx.x % 8) * per + blockIdx.x / 8 : blockIdx.x;
    const int64_t r0 = (int64_t)(id / nt) * T::WR, t0 = (int64_t)(id % nt) * MT;
    const int rw = 32 * RW * (wave >> 1), tw = 64 * (wave & 1);

    // buffers over the tile's rows: they end with the matrix
    const int64_t wn = min((int64_t)T::WR, a.d_out - r0), xn = min((int64_t)MT, a.n_tok - t0);
    const u32x4_t wb = buffer_of(a.W + r0 * a.w_row, wn * a.w_row), sb = buffer_of(a.S + r0 * a.s_row, wn * a.s_row);
    const u32x4_t xb = buffer_of((const uint16_t*)a.X + t0 * a.ld_x, 2 * ((xn - 1) * a.ld_x + a.d_in));
    uint32_t woff[T::W_DMA], xoff[T::X_DMA], soff[4];
#pragma unroll
    for (int j = 0; j < T::W_DMA; ++j) {
        const int r = 16 * (wave + NW * j) + (lane >> 2), c = (lane & 3) ^ (r >> 2 & 3);
        woff[j] = (uint32_t)(min((int64_t)r, wn - 1) * a.w_row + 16 * c);
    }
#pragma unroll
    for (int j = 0; j < T::X_DMA; ++j) {
        const int r = 4 * (wave + NW * j) + (lane >> 4), c = (lane & 15) ^ (r & 15);
        xoff[j] = (uint32_t)(min((int64_t)r, xn - 1) * 2 * a.ld_x + 16 * c);
    }
    // the waves bring some scales twice
#pragma unroll
    for (int k = 0; k < 4; ++k)
        soff[k] = (uint32_t)(min((int64_t)(16 * ((wave + NW * k) % (T::WR / 16)) + (lane >> 2)), wn - 1) * a.s_row + 4 * (lane & 3));
    const uint32_t base = (uint32_t)(uintptr_t)lds;
    const int stages = a.full, quads = (stages + 3) / 4;
    // stage f's codes and activations, and a quarter of the scales of the four
    // stages after its own four
    const auto fetch_scales = [&](int quad, int k) {
        dma_4(base + T::RING * T::STAGE + (quad & 1) * T::SCALES + 256 * ((wave + NW * k) % (T::WR / 16)),
              soff[k] + __builtin_amdgcn_readfirstlane(16 * min(quad, quads - 1)), sb);
    };
    // every eighth of a stage's pieces from e on
    constexpr int PIECES = T::W_DMA + T::X_DMA;
    const auto fetch = [&](int f, int slot, int e) {
        const int st = min(f, stages - 1);
        const uint32_t at = base + slot * T::STAGE;
#pragma unroll
        for (int j = e; j < PIECES; j += 8) {
            if (j < T::X_DMA)
                dma_16(at + T::W_BYTES + 1024 * (wave + NW * j), xoff[j] + __builtin_amdgcn_readfirstlane(256 * st), xb);
            else
                dma_16(at + 1024 * (wave + NW * (j - T::X_DMA)), woff[j - T::X_DMA] + __builtin_amdgcn_readfirstlane(64 * st), wb);
        }
    };

    f16_t acc[RW][2];
#pragma unroll
    for (int i = 0; i < RW; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
    bool left = false;       // float16: a block was left out
    int slot = 0;
    u32x4_t ws[RW];
    const auto multiply = [&](int st, auto kk) {
        constexpr int K = decltype(kk)::value;              // st % 4
        wait_vmem<DMA>();                                   // this stage has landed, the next may be under way
        meet();
        // The slot of the stage before is free: the stage after next goes there,
        // a few pieces with each step, so that the products need not wait until
        // all of it is asked for.
        const int fslot = slot == 0 ? 2 : slot - 1;
        if constexpr (K == 0) {
            const u32x4_t* p = (const u32x4_t*)(lds + T::RING * T::STAGE + (st >> 2 & 1) * T::SCALES) + rw + i32;
#pragma unroll
            for (int i = 0; i < RW; ++i) ws[i] = p[32 * i];
        }
        const char* wp = lds + slot * T::STAGE + (rw + i32) * 64;
        const char* xp = lds + slot * T::STAGE + T::W_BYTES + (tw + i32) * 256;
        u32x4_t w[2][RW], x[2][2];
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int i = 0; i < RW; ++i)
                w[q][i] = *(const u32x4_t*)(wp + 32 * 64 * i + 16 * ((2 * q + h) ^ (i32 >> 2 & 3)));
        // a step's activations are read while the one before multiplies
        const auto read = [&](int e) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
                x[e & 1][j] = *(const u32x4_t*)(xp + 32 * 256 * j + 16 * ((8 * (e >> 2) + 4 * h + (e & 3)) ^ (i32 & 15)));
        };
        read(0);
        float sc[RW];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int q = e >> 2, c = e & 3;
            if (e < 7) read(e + 1);
            if (c == 0) {
#pragma unroll
                for (int i = 0; i < RW; ++i) {
                    uint32_t byte = ws[i][K] >> (16 * q + 8 * h) & 255u;
                    if constexpr (HALF) {
                        const bool fits = scale_fits_f16(byte);
                        left |= !fits && (some(w[q][i]) || byte == 255u);
                        w[q][i] = codes_if(fits, w[q][i]);
                        byte = fits ? byte : 127u;
                    }
                    sc[i] = mx_scale(byte);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < RW; ++i) {
                const u32x4_t v = fp4x8<!HALF>(w[q][i][c], sc[i]);
#pragma unroll
                for (int j = 0; j < 2; ++j) acc[i][j] = H16<!HALF>::mfma32(v, x[e & 1][j], acc[i][j]);
            }
            fetch(st + 2, fslot, e);
            if (e == 7) fetch_scales(((st + 2) >> 2) + 1, (K + 2) & 3);
        }
        slot = slot == 2 ? 0 : slot + 1;
    };
#pragma unroll
    for (int k = 0; k < 4; ++k) fetch_scales(0, k);
#pragma unroll
    for (int e = 0; e < 8; ++e) fetch(0, 0, e);
    fetch_scales(1, 0);
#pragma unroll
    for (int e = 0; e < 8; ++e) fetch(1, 1, e);
    fetch_scales(1, 1);
    for (int st = 0; st < stages; st += 4) {
        multiply(st, std::integral_constant<int, 0>{});
        if (st + 1 < stages) multiply(st + 1, std::integral_constant<int, 1>{});
        if (st + 2 < stages) multiply(st + 2, std::integral_constant<int, 2>{});
        if (st + 3 < stages) multiply(st + 3, std::integral_constant<int, 3>{});
    }
    wait_vmem<0>();                                         // nothing lands in LDS that is another's by then

    // the columns after the last whole stage, or all of them
    const int last = 2 * a.steps;
    const bool again = DT == ACT_F16 && __any(left);
    if constexpr (DT == ACT_F16) {
#pragma unroll
        for (int i = 0; i < RW; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int e = 0; e < 16; ++e) acc[i][j][e] = again ? 0.f : acc[i][j][e];
    }
    for (int st = again ? 0 : 2 * stages; st < last; ++st) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                Raw<DT, 1> y;
                y.template load<false>(a, min(t0 + tw + 32 * j + i32, a.n_tok - 1), (int64_t)MK * st + 32 * h + 8 * c);
                u32x4_t p[parts_of<DT>()];
                parts<true>(y, 0, p);
#pragma unroll
                for (int i = 0; i < RW; ++i) {
                    const int64_t row = min(r0 + rw + 32 * i + i32, a.d_out - 1);
                    const uint32_t code = *(const uint32_t*)(a.W + row * a.w_row + 32 * (int64_t)st + 16 * h + 4 * c);
                    const u32x4_t v = fp4x8<true>(code, mx_scale(a.S[row * a.s_row + 2 * (int64_t)st + h]));
#pragma unroll
                    for (int k = 0; k < parts_of<DT>(); ++k) acc[i][j] = H16<true>::mfma32(v, p[k], acc[i][j]);
                }
            }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int64_t t = t0 + tw + 32 * j + i32;
        if (t >= a.n_tok) continue;
#pragma unroll
        for (int i = 0; i < RW; ++i)
#pragma unroll
            for (int e = 0; e < 16; e += 4)
                store4(a, t, r0 + rw + 32 * i + 2 * e + 4 * h, acc[i][j][e], acc[i][j][e + 1], acc[i][j][e + 2], acc[i][j][e + 3]);
    }
}

// ---------------------------------------------------------------------------
// Both operands e2m1: v_mfma_scale_f32_32x32x64_f8f6f4.  Lane l holds row
// (token) l % 32 and block l / 32 of the 64 columns, 16 bytes, with that
// block's scale.  (Checked on the GPU against float64.)
//
// 64 RW weight rows x 128 tokens per workgroup of 2 x 2 waves, each 32 RW x
// 64: at four bits a matrix instruction consumes its operands so fast that
// LDS feeds it only if each is used RW (or two) times.  Stages of 256 columns
// of codes go from memory to a ring of three LDS slots, two stages ahead.  Of
// a row's eight 16-byte chunks number c sits at slot c ^ (row / 2 % 8), so
// that sixteen rows' reads of one chunk hit all banks.  Scales are fetched for
// two stages at once (16 bytes of a row by four lanes: a request to the cache
// per row, where a word per lane was 64 of them and took as long as the
// codes), half of the rows with each stage, and held in registers from there.
// Measured: 2048 x 11008 -> 4096 55 to 58 us (3200 to 3350 TFLOP/s) with 256 x
// 128 tiles; 65 us with scales a word per lane, 102 us through registers and two
// LDS buffers.  Bound by the codes' way to LDS, 21 bytes a clock and compute
// unit, beside the matrix instructions: 42 to 48 us without fetching codes, 49
// without reading operands from LDS, 56 without fetching scales, 39.5 with
// matrix instructions alone (the chip runs at 1.8 GHz there).  The matrix cores
// are busy for 44 % of the time, LDS reads for 18 %.
// ---------------------------------------------------------------------------
template <int RW>
struct MxTile {
    static constexpr int WR = 64 * RW, ROWS = WR + 128;
    static constexpr int STAGE = 128 * ROWS, RING = 3, SCALES = 16 * ROWS;
    static constexpr int C_DMA = ROWS / 32, S_DMA = ROWS / 128;   // per wave and stage: 8 rows of codes, 16 of scales
    static constexpr int LDS = RING * STAGE + 2 * SCALES;
};

template <int Q>
__device__ __forceinline__ f16_t mfma_fp4(u32x4_t w, u32x4_t x, f16_t c, uint32_t ws, uint32_t xs) {
    const i32x8_t a = {(int)w.x, (int)w.y, (int)w.z, (int)w.w, 0, 0, 0, 0};
    const i32x8_t b = {(int)x.x, (int)x.y, (int)x.z, (int)x.w, 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 4, 4, 2 * (Q & 1), (int)ws, 2 * (Q & 1), (int)xs);
}

template <int RW>
__global__ __launch_bounds__(256, 1) void mx_mx_kernel(MatArgs a) {
    using T = MxTile<RW>;
    constexpr int DMA = T::C_DMA + T::S_DMA;
    extern __shared__ __attribute__((aligned(16))) char lds[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int i32 = lane & 31, h = lane >> 5;
    const uint32_t nt = (uint32_t)((a.n_tok + 127) / 128), n = gridDim.x, per = n / 8;
    const uint32_t id = blockIdx.x < per * 8 ? (blockIdx.x % 8) * per + blockIdx.x / 8 : blockIdx.x;
    const int64_t r0 = (int64_t)(id / nt) * T::WR, t0 = (int64_t)(id % nt) * 128;
    const int rw = 32 * RW * (wave >> 1), tw = 64 * (wave & 1);

    // Buffers over the tile's rows (they end with the matrix; the last stage
    // may read past a row's end, into columns that are not multiplied).
    const int64_t wn = min((int64_t)T::WR, a.d_out - r0), xn = min((int64_t)128, a.n_tok - t0);
    const u32x4_t wb = buffer_of(a.W + r0 * a.w_row, wn * a.w_row), xb = buffer_of((const uint8_t*)a.X + t0 * a.w_row, xn * a.w_row);
    const u32x4_t wsb = buffer_of(a.S + r0 * a.s_row, wn * a.s_row), xsb = buffer_of(a.XS + t0 * a.s_row, xn * a.s_row);
    // Codes: instruction j of wave w takes rows 8 (w + 4 j) .. + 7, lane l row
    // l / 8 and slot l % 8 of them.
    uint32_t coff[T::C_DMA];
#pragma unroll
    for (int j = 0; j < T::C_DMA; ++j) {
        const int r = 8 * (wave + 4 * j) + (lane >> 3), c = (lane & 7) ^ (r >> 1 & 7);
        const int64_t row = r < T::WR ? min((int64_t)r, wn - 1) : min((int64_t)r - T::WR, xn - 1);
        coff[j] = (uint32_t)(row * a.w_row + 16 * c);
    }
    // Scales of two stages: instruction j of wave w takes rows 16 (w + 4 j) ..
    // + 15, lane l word l % 4 of row l / 4; the first S_DMA of them make one
    // half, the others the other.
    uint32_t soff[2 * T::S_DMA];
#pragma unroll
    for (int j = 0; j < 2 * T::S_DMA; ++j) {
        const int r = 16 * (wave + 4 * j) + (lane >> 2);
        const int64_t row = r < T::WR ? min((int64_t)r, wn - 1) : min((int64_t)r - T::WR, xn - 1);
        soff[j] = (uint32_t)(row * a.s_row + 4 * (lane & 3));
    }
    const uint32_t base = (uint32_t)(uintptr_t)lds;
    const int stages = (a.steps + 1) / 2, pairs = (stages + 1) / 2;
    // quarter q of a stage's codes
    const auto fetch = [&](int st, int slot, int q) {
        const uint32_t at = base + slot * T::STAGE, co = __builtin_amdgcn_readfirstlane(128 * st);
#pragma unroll
        for (int i = 0; i < T::C_DMA / 4; ++i) {
            const int j = q * (T::C_DMA / 4) + i;
            dma_16(at + 1024 * (wave + 4 * j), coff[j] + co, 32 * j < T::WR ? wb : xb);
        }
    };
    const auto fetch_scales = [&](int pair, auto half) {
        const uint32_t at = base + T::RING * T::STAGE + (pair & 1) * T::SCALES;
        const uint32_t so = __builtin_amdgcn_readfirstlane(16 * min(pair, pairs - 1));
#pragma unroll
        for (int i = 0; i < T::S_DMA; ++i) {
            constexpr int H = decltype(half)::value;
            const int j = H * T::S_DMA + i;
            dma_4(at + 256 * (wave + 4 * j), soff[j] + so, 64 * j + 16 * wave < T::WR ? wsb : xsb);
        }
    };

    f16_t acc[RW][2];
#pragma unroll
    for (int i = 0; i < RW; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
    using First = std::integral_constant<int, 0>;
    using Second = std::integral_constant<int, 1>;
    fetch_scales(0, First{});
    fetch_scales(0, Second{});
#pragma unroll
    for (int q = 0; q < 4; ++q) fetch(0, 0, q);
#pragma unroll
    for (int q = 0; q < 4; ++q) fetch(min(1, stages - 1), 1, q);
    fetch_scales(1, First{});
    int slot = 0;
    u32x4_t ws[RW], xs[2];
    // Stage 2 p + k: PAIR k of the scales of pair p.
    const auto multiply = [&](int st, auto k) {
        constexpr int K = decltype(k)::value;
        wait_vmem<DMA>();                               // this stage has landed, the next may be under way
        meet();
        // The slot of the stage before is free: the stage after next goes there,
        // a quarter with each step, so that the products need not wait until
        // all of it is asked for.
        const int far = min(st + 2, stages - 1), fslot = slot == 0 ? 2 : slot - 1;
        if constexpr (K == 0) {
            const u32x4_t* sb = (const u32x4_t*)(lds + T::RING * T::STAGE + (st >> 1 & 1) * T::SCALES) + i32;
#pragma unroll
            for (int i = 0; i < RW; ++i) ws[i] = sb[rw + 32 * i];
#pragma unroll
            for (int j = 0; j < 2; ++j) xs[j] = sb[T::WR + tw + 32 * j];
        }
        const char* cb = lds + slot * T::STAGE;
        const char* wp = cb + (rw + i32) * 128;
        const char* xp = cb + (T::WR + tw + i32) * 128;
        // a step's operands are read while the one before multiplies
        u32x4_t x[2][2], w[2][RW];
        const auto read = [&](auto q) {
            constexpr int Q = decltype(q)::value;
            const int c = 16 * ((2 * Q + h) ^ (i32 >> 1 & 7));
#pragma unroll
            for (int j = 0; j < 2; ++j) x[Q & 1][j] = *(const u32x4_t*)(xp + 32 * 128 * j + c);
#pragma unroll
            for (int i = 0; i < RW; ++i) w[Q & 1][i] = *(const u32x4_t*)(wp + 32 * 128 * i + c);
            __builtin_amdgcn_sched_barrier(0);
        };
        const auto step = [&](auto q) {
            constexpr int Q = decltype(q)::value, W = 2 * K + (Q >> 1);
#pragma unroll
            for (int i = 0; i < RW; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    acc[i][j] = mfma_fp4<Q>(w[Q & 1][i], x[Q & 1][j], acc[i][j], ws[i][W] >> (8 * h), xs[j][W] >> (8 * h));
        };
        using Q0 = std::integral_constant<int, 0>;
        using Q1 = std::integral_constant<int, 1>;
        using Q2 = std::integral_constant<int, 2>;
        using Q3 = std::integral_constant<int, 3>;
        const bool both = 2 * st + 1 < a.steps;       // uniform: the last stage can be half a one
        read(Q0{});
        read(Q1{});
        step(Q0{});
        fetch(far, fslot, 0);
        if (both) read(Q2{});
        step(Q1{});
        fetch(far, fslot, 1);
        if constexpr (K == 0) fetch_scales((st >> 1) + 1, Second{});
        else fetch_scales((st >> 1) + 2, First{});      // this pair's scales are in registers
        if (both) {
            read(Q3{});
            step(Q2{});
        }
        fetch(far, fslot, 2);
        if (both) step(Q3{});
        fetch(far, fslot, 3);
        slot = slot == 2 ? 0 : slot + 1;
    };
    for (int st = 0; st < stages; st += 2) {
        multiply(st, First{});
        if (st + 1 < stages) multiply(st + 1, Second{});
    }
    wait_vmem<0>();                                     // nothing lands in LDS that is another's by then
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int64_t t = t0 + tw + 32 * j + i32;
        if (t >= a.n_tok) continue;
#pragma unroll
        for (int i = 0; i < RW; ++i)
#pragma unroll
            for (int e = 0; e < 16; e += 4)
                store4(a, t, r0 + rw + 32 * i + 2 * e + 4 * h, acc[i][j][e], acc[i][j][e + 1], acc[i][j][e + 2], acc[i][j][e + 3]);
    }
}

template <Act DT, int RT, int TT>
gptq_status launch_few(const MatArgs& a, hipStream_t s) {
    using T = FewTile<DT, RT, TT>;
    GPTQ_HIP(ensure_lds_limit((const void*)mx_few_kernel<DT, RT, TT>, T::BYTES));
    hipLaunchKernelGGL((mx_few_kernel<DT, RT, TT>),
                       dim3((unsigned)ceil_div(a.d_out, 16 * RT), (unsigned)ceil_div(a.n_tok, 16 * TT)),
                       dim3(64 * T::WAVES), T::BYTES, s, a);
    return GPTQ_OK;
}

template <Act DT>
gptq_status launch_many(const MatArgs& a, hipStream_t s) {
    constexpr int lds = 2 * (DT == ACT_F32 ? 3 : 1) * MT * X_ROW;
    GPTQ_HIP(ensure_lds_limit((const void*)mx_many_kernel<DT>, lds));
    hipLaunchKernelGGL(mx_many_kernel<DT>, dim3((unsigned)(ceil_div(a.d_out, 128) * ceil_div(a.n_tok, MT))), dim3(256), lds,
                       s, a);
    return GPTQ_OK;
}

template <Act DT, int RG>
gptq_status launch_wide(const MatArgs& a, hipStream_t s) {
    constexpr int lds = WideTile<RG>::LDS;
    GPTQ_HIP(ensure_lds_limit((const void*)mx_wide_kernel<DT, RG>, lds));
    hipLaunchKernelGGL((mx_wide_kernel<DT, RG>), dim3((unsigned)(ceil_div(a.d_out, 64 * RG) * ceil_div(a.n_tok, MT))),
                       dim3(128 * RG), lds, s, a);
    return GPTQ_OK;
}

template <int RW>
gptq_status launch_mx(const MatArgs& a, hipStream_t s) {
    constexpr int lds = MxTile<RW>::LDS;
    GPTQ_HIP(ensure_lds_limit((const void*)mx_mx_kernel<RW>, lds));
    hipLaunchKernelGGL(mx_mx_kernel<RW>, dim3((unsigned)(ceil_div(a.d_out, 64 * RW) * ceil_div(a.n_tok, 128))),
                       dim3(256), lds, s, a);
    return GPTQ_OK;
}

// Workgroups of tiles of r rows x t tokens, in rounds of one per compute unit.
double rounds(const MatArgs& a, int64_t r, int64_t t) {
    return std::ceil((double)(ceil_div(a.d_out, r) * ceil_div(a.n_tok, t)) / 256.0);
}

// Which kernel, and which tile: the least of rounds x time per round, measured
// in us at 4096 columns (they grow alike with the columns).  Few-token tiles of
// 16 RT x 16 TT for (RT, TT) = (1,1) (2,1) (3,1) (4,1) (2,2) (4,2) (4,4), 0
// where LDS does not hold two steps per wave, and for e2m1 (4,4), which took
// 13.3 where 128 x 128 takes 13.0 and never has fewer workgroups; then the
// others: 16-bit 128 x 128 and 256 x 128 from LDS rings, and so e2m1 by e2m1;
// else 128 x 128 through registers, where two (float32) or three workgroups
// share a compute unit.  For example bf16 4096 -> 4096: 32 tokens (2,1) 6.6 us,
// (1,1) 9.0, (4,2) 9.0; 256 tokens (4,2) 20, 128 x 128 26; 2048 tokens 256 x 128
// 63, 128 x 128 72.  One token 4096 -> 11008: (3,1) 8.5, (4,1) 9.9, (2,1) 11.3,
// (1,1) 13.0.
constexpr double FEW_US[5][7] = {{7.8, 10.5, 12.0, 13.5, 20, 0, 0},        // float32
                                 {3.9, 5.0, 6.0, 6.9, 6.4, 9.4, 0},        // float16
                                 {3.9, 5.0, 6.0, 6.9, 6.4, 9.4, 0},        // bfloat16
                                 {3.5, 4.8, 5.7, 6.6, 5.9, 9.1, 13.4},     // e4m3
                                 {2.1, 4.1, 5.4, 6.6, 5.9, 8.7, 0}};      // e2m1
// Where X's rows do not start on 16 bytes (or have no 128 columns), every step
// is read by single elements, without the ring: one round of the tiles in the
// same order, float32 and 16 bits (float32 (1,1): 29 for 13 tokens, 48 for 16).
// Times of the general kernel there: float32 226 a round, 16 bits 250 for one
// and 305 for two rounds.  64 tokens 4096 -> 4096 bf16: (4,1) 27 us, (2,2) 46,
// which the ring's times would choose.
constexpr double DIRECT_US[2][7] = {{40, 41, 43, 44, 81, 0, 0}, {21, 24, 26, 28, 52, 57, 0}};
static_assert(ACT_F32 == 0 && ACT_F16 == 1 && ACT_BF16 == 2 && ACT_FP8 == 3 && ACT_FP4 == 4, "rows of the table");
constexpr int FEW_RT[7] = {1, 2, 3, 4, 2, 4, 4}, FEW_TT[7] = {1, 1, 1, 1, 2, 2, 4};

// 0 .. 6: a few-token tile; 7, 8: 128 (256) x 128 from LDS rings; 9: 128 x 128 through registers.
template <Act DT>
int choose(const MatArgs& a) {
    int best = 0;
    double least = 1e30;
    const auto offer = [&](int id, double cost) {
        if (cost < least) {
            least = cost;
            best = id;
        }
    };
    const double* us = a.full > 0 ? FEW_US[DT] : DIRECT_US[DT != ACT_F32];
    for (int i = 0; i < 7; ++i)
        if (us[i] > 0) offer(i, rounds(a, 16 * FEW_RT[i], 16 * FEW_TT[i]) * us[i]);
    if constexpr (DT == ACT_BF16 || DT == ACT_F16) {
        if (a.full > 0) {
            offer(7, rounds(a, 128, MT) * 25.0);
            offer(8, rounds(a, 256, MT) * 43.0);
        } else {
            offer(9, std::max(1.0, 0.61 * rounds(a, 128, MT)) * 250.0);
        }
    } else if constexpr (DT == ACT_F32) {
        offer(9, rounds(a, 128, MT) * (a.full > 0 ? 130.0 : 226.0));
    } else if constexpr (DT == ACT_FP8) {
        offer(9, std::max(1.0, 0.68 * rounds(a, 128, MT)) * 69.0);
    } else {
        offer(7, rounds(a, 128, MT) * 13.0);
        offer(8, rounds(a, 256, MT) * 25.0);
    }
    return best;
}

template <Act DT, int I>
gptq_status launch_tile(const MatArgs& a, hipStream_t s) {
    static_assert((FEW_US[DT][I] > 0) == (FewTile<DT, FEW_RT[I], FEW_TT[I]>::FITS && !(DT == ACT_FP4 && I == 6)),
                  "zeros where a tile does not fit, or is never the best");
    if constexpr (FEW_US[DT][I] > 0) return launch_few<DT, FEW_RT[I], FEW_TT[I]>(a, s);
    else return GPTQ_ERR_UNSUPPORTED;      // never chosen
}

template <Act DT>
gptq_status launch_parts(const MatArgs& a, hipStream_t s) {
    const int best = choose<DT>(a);
    switch (best) {
        case 0: return launch_tile<DT, 0>(a, s);
        case 1: return launch_tile<DT, 1>(a, s);
        case 2: return launch_tile<DT, 2>(a, s);
        case 3: return launch_tile<DT, 3>(a, s);
        case 4: return launch_tile<DT, 4>(a, s);
        case 5: return launch_tile<DT, 5>(a, s);
        case 6: return launch_tile<DT, 6>(a, s);
        default: break;
    }
    if constexpr (DT == ACT_BF16 || DT == ACT_F16) {
        if (best == 7) return launch_wide<DT, 2>(a, s);
        if (best == 8) return launch_wide<DT, 4>(a, s);
    }
    if constexpr (DT == ACT_FP4) return best == 7 ? launch_mx<2>(a, s) : launch_mx<4>(a, s);
    else return launch_many<DT>(a, s);
}


MatArgs mat_args(const uint8_t* codes, const uint8_t* scales, int64_t n_tok, int64_t d_in, int64_t d_out, float* Y,
                 int64_t ld_y) {
    MatArgs a;
    a.X = nullptr;
    a.XS = nullptr;
    a.ld_x = 0;
    a.aligned = false;
    a.full = (int)ceil_div(d_in, MX_PAD);
    a.y_aligned = ((uintptr_t)Y | (uintptr_t)(4 * ld_y)) % 16 == 0;
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

// Steps of 16-bit or float32 activations that are read in whole pieces: offsets
// within a tile's tokens stay below 2^30.
int whole_steps(bool aligned, int64_t d_in, int64_t ld_x) {
    return aligned && ld_x <= (int64_t(1) << 20) ? (int)(d_in / MX_PAD) : 0;
}

}  // namespace

int mx_matmul_kernel(gptq_dtype dt, gptq_mx_format xf, int64_t n_tok, int64_t d_in, int64_t d_out, bool aligned) {
    MatArgs a = mat_args(nullptr, nullptr, n_tok, d_in, d_out, nullptr, d_out);
    if (xf == GPTQ_MX_FP8) return choose<ACT_FP8>(a);
    if (xf == GPTQ_MX_FP4) return choose<ACT_FP4>(a);
    a.full = whole_steps(aligned, d_in, d_in);
    return dt == GPTQ_BF16 ? choose<ACT_BF16>(a) : dt == GPTQ_F16 ? choose<ACT_F16>(a) : choose<ACT_F32>(a);
}

gptq_status mx_matmul_launch(const void* X, gptq_dtype dt, int64_t n_tok, int64_t d_in, int64_t ld_x,
                             const uint8_t* codes, const uint8_t* scales, int64_t d_out, float* Y, int64_t ld_y,
                             hipStream_t s) {
    MatArgs a = mat_args(codes, scales, n_tok, d_in, d_out, Y, ld_y);
    a.X = X;
    a.ld_x = ld_x;
    if (n_tok == 1) ld_x = a.ld_x = ceil_div(d_in, 8) * 8;   // of no use
    a.aligned = ((uintptr_t)X | (uintptr_t)(ld_x * (dt == GPTQ_F32 ? 4 : 2))) % 16 == 0;
    a.full = whole_steps(a.aligned, d_in, ld_x);
    gptq_status st;
    switch (dt) {
        case GPTQ_BF16: st = launch_parts<ACT_BF16>(a, s); break;
        case GPTQ_F16: st = launch_parts<ACT_F16>(a, s); break;
        default: st = launch_parts<ACT_F32>(a, s); break;
    }
    if (st != GPTQ_OK) return st;
    GPTQ_LAUNCH_CHECK();
    return GPTQ_OK;
}

gptq_status mx_matmul_quantized_launch(const uint8_t* xc, const uint8_t* xs, gptq_mx_format xf, int64_t n_tok,
                                       int64_t d_in, const uint8_t* codes, const uint8_t* scales, int64_t d_out,
                                       float* Y, int64_t ld_y, hipStream_t s) {
    MatArgs m = mat_args(codes, scales, n_tok, d_in, d_out, Y, ld_y);
    m.X = xc;
    m.XS = xs;
    m.ld_x = mx_code_bytes(d_in, xf);
    const gptq_status st = xf == GPTQ_MX_FP8 ? launch_parts<ACT_FP8>(m, s) : launch_parts<ACT_FP4>(m, s);
    if (st != GPTQ_OK) return st;
    GPTQ_LAUNCH_CHECK();
    return GPTQ_OK;
}

}  // namespace gptq
