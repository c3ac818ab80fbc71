// Gradients of products with e2m1 weights for their activations:
// dX = dY W (include/gptq.h, gptq_mx_matmul_backward), and of gated products,
// dX = dG Wg + dU Wu (gptq_mx_gated_backward).
#include <algorithm>
#include <type_traits>
#include <utility>

#include "gated.hpp"

namespace gptq {
namespace {

// 16-bit planes that a call's gradients are given to the matrix cores in: dY is
// taken as it is, dG and dU as below.
constexpr int planes_of(gptq_dtype dt) { return dt == GPTQ_F32 ? 3 : 1; }
constexpr int gate_planes(gptq_dtype dt) { return dt == GPTQ_F32 ? 3 : dt == GPTQ_F16 ? 2 : 1; }

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

// One call, as the kernels see it.  The sum runs over segments: a matrix's rows
// with one plane of the gradients (one to three, planes_of and gate_planes), each
// in stages of 64 rows; rows past a segment's end are zeros in both operands.
struct Call {
    BackArgs b;
    const uint16_t* D;         // planes of 16-bit values: [token][segment][pad]
    int64_t ld, pad;           // of D: token to token, segment to segment (elements, 16-byte multiples)
    bool half;                 // the planes hold float16, not bfloat16
    int planes;                // segments of one matrix
    int64_t w_row, s_row;      // bytes per row
    int stages, per;           // stages of one segment; stages of one part
    int parts;
    bool joined;               // to sums, not to dX
    float* sums;               // [part][token][pitch]
    int64_t pitch;             // d_in, to whole groups of eight
};

// ---------------------------------------------------------------------------
// 256 columns x 64 TF tokens per workgroup of 2 x 2 waves, each 128 columns x 32
// TF tokens in v_mfma_f32_32x32x16, in stages of 64 rows of the matrix.
//
// The weights' rows are the sum's index here, and a lane of the instruction
// wants eight rows of one column, while memory holds a column's rows apart.  So
// a thread takes eight rows of eight columns, converts the two columns of
// a byte with their row's scale in one instruction, puts two rows' halves together
// with a byte permute, and stores eight rows of each column in a row: one
// instruction a value, once a workgroup.
//
// Codes, scales and gradients come from memory to rings of LDS slots without
// registers, some stages ahead; a stage's codes are converted during the stage
// before.  A step's operands are read while the one before multiplies, and the
// barrier of a stage stands before its last step, whose operands are in
// registers by then, so that the matrix instructions run on behind it.
//
// 2048 tokens through 4096 rows of 11008 bf16: 192 us (960 TFLOP/s; matrix
// instructions busy 52 % of the clocks, on a chip that lowers its clock as they run:
// alone they would take 1180 of a stage's 1600 ns), through 2 x 11008 rows of 4096, in
// float16 values, 345 us (1070; busy 60 %).  24 tokens, 4096 x 4096: 13 us, of which
// the four stages of each part take some 4 and the way in and out the rest.
//
// Tokens lie in LDS in order, column c at place (c % 4) 64 + c / 4; 16-byte chunk
// q (eight rows) of place i at slot q ^ (i / 2 % 8), so that sixteen lanes' reads
// of one chunk of neighbouring places hit all banks.  Lane l ends with columns 4 m + c of its tokens (m the row of
// the instruction's result, c the column of its four): sixteen neighbours at a
// time.
// ---------------------------------------------------------------------------
constexpr int BN = 256, SK = 64;
constexpr int RAW = SK * BN / 2, RAW_S = SK * BN / 32;     // bytes of a stage's codes and scales
constexpr int WT = SK * BN * 2;                            // and of its weights
template <int TF>
struct BackTile {
    static constexpr int BT = 64 * TF, X = BT * SK * 2, WAVES = 4;
    static constexpr int R = BT > 128 ? 2 : BT > 64 ? 3 : 4;                             // slots of a ring
    static constexpr int W = R * X, RAWS = W + 2 * WT, RAW_SCALES = RAWS + R * RAW, BYTES = RAW_SCALES + R * RAW_S;
    // per wave and stage; the scales are two instructions, which some waves repeat
    static constexpr int X_DMA = X / 1024 / WAVES, W_DMA = RAW / 1024 / WAVES, DMA = X_DMA + W_DMA + 1;
    // Behind the barrier of stage s - 1 the codes of s + R and the gradients of
    // s + R - 1 are asked for, into the slots that it let go.  At that of s the codes
    // of s + 2 and the gradients of s + 1 have landed if only what R - 2 stages
    // asked for since is under way.
    static constexpr int WAIT = (R - 2) * DMA;
    static_assert(BYTES <= 160 * 1024 - 1024 && WAIT < 64, "LDS and counters");
};

// As dma_16 of mx.hpp, with the address in LDS and that in memory each the sum of
// a register and something the wave shares.
__device__ __forceinline__ void dma_16_at(uint32_t to, int plus, uint32_t off, int at, u32x4_t buf) {
    asm volatile("s_add_u32 m0, %0, %1\n\ts_nop 0\n\tbuffer_load_dwordx4 %2, %3, %4 offen lds"
                 : : "s"(to), "n"(plus), "v"(off), "s"(buf), "s"(at) : "memory", "scc");
}
// A raw buffer from uniform values.
__device__ __forceinline__ u32x4_t buffer_at(const void* p, uint32_t bytes) {
    const uint64_t b = (uint64_t)(uintptr_t)p;
    return u32x4_t{(uint32_t)b, (uint32_t)(b >> 32) & 0xFFFFu, bytes, 0x00020000u};
}

// f(0), f(1), .. f(N - 1), each number a constant.
template <class F, int... I>
__device__ __forceinline__ void for_each(F&& f, std::integer_sequence<int, I...>) {
    (f(std::integral_constant<int, I>{}), ...);
}
template <int N, class F>
__device__ __forceinline__ void for_each(F&& f) {
    for_each(f, std::make_integer_sequence<int, N>{});
}

// An address in LDS that stays in its register, for constants to be added by the
// instructions (which have room for 16 bits of them).
__device__ __forceinline__ uint32_t held(uint32_t at) {
    asm volatile("" : "+v"(at));
    return at;
}
template <class V>
__device__ __forceinline__ __attribute__((address_space(3))) V& lds_at(uint32_t at, int plus) {
    return *(__attribute__((address_space(3))) V*)(uintptr_t)(at + plus);
}

// A workgroup's tile: columns n0 .. and tokens t0 .., and its stages of the sum.
// Consecutive workgroups go to different dies: give each die a run of tiles,
// four of tokens by as many of columns (a stage's gradients are four times its
// codes: of 32 tiles 4 x 8 have the fewest bytes to share).
struct Place {
    int64_t n0, t0;
    int part, first, end;
};
template <int BT, class C>
__device__ __forceinline__ Place place_of(const C& c) {
    const uint32_t nt = (uint32_t)((c.b.n_tok + BT - 1) / BT), nn = (uint32_t)((c.b.d_in + BN - 1) / BN);
    const uint32_t n = gridDim.x, each = n / 8;
    const uint32_t id = blockIdx.x < each * 8 ? (blockIdx.x % 8) * each + blockIdx.x / 8 : blockIdx.x;
    const int part = (int)(id / (nt * nn));
    const uint32_t tile = id % (nt * nn), rows4 = tile / (4 * nn) * 4, in4 = tile % (4 * nn), of4 = min(4u, nt - rows4);
    const int first = part * c.per;
    return Place{(int64_t)(in4 / of4) * BN, (int64_t)(rows4 + in4 % of4) * BT, part, first,
                 min(first + c.per, c.stages * c.b.matrices * c.planes)};
}

template <bool HALF, int TF>
__global__ __launch_bounds__(256, 1) void mx_back_kernel(Call c) {
    using T = BackTile<TF>;
    extern __shared__ __attribute__((aligned(16))) char lds[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int i32 = lane & 31, h = lane >> 5, nw = 128 * (wave / 2), tw = 32 * TF * (wave % 2);
    f16_t acc[4][TF];
    uint32_t left = 0;       // not 0: codes whose scale float16 lacks
    // The tile's sums.  FAR: of float16 gradients beside such weights.
    const auto sum = [&](auto far, const auto& c) __attribute__((always_inline)) {
        constexpr bool FAR = decltype(far)::value, F16 = HALF && !FAR;
        const auto& a = c.b;
        const auto [n0, t0, part, first, end] = place_of<T::BT>(c);
        const int S = end - first;

        // this thread's pieces
        const int64_t tn = min((int64_t)T::BT, a.n_tok - t0);
        uint32_t xoff[T::X_DMA], woff[T::W_DMA], soff;
#pragma unroll
        for (int j = 0; j < T::X_DMA; ++j) {                  // eight tokens an instruction
            const int t = 8 * (wave + T::WAVES * j) + (lane >> 3), ch = (lane & 7) ^ (t >> 1 & 7);
            xoff[j] = (uint32_t)(min((int64_t)t, tn - 1) * c.ld * 2 + 16 * ch);
        }
#pragma unroll
        for (int j = 0; j < T::W_DMA; ++j) {                  // eight rows an instruction
            const int k = 8 * (wave + T::WAVES * j) + (lane >> 3);
            const int64_t at = n0 / 2 + 16 * (lane & 7);
            woff[j] = at < c.w_row ? (uint32_t)(k * c.w_row + at) : 1u << 31;
        }
        {                                                     // 32 rows an instruction
            const int k = 32 * (wave & 1) + (lane >> 1);
            const int64_t at = n0 / 32 + 4 * (lane & 1);
            soff = at < c.s_row ? (uint32_t)(k * c.s_row + at) : 1u << 31;
        }
        const uint32_t base = (uint32_t)(uintptr_t)lds;
        // Stages come one after another in D's rows, over the segments.  Past the
        // last one the fetches repeat it, into slots that nobody reads.
        const u32x4_t xb = buffer_of(c.D + t0 * c.ld, ((tn - 1) * c.ld + (int64_t)c.stages * a.matrices * c.planes * SK) * 2);
        int xcol = 2 * SK * first;
        const int xlast = 2 * SK * (end - 1);
        const auto fetch_x = [&](int slot, int from, int to) {
#pragma unroll
            for (int j = from; j < to; ++j) dma_16_at(base + slot * T::X + 1024 * wave, 1024 * T::WAVES * j, xoff[j], xcol, xb);
            if (to == T::X_DMA) xcol = min(xcol + 2 * SK, xlast);
        };
        // codes and scales from here on, and of the matrices
        const uint8_t *wp, *sp, *wp0 = a.codes[0], *sp0 = a.scales[0], *wp1 = a.codes[1], *sp1 = a.scales[1];
        int64_t wrows;                                                    // left of the segment
        int wseg = first / c.stages, wleft = S;
        {
            const int64_t k0 = (int64_t)(first - wseg * c.stages) * SK;
            const int m = wseg >= c.planes;
            wp = a.codes[m] + k0 * c.w_row;
            sp = a.scales[m] + k0 * c.s_row;
            wrows = a.rows - k0;
        }
        u32x4_t wb, sb;
        const auto fetch_w = [&](int slot, int piece) {
            if (piece == 0) {
                const uint32_t rows = (uint32_t)min((int64_t)SK, wrows);
                wb = buffer_at(wp, rows * (uint32_t)c.w_row);
                sb = buffer_at(sp, rows * (uint32_t)c.s_row);
            }
            if (piece < T::W_DMA) {
                dma_16_at(base + T::RAWS + slot * RAW + 1024 * wave, 1024 * T::WAVES * piece, woff[piece], 0, wb);
                return;
            }
            dma_4(base + T::RAW_SCALES + slot * RAW_S + 256 * (wave & 1), soff, sb);
            // on to the next rows, or the next segment's first (no branch: it would
            // part the loop, and with it what is ordered among the products)
            const bool more = --wleft > 0, turns = more && wrows <= SK;
            wseg += turns;
            const bool second = wseg >= c.planes;
            wp = turns ? (second ? wp1 : wp0) : wp + (more ? SK * c.w_row : 0);
            sp = turns ? (second ? sp1 : sp0) : sp + (more ? SK * c.s_row : 0);
            wrows = turns ? a.rows : wrows - (more ? SK : 0);
        };

#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < TF; ++j)
#pragma unroll
                for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;

        // conversion: thread (q, o) has rows 8 q .. + 7 of the o-th group of eight columns,
        // whose codes a word holds
        const int q8 = threadIdx.x / 32, o8 = threadIdx.x % 32;
        struct Raw {
            uint32_t w[8], s[8];
        };
        uint32_t code_at = held(base + T::RAWS + 8 * q8 * (BN / 2) + 4 * o8);
        uint32_t scale_at = held(base + T::RAW_SCALES + 8 * q8 * (BN / 32) + o8 / 4);
        const auto raw_read = [&](Raw& r, int k) {
            r.w[k] = lds_at<uint32_t>(code_at, k * (BN / 2));
            r.s[k] = lds_at<uint8_t>(scale_at, k * (BN / 32));
        };
        // codes that are not all zero with a scale byte outside 104 .. 140 (byte 255
        // makes NaN of float16, too)
        const auto look = [&](const Raw& r, int k) {
            left |= min(__builtin_elementwise_sub_sat(r.s[k] - 104u, 36u), r.w[k]);
        };
        // two rows of a pair of columns
        const auto convert = [](const Raw& r, const float (&sc)[8], auto pair, int k, u32x4_t (&v)[2]) {
            constexpr int P = decltype(pair)::value;
            const uint32_t a = H16<!F16>::template fp4<P>(r.w[2 * k], sc[2 * k]);
            const uint32_t b = H16<!F16>::template fp4<P>(r.w[2 * k + 1], sc[2 * k + 1]);
            v[0][k] = __builtin_amdgcn_perm(b, a, 0x05040100u);
            v[1][k] = __builtin_amdgcn_perm(b, a, 0x07060302u);
        };
        // column c of the group: column 8 o + c of the tile, at place (c % 4) 64 + 2 o + c / 4
        uint32_t to = held(base + T::W + 2 * o8 * (SK * 2) + 16 * ((q8 ^ o8) & 7));
        const auto write = [&](int c, u32x4_t v) { lds_at<u32x4_t>(to, ((c & 3) * 64 + (c >> 2)) * (SK * 2)) = v; };

        // a step's operands
        struct Step {
            u32x4_t w[4], x[TF];
        };
        // in the order of their use: x0, the weights (columns 4 i32 + i), the other x
        uint32_t x_at[4], w_at[4];
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
            const int chunk = 16 * ((2 * ks + h) ^ (i32 >> 1 & 7));
            x_at[ks] = held(base + (tw + i32) * (SK * 2) + chunk);
            w_at[ks] = held(base + T::W + (nw / 4 + i32) * (SK * 2) + chunk);
        }
        const auto read = [&](uint32_t x, uint32_t w, Step& r, int n) {
            if (n == 0 || n > 4) {
                const int j = n == 0 ? 0 : n - 4;
                r.x[j] = lds_at<u32x4_t>(x, 32 * j * (SK * 2));
            } else {
                r.w[n - 1] = lds_at<u32x4_t>(w, 64 * (n - 1) * (SK * 2));
            }
        };

        // float16 gradients in two bfloat16 parts
        int e2[TF];
        u32x4_t xp[2];
        if constexpr (FAR) {
#pragma unroll
            for (int j = 0; j < TF; ++j) e2[j] = a.exps ? a.exps[min(t0 + tw + 32 * j + i32, a.n_tok - 1)] : 0;
        }
        const auto parts = [](u32x4_t x, int e2, u32x4_t (&p)[2]) {
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = ldexpf(H16<false>::to_f32((uint16_t)(x[e >> 1] >> (16 * (e & 1)))), e2);
            cut(f, p);
        };

        const auto ask_w = [&](int slot) {
#pragma unroll
            for (int e = 0; e <= T::W_DMA; ++e) fetch_w(slot, e);
        };
        for_each<T::R>([&](auto f) { ask_w(f); });
        for_each<T::R - 1>([&](auto f) { fetch_x(f, 0, T::X_DMA); });
        wait_vmem<0>();
        meet();
        Raw r;
        float sc[8];
        u32x4_t v[2][2];
        for_each<8>([&](auto k) {
            raw_read(r, k);
            sc[k] = mx_scale(r.s[k]);
        });
        for_each<4>([&](auto p) {
            for_each<4>([&](auto k) { convert(r, sc, p, k, v[0]); });
            write(2 * p, v[0][0]);
            write(2 * p + 1, v[0][1]);
        });
        if constexpr (F16) for_each<8>([&](auto k) { look(r, k); });
        meet();
        ask_w(0);
        Step d0, d1;
        for_each<4 + TF>([&](auto n) { read(x_at[0], w_at[0], d0, n); });

        // The ring's slots of this stage, as scalars; the lanes' addresses point at the
        // stage's gradients and weights, at the next one's codes and where its weights
        // go, and move on with the stages.
        int slot = 0, wslot = 0;
        const auto onward = [](int at, int bytes) { return at == T::R - 1 ? -(T::R - 1) * bytes : bytes; };
        code_at += RAW;
        scale_at += RAW_S;
        to += WT;
        for (int s = 0; s < S; ++s) {
            const int next = slot == T::R - 1 ? 0 : slot + 1, last = slot == 0 ? T::R - 1 : slot - 1;
            const int dx = onward(slot, T::X), dw = wslot ? -WT : WT;
            // Sixteen slots of a step beside its products, so that none waits for
            // another's: the first half of a product's 32 clocks issues it, and four
            // instructions or so are free in the second.  Requests to LDS and memory
            // come one to a slot, or the waves' would wait in line.
            const auto step = [&](auto k, Step& d, Step& dn) {
                constexpr int ks = decltype(k)::value;
                const auto work = [&](auto at) {
                    constexpr int n = decltype(at)::value;
                    if constexpr (ks < 3) {
                        if constexpr (n < 4 + TF) read(x_at[(ks + 1) % 4], w_at[(ks + 1) % 4], dn, n);
                    } else {
                        if constexpr (n == 0) {
                            // before the last step's other products, whose operands are
                            // here: the next stage's gradients, and the codes after its
                            // own, have landed
                            wait_vmem<T::WAIT>();
                            meet();
                            for_each<4>([&](auto i) {
                                x_at[i] = held(x_at[i] + dx);
                                w_at[i] = held(w_at[i] + dw);
                            });
                        }
                        if constexpr (n > 0 && n < 5 + TF) read(x_at[0], w_at[0], dn, n - 1);
                        // the slot of the codes converted last
                        if constexpr (n >= 10 && n % 2 == 0 && n / 2 - 5 <= T::W_DMA) fetch_w(next, n / 2 - 5);
                        if constexpr (n == 15) {
                            code_at = held(code_at + onward(next, RAW));
                            scale_at = held(scale_at + onward(next, RAW_S));
                            to = held(to - dw);
                        }
                    }
                    if constexpr (ks == 0) {
                        // that of the last stage's gradients, an eighth at a time
                        constexpr int from = n / 2 * T::X_DMA / 8, end = (n / 2 + 1) * T::X_DMA / 8;
                        if constexpr (n % 2 == 0 && end > from) fetch_x(last, from, end);
                        if constexpr (n >= 7 && n < 15) raw_read(r, n - 7);
                    }
                    if constexpr (ks == 1) {
                        if constexpr (n == 3) for_each<8>([&](auto e8) { sc[e8] = mx_scale(r.s[e8]); });
                        if constexpr (F16 && n >= 8) look(r, n - 8);
                    }
                    // the conversion's units, of four pairs of columns four each: eight to a step
                    constexpr int at_unit = ks == 1 ? n - 4 : n;
                    if constexpr ((ks == 1 || ks == 2) && at_unit >= 0 && at_unit < 12 && at_unit % 3 < 2) {
                        constexpr int unit = (ks - 1) * 8 + at_unit / 3 * 2 + at_unit % 3, pair = unit / 4;
                        convert(r, sc, std::integral_constant<int, pair>{}, unit % 4, v[pair & 1]);
                        if constexpr (unit % 4 == 3) {
                            write(2 * pair, v[pair & 1][0]);
                            write(2 * pair + 1, v[pair & 1][1]);
                        }
                    }
                };
                for_each<4 * TF>([&](auto p) {
                    constexpr int P = decltype(p)::value, from = P * 4 / TF, end = (P + 1) * 4 / TF;
                    if constexpr (FAR) {
                        if constexpr (P % 4 == 0) parts(d.x[P / 4], e2[P / 4], xp);
                        acc[P % 4][P / 4] = H16<true>::mfma32(d.w[P % 4], xp[0], acc[P % 4][P / 4]);
                        acc[P % 4][P / 4] = H16<true>::mfma32(d.w[P % 4], xp[1], acc[P % 4][P / 4]);
                    } else {
                        acc[P % 4][P / 4] = H16<!F16>::mfma32(d.w[P % 4], d.x[P / 4], acc[P % 4][P / 4]);
                    }
                    for_each<end - from>([&](auto e) { work(std::integral_constant<int, from + decltype(e)::value>{}); });
                    __builtin_amdgcn_sched_barrier(0);
                });
            };
            step(std::integral_constant<int, 0>{}, d0, d1);
            step(std::integral_constant<int, 1>{}, d1, d0);
            step(std::integral_constant<int, 2>{}, d0, d1);
            step(std::integral_constant<int, 3>{}, d1, d0);
            slot = next;
            wslot ^= 1;
        }
        wait_vmem<0>();              // nothing lands in LDS that is another's by then
    };
    const int32_t* exps = c.b.exps;
    sum(std::false_type{}, c);
    if constexpr (HALF) {
        // Again in bfloat16, with the gradients in two parts and as large as they are:
        // with a token's power of two the products of large weights would pass
        // float32's range.  One such block among 2 x 11008 rows of 4096, 2048 bfloat16
        // tokens: 1330 us for 390 (3780 by loads of operands straight from memory).
        if (__syncthreads_or(left != 0)) {
            exps = nullptr;
            // the arguments are read anew: kept in registers meanwhile, scalars would
            // spill, into lanes that the loads to LDS cannot take them from in time
            const auto* again = (const __attribute__((address_space(4))) Call*)__builtin_amdgcn_kernarg_segment_ptr();
            asm volatile("" : "+s"(again));
            sum(std::true_type{}, *again);
        }
    }

    const BackArgs& a = c.b;
    const auto [n0, t0, part, first, end] = place_of<T::BT>(c);
    // Out through LDS, 32 tokens of a wave at a time, in a region of its own: 128
    // columns of a token in a row, which sixteen lanes read and store as eight each.
    // (Straight from the registers, with all types and edges unrolled 32 times,
    // the code alone took 17 us to come in.)  16-byte chunk q of token i at slot
    // q ^ (i % 16).
    meet();
    char* const own = lds + wave * (32 * 512);
#pragma unroll
    for (int j = 0; j < TF; ++j) {
#pragma unroll
        for (int g = 0; g < 4; ++g)
#pragma unroll
            for (int e = 0; e < 4; ++e) {                 // columns 4 m .. + 3 of row m = 8 g + 4 h + e
                const f32x4_t v = {acc[0][j][4 * g + e], acc[1][j][4 * g + e], acc[2][j][4 * g + e], acc[3][j][4 * g + e]};
                *(f32x4_t*)(own + i32 * 512 + 16 * ((8 * g + 4 * h + e) ^ (i32 & 15))) = v;
            }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        const int64_t col = n0 + nw + 8 * (lane & 15);
        const int m = (int)max((int64_t)0, min((int64_t)8, a.d_in - col));
#pragma unroll 1
        for (int q = 0; q < 8; ++q) {
            const int i = 4 * q + (lane >> 4);
            const int64_t t = t0 + tw + 32 * j + i;
            const f32x4_t lo = *(const f32x4_t*)(own + i * 512 + 16 * ((2 * (lane & 15)) ^ (i & 15)));
            const f32x4_t hi = *(const f32x4_t*)(own + i * 512 + 16 * ((2 * (lane & 15) + 1) ^ (i & 15)));
            float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
            if (t >= a.n_tok || m == 0) continue;
            const int e2 = exps ? exps[t] : 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = ldexpf(v[e], e2);
            if (c.joined) store8(c.sums, GPTQ_F32, ((int64_t)part * a.n_tok + t) * c.pitch + col, 8, true, v);
            else store8(a.dX, a.dx_dt, t * a.ld_dx + col, m, m == 8, v);
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
}

// dX from the parts' sums (zeros of none): four columns of a token by S threads,
// each a share of the parts, in their order, eight on their way at once; their
// sums meet in LDS.  218 parts of one token's 249 columns: 105 us by one thread
// one part after the other, 4 so.
template <int S>
__global__ __launch_bounds__(256) void mx_back_join_kernel(Call c) {
    constexpr int Q = 256 / S;
    __shared__ f32x4_t lds[S][Q];
    const BackArgs& a = c.b;
    const int64_t row = c.pitch / 4, all = a.n_tok * row;
    const int lane = threadIdx.x % Q, share = threadIdx.x / Q;
    const int first = (int)((int64_t)c.parts * share / S), end = (int)((int64_t)c.parts * (share + 1) / S);
    for (int64_t q0 = (int64_t)blockIdx.x * Q; q0 < all; q0 += (int64_t)gridDim.x * Q) {
        const int64_t q = q0 + lane;
        float v[4] = {0.f, 0.f, 0.f, 0.f};
        if (q < all) {
            const f32x4_t* s = (const f32x4_t*)c.sums + q;
            for (int p = first; p < end; p += 8) {
                f32x4_t x[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = s[min(p + e, end - 1) * all];
#pragma unroll
                for (int e = 0; e < 8; ++e)
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[i] += p + e < end ? x[e][i] : 0.0f;
            }
        }
        if constexpr (S > 1) {
            lds[share][lane] = f32x4_t{v[0], v[1], v[2], v[3]};
            __syncthreads();
            if (share == 0) {
#pragma unroll
                for (int k = 1; k < S; ++k)
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[i] += lds[k][lane][i];
            }
            __syncthreads();
        }
        if (share != 0 || q >= all) continue;
        const int64_t t = q / row, n = 4 * (q - t * row);
        if (n >= a.d_in) continue;
        put4(a.dX, a.dx_dt, t * a.ld_dx + n, (int)min((int64_t)4, a.d_in - n), v);
    }
}

// The caller's gradients as planes: padded to whole stages, on 16 bytes, and
// float32 ones cut into three bfloat16 parts.
struct Planes {
    const void* D;
    gptq_dtype dt;
    int64_t n_tok, rows, ld, pad, to;
    uint16_t* out;             // [token][plane][pad], token to token `to` elements
};
__global__ __launch_bounds__(256) void mx_planes_kernel(Planes c) {
    const int64_t k = 8 * ((int64_t)blockIdx.x * 256 + threadIdx.x);
    if (k >= c.pad) return;
    for (int64_t t = blockIdx.y; t < c.n_tok; t += gridDim.y) {
        const int n = (int)max((int64_t)0, min((int64_t)8, c.rows - k));
        if (c.dt == GPTQ_F32) {
            float v[8];
            load8_f32(c.D, GPTQ_F32, t * c.ld + k, n, n == 8, v);
            u32x4_t p[3];
            cut(v, p);
#pragma unroll
            for (int j = 0; j < 3; ++j) *(u32x4_t*)(c.out + t * c.to + j * c.pad + k) = p[j];
        } else {
            const uint16_t* d = (const uint16_t*)c.D + t * c.ld + k;
            u32x4_t w;
            if (n == 8) {
                w = *(const u32x4_any_t*)d;
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    w[i] = (2 * i < n ? d[2 * i] : 0u) | (2 * i + 1 < n ? (uint32_t)d[2 * i + 1] : 0u) << 16;
            }
            *(u32x4_t*)(c.out + t * c.to + k) = w;
        }
    }
}

// ---------------------------------------------------------------------------
// dG and dU as planes.  They are products that have more bits than their factors'
// type, and the result is not to show that they were rounded: it should be off by
// its own rounding alone.  So float32 ones are kept whole, in three bfloat16
// parts; bfloat16's in a float16 value (11 bits: 0.00171 of the result's norm, as
// of float32 ones, where bfloat16 has 0.0023), float16's in two (22 bits: 0.00021
// against 0.00029 with one).  Float16 values lack range, so each token's are
// scaled by a power of two that brings the largest finite one to 2^14 .. 2^15, for
// which a workgroup holds the token's values until it has seen them all.  Bound
// by memory: 2048 x 11008 bf16 45 us (5.0 TB/s), 300 x 2050 f16 8.6.
// ---------------------------------------------------------------------------
struct Gates {
    GatedBackArgs a;
    uint16_t* D;               // [token][matrix][plane][pad], or [plane][token][matrix][pad]
    int64_t pad, ld;           // token to token ld elements,
    int64_t matrix, plane;     // matrix to matrix and plane to plane as many as these
    int rows;                  // planes that are rows of their own
    int32_t* exps;             // of 16-bit types, for each row
};

// Eight values of both gradients from column k of a token on, of which n exist; to
// dG and dU, which may be G and U, with `out`: the last time that they are computed.
template <gptq_dtype DT, gptq_activation ACT>
__device__ __forceinline__ void gate_gradients(const Gates& c, int64_t t, int64_t k, int n, bool out, float (&g)[8], float (&u)[8]) {
    const GatedBackArgs& a = c.a;
    float dy[8], gv[8], uv[8];
    load8_f32(a.dY, DT, t * a.ld_dy + k, n, n == 8, dy);
    load8_f32(a.G, DT, t * a.ld_gu + k, n, n == 8, gv);
    load8_f32(a.U, DT, t * a.ld_gu + k, n, n == 8, uv);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float value, slope;
        activate_with_slope<DT != GPTQ_F32>(ACT, gv[i], value, slope);
        g[i] = i < n ? dy[i] * uv[i] * slope : 0.0f;      // zeros past d_ff, whatever act(0) is
        u[i] = i < n ? dy[i] * value : 0.0f;
    }
    if (out && a.dG && n > 0) {
        store8(a.dG, DT, t * a.ld_dgu + k, n, n == 8, g);
        store8(a.dU, DT, t * a.ld_dgu + k, n, n == 8, u);
    }
}

template <gptq_activation ACT>
__global__ __launch_bounds__(256) void mx_gates_f32_kernel(Gates c) {
    const int64_t k = 8 * ((int64_t)blockIdx.x * 256 + threadIdx.x);
    if (k >= c.pad) return;
    for (int64_t t = blockIdx.y; t < c.a.n_tok; t += gridDim.y) {
        const int n = (int)max((int64_t)0, min((int64_t)8, c.a.d_ff - k));
        float g[8], u[8];
        gate_gradients<GPTQ_F32, ACT>(c, t, k, n, true, g, u);
        uint16_t* to = c.D + t * c.ld + k;
        u32x4_t p[3];
        cut(g, p);
#pragma unroll
        for (int j = 0; j < 3; ++j) *(u32x4_t*)(to + j * c.plane) = p[j];
        cut(u, p);
#pragma unroll
        for (int j = 0; j < 3; ++j) *(u32x4_t*)(to + c.matrix + j * c.plane) = p[j];
    }
}

// A token by a workgroup, eight values P times a thread; P = 0: more than 2 x 1024
// x 8, taken twice.
template <gptq_dtype DT, gptq_activation ACT, int P>
__global__ __launch_bounds__(1024) void mx_gates_kernel(Gates c) {
    constexpr int PLANES = gate_planes(DT);
    __shared__ float top[16];
    const int64_t t = blockIdx.x, step = 8 * (int64_t)blockDim.x;
    const auto finite_max = [](float m, float v) { return __builtin_isfinite(v) ? fmaxf(m, fabsf(v)) : m; };
    const auto left = [&](int64_t k) { return (int)max((int64_t)0, min((int64_t)8, c.a.d_ff - k)); };
    float g[P ? P : 1][8], u[P ? P : 1][8], m = 0.0f;
    if constexpr (P > 0) {
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int64_t k = 8 * threadIdx.x + p * step;
            gate_gradients<DT, ACT>(c, t, min(k, c.a.d_ff), left(k), true, g[p], u[p]);
#pragma unroll
            for (int i = 0; i < 8; ++i) m = finite_max(finite_max(m, g[p][i]), u[p][i]);
        }
    } else {
        for (int64_t k = 8 * threadIdx.x; k < c.a.d_ff; k += step) {
            gate_gradients<DT, ACT>(c, t, k, left(k), false, g[0], u[0]);
#pragma unroll
            for (int i = 0; i < 8; ++i) m = finite_max(finite_max(m, g[0][i]), u[0][i]);
        }
    }
#pragma unroll
    for (int s = 32; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor(m, s, 64));
    if ((threadIdx.x & 63) == 0) top[threadIdx.x >> 6] = m;
    __syncthreads();
    for (int w = 0; w < (int)(blockDim.x >> 6); ++w) m = fmaxf(m, top[w]);
    int e2 = 0;
    if (m > 0.0f) {
        frexpf(m, &e2);                          // m = f 2^e2, f in [1/2, 1)
        e2 = 15 - e2;
    }
    if (threadIdx.x < c.rows) c.exps[threadIdx.x * c.a.n_tok + t] = -e2;
    const auto put = [&](int64_t at, float (&x)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = ldexpf(x[i], e2);
#pragma unroll
        for (int j = 0; j < PLANES; ++j) {
            store8(c.D, GPTQ_F16, t * c.ld + at + j * c.plane, 8, true, x);
            if (j + 1 < PLANES) {                // what the value lacks; nothing beside an infinity or NaN
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = __builtin_isfinite(x[i]) ? x[i] - (float)(_Float16)x[i] : 0.0f;
            }
        }
    };
    if constexpr (P > 0) {
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int64_t k = 8 * threadIdx.x + p * step;
            if (k >= c.pad) continue;
            put(k, g[p]);
            put(k + c.matrix, u[p]);
        }
    } else {
        for (int64_t k = 8 * threadIdx.x; k < c.pad; k += step) {
            gate_gradients<DT, ACT>(c, t, min(k, c.a.d_ff), left(k), true, g[0], u[0]);
            put(k, g[0]);
            put(k + c.matrix, u[0]);
        }
    }
}

template <gptq_dtype DT, gptq_activation ACT>
void launch_gates_of(const Gates& c, hipStream_t s) {
    const int64_t pieces = c.pad / 8;
    const unsigned n = (unsigned)c.a.n_tok;
    if (pieces <= 1024) mx_gates_kernel<DT, ACT, 1><<<n, (unsigned)(ceil_div(pieces, 64) * 64), 0, s>>>(c);
    else if (pieces <= 2048) mx_gates_kernel<DT, ACT, 2><<<n, (unsigned)(ceil_div(pieces, 128) * 64), 0, s>>>(c);
    else mx_gates_kernel<DT, ACT, 0><<<n, 1024, 0, s>>>(c);
}
template <gptq_activation ACT>
void launch_gates(const Gates& c, hipStream_t s) {
    const dim3 grid((unsigned)ceil_div(c.pad, 2048), (unsigned)std::min<int64_t>(c.a.n_tok, 65535));
    if (c.a.dt == GPTQ_F32) mx_gates_f32_kernel<ACT><<<grid, 256, 0, s>>>(c);
    else if (c.a.dt == GPTQ_F16) launch_gates_of<GPTQ_F16, ACT>(c, s);
    else launch_gates_of<GPTQ_BF16, ACT>(c, s);
}

// How a call is computed: the tile's tokens (64 TF), and the parts of the sum's
// stages, by the least of measured times.  A stage takes STAGE_US where one, half
// and all of the compute units have a tile (the chip lowers its clock as they
// run); a tile TILE_US besides, for its first stages' way in and its results' out;
// parts 3 us for the join's launch and their sums at 4.5 TB/s.  For example 2048
// tokens through 4096 rows of 11008 columns: 190 us in 473 tiles of 192 tokens
// (two rounds, the second 85 % full), 211 in 344 of 256 (34 % full); through 2 x
// 11008 rows of 4096 columns, in bfloat16: 344 us in 128 tiles of 256 and two parts,
// with their join, 443 in 176 of 192 (float16 values 360 in the former).
constexpr double STAGE_US[4][3] = {{0.73, 0.81, 0.87}, {0.89, 1.00, 1.12}, {1.04, 1.17, 1.30}, {1.22, 1.31, 1.60}};
constexpr double TILE_US[4] = {6, 9, 12, 15};
// Where float16's gradients have a second value, it is a segment of its own, or a
// token of its own behind all others (`rows` for each token), whose sums the join
// adds: free where a tile has room (24 tokens, 2 x 11008 rows of 4096: 41 us against 57).
struct Plan {
    int tf, stages, per, parts;
    int planes, rows;          // segments of one matrix; rows of D and of the sums for each token
};
void offer_plans(Plan& best, double& least, int matrices, int planes, int rows, int64_t tokens, int64_t d_in) {
    const int64_t all = (int64_t)best.stages * matrices * planes, n_tok = tokens * rows;
    for (int tf = 1; tf <= 4; ++tf) {
        const int64_t tiles = ceil_div(d_in, BN) * ceil_div(n_tok, 64 * tf);
        const double* us = STAGE_US[tf - 1];
        // more parts than make two rounds of the chip cost a join and save nothing,
        // nor do those of one stage with half of its values' bits
        const int64_t most = std::max<int64_t>(1, std::min<int64_t>(512 / tiles, planes == 2 ? all / 2 : all));
        for (int64_t want = 1, per; want <= most; want = per > 1 ? ceil_div(all, per - 1) : most + 1) {
            per = ceil_div(all, want);
            const int64_t parts = ceil_div(all, per);
            const int64_t full = tiles * parts / 256, rest = tiles * parts % 256;
            const double fill = rest / 256.0, stage = fill < 0.5 ? us[0] + 2 * fill * (us[1] - us[0]) : us[1] + (2 * fill - 1) * (us[2] - us[1]);
            const double cost = full * (per * us[2] + TILE_US[tf - 1]) + (rest ? per * stage + TILE_US[tf - 1] : 0) +
                                (parts * rows > 1 ? 3 + 4e-6 * parts * n_tok * d_in / 4.5 : 0);
            if (cost < least) {
                least = cost;
                best.tf = tf;
                best.per = (int)per;
                best.parts = (int)parts;
                best.planes = planes;
                best.rows = rows;
            }
        }
    }
}
Plan plan_of(int matrices, int planes, int64_t n_tok, int64_t d_in, int64_t rows) {
    Plan best{1, (int)ceil_div(rows, SK), 1, 0, planes, 1};
    if (rows == 0) return best;
    double least = 1e30;
    offer_plans(best, least, matrices, planes, 1, n_tok, d_in);
    if (planes == 2) offer_plans(best, least, matrices, 1, 2, n_tok, d_in);
    return best;
}

int64_t padded(int64_t rows) { return ceil_div(rows, SK) * SK; }
// elements from token to token in the planes
int64_t row_of(int64_t rows, int segments) { return padded(rows) * segments; }
int64_t pitch_of(int64_t d_in) { return ceil_div(d_in, 8) * 8; }
// bytes of the planes that a call makes of n_tok rows
size_t planes_bytes(int64_t n_tok, int64_t rows, int segments) {
    return align_up((size_t)n_tok * row_of(rows, segments) * 2, 256);
}
size_t sums_bytes(int matrices, int planes, int64_t n_tok, int64_t d_in, int64_t rows) {
    const Plan p = plan_of(matrices, planes, n_tok, d_in, rows);
    return p.parts * p.rows > 1 ? (size_t)p.parts * p.rows * n_tok * pitch_of(d_in) * sizeof(float) : 0;
}

template <bool HALF, int TF>
gptq_status launch_tile(const Call& c, hipStream_t s) {
    using T = BackTile<TF>;
    GPTQ_HIP(ensure_lds_limit((const void*)mx_back_kernel<HALF, TF>, T::BYTES));
    const int64_t tiles = ceil_div(c.b.d_in, BN) * ceil_div(c.b.n_tok, T::BT) * c.parts;
    mx_back_kernel<HALF, TF><<<(unsigned)tiles, 256, T::BYTES, s>>>(c);
    GPTQ_LAUNCH_CHECK();
    return GPTQ_OK;
}

gptq_status launch_sum(Call& c, const Plan& p, hipStream_t s) {
    BackArgs& a = c.b;
    c.w_row = mx_code_bytes(a.d_in, GPTQ_MX_FP4);
    c.s_row = mx_scale_bytes(a.d_in);
    c.planes = p.planes;
    c.stages = p.stages;
    c.per = p.per;
    c.parts = p.parts;
    c.joined = p.parts * p.rows > 1;
    c.pitch = pitch_of(a.d_in);
    if (c.parts > 0) {
        gptq_status st;
        a.n_tok *= p.rows;
        if (p.tf == 1) st = c.half ? launch_tile<true, 1>(c, s) : launch_tile<false, 1>(c, s);
        else if (p.tf == 2) st = c.half ? launch_tile<true, 2>(c, s) : launch_tile<false, 2>(c, s);
        else if (p.tf == 3) st = c.half ? launch_tile<true, 3>(c, s) : launch_tile<false, 3>(c, s);
        else st = c.half ? launch_tile<true, 4>(c, s) : launch_tile<false, 4>(c, s);
        if (st != GPTQ_OK) return st;
        a.n_tok /= p.rows;
        c.parts *= p.rows;       // the second values' sums are parts as well
    }
    if (c.parts != 1) {
        const auto groups = [&](int shares) { return (unsigned)std::min<int64_t>(ceil_div(a.n_tok * c.pitch / 4, 256 / shares), 1 << 20); };
        if (c.parts <= 8) mx_back_join_kernel<1><<<groups(1), 256, 0, s>>>(c);
        else if (c.parts <= 32) mx_back_join_kernel<4><<<groups(4), 256, 0, s>>>(c);
        else mx_back_join_kernel<16><<<groups(16), 256, 0, s>>>(c);
        GPTQ_LAUNCH_CHECK();
    }
    return GPTQ_OK;
}

}  // namespace

void mx_backward_plan(gptq_dtype dt, int matrices, int64_t n_tok, int64_t d_in, int64_t rows, int64_t* plan) {
    const Plan p = plan_of(matrices, matrices == 2 ? gate_planes(dt) : planes_of(dt), n_tok, d_in, rows);
    plan[0] = 64 * p.tf;
    plan[1] = p.parts;
}

size_t mx_backward_ws(gptq_dtype dt, int64_t n_tok, int64_t d_in, int64_t rows) {
    const int planes = planes_of(dt);
    return planes_bytes(n_tok, rows, planes) + sums_bytes(1, planes, n_tok, d_in, rows);
}

gptq_status mx_backward_launch(const BackArgs& a, const void* D, int64_t ld, void* ws, hipStream_t s) {
    Call c{};
    c.b = a;
    const int planes = planes_of(a.dt), size = a.dt == GPTQ_F32 ? 4 : 2;
    c.half = a.dt == GPTQ_F16;
    c.pad = padded(a.rows);
    c.sums = (float*)((char*)ws + planes_bytes(a.n_tok, a.rows, planes));
    const bool on16 = ((uintptr_t)D | (uintptr_t)(ld * size)) % 16 == 0;
    if (planes == 1 && on16 && a.rows % SK == 0 && ld <= (int64_t(1) << 20)) {
        c.D = (const uint16_t*)D;
        c.ld = a.n_tok == 1 ? c.pad : ld;
    } else {
        c.D = (const uint16_t*)ws;
        c.ld = row_of(a.rows, planes);
        if (a.rows > 0) {
            Planes p{D, a.dt, a.n_tok, a.rows, ld, c.pad, c.ld, (uint16_t*)ws};
            mx_planes_kernel<<<dim3((unsigned)ceil_div(c.pad, 2048), (unsigned)std::min<int64_t>(a.n_tok, 65535)), 256, 0, s>>>(p);
            GPTQ_LAUNCH_CHECK();
        }
    }
    return launch_sum(c, plan_of(1, planes, a.n_tok, a.d_in, a.rows), s);
}

// bytes of the tokens' exponents, for each of D's rows
size_t exps_bytes(gptq_dtype dt, int64_t n_tok) { return align_up(4 * (size_t)n_tok * gate_planes(dt), 256); }

size_t mx_gated_backward_ws(gptq_dtype dt, int64_t n_tok, int64_t d_in, int64_t d_ff) {
    const int planes = gate_planes(dt);
    return planes_bytes(n_tok, d_ff, 2 * planes) + exps_bytes(dt, n_tok) + sums_bytes(2, planes, n_tok, d_in, d_ff);
}

gptq_status mx_gated_backward_launch(const GatedBackArgs& a, void* ws, hipStream_t s) {
    Call c{};
    c.half = a.dt != GPTQ_F32;
    const int planes = gate_planes(a.dt);
    const Plan p = plan_of(2, planes, a.n_tok, a.d_in, a.d_ff);
    BackArgs& b = c.b;
    b.dt = a.dt;
    b.n_tok = a.n_tok;
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
    c.D = (const uint16_t*)ws;
    c.pad = padded(a.d_ff);
    c.ld = row_of(a.d_ff, 2 * p.planes);
    char* exps = (char*)ws + planes_bytes(a.n_tok, a.d_ff, 2 * planes);
    c.sums = (float*)(exps + exps_bytes(a.dt, a.n_tok));
    if (a.d_ff > 0) {
        Gates g{};
        g.a = a;
        g.D = (uint16_t*)ws;
        g.pad = c.pad;
        g.ld = c.ld;
        g.matrix = p.planes * c.pad;
        g.plane = p.rows > 1 ? a.n_tok * c.ld : c.pad;
        g.rows = p.rows;
        g.exps = c.half ? (int32_t*)exps : nullptr;
        switch (a.act) {
            case GPTQ_ACT_SILU: launch_gates<GPTQ_ACT_SILU>(g, s); break;
            case GPTQ_ACT_GELU: launch_gates<GPTQ_ACT_GELU>(g, s); break;
            case GPTQ_ACT_GELU_TANH: launch_gates<GPTQ_ACT_GELU_TANH>(g, s); break;
            default: launch_gates<GPTQ_ACT_RELU>(g, s); break;
        }
        GPTQ_LAUNCH_CHECK();
        b.exps = g.exps;
    }
    return launch_sum(c, p, s);
}

}  // namespace gptq
