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

// One call, as the kernels see it.  The sum runs over segments: a matrix's rows
// with one plane of the gradients (three planes where they are float32), each
// in stages of 64 rows; rows past a segment's end are zeros in both operands.
struct Call {
    BackArgs b;
    const uint16_t* D;         // planes of 16-bit values: [token][segment][pad]
    int64_t ld, pad;           // of D: token to token, segment to segment (elements, 16-byte multiples)
    int planes;                // segments of one matrix
    int64_t w_row, s_row;      // bytes per row
    int stages, per;           // stages of one segment; stages of one part
    int parts;
    float* sums;               // [part][token][d_in], of more than one part
    bool out8;                 // dX's groups of eight start on 16 bytes
};

// ---------------------------------------------------------------------------
// 256 columns x 64 TF tokens per workgroup of 2 x 2 waves, each 128 columns x
// 32 TF tokens in v_mfma_f32_32x32x16, in stages of 64 rows of the matrix.
//
// The weights' rows are the sum's index here, and a lane of the instruction
// wants eight rows of one column, while memory holds a column's rows apart.  So
// codes are turned once per workgroup, byte by byte: a thread takes eight rows
// of eight columns (eight words), and stores for each of the four bytes of a
// word (a pair of columns) its eight rows in a row.  A lane then reads the eight
// rows of four neighbouring columns as 16 bytes, converts the two columns of a
// byte with their row's scale in one instruction, and puts two rows' halves
// together with a byte permute: five instructions for four values, of which each
// wave's serve TF products.  Scale bytes are turned alike, and enter the
// conversions shifted to a float's exponent (bits beside it are ignored).
//
// Everything comes from memory to LDS without registers: gradients to a ring of
// three slots two stages ahead (16-byte chunk c of a token at slot c ^ (token %
// 8)), codes and scales as they are to another ring, three stages ahead, from
// where they are turned during the stage before theirs.  A step's operands are
// read from LDS, and its weights converted, while the one before multiplies;
// the barrier of a stage stands before its last step, whose operands are in
// registers by then, so that the matrix instructions run on behind it.
//
// Lane l ends with columns 4 m + c of its tokens (m the row of the instruction's
// result, c the column of its four): sixteen neighbours at a time.
// ---------------------------------------------------------------------------
constexpr int BN = 256, SK = 64;
constexpr int RAW = SK * BN / 2, RAW_S = SK * BN / 32;     // bytes of a stage's codes and scales
template <int TF>
struct BackTile {
    static constexpr int BT = 64 * TF, X = BT * SK * 2;
    static constexpr int CODES = 3 * X, RAWS = CODES + 2 * RAW, SCALES = RAWS + 3 * RAW, RAW_SCALES = SCALES + 2 * RAW_S;
    static constexpr int BYTES = RAW_SCALES + 3 * RAW_S;
    static constexpr int X_DMA = X / 1024 / 4, W_DMA = RAW / 1024 / 4, DMA = X_DMA + W_DMA + 1;   // per wave and stage
};

// A float whose exponent is byte E of w.
template <int E>
__device__ __forceinline__ float scale_of(uint32_t w) {
    return __uint_as_float(E == 0 ? w << 23 : E == 1 ? w << 15 : E == 2 ? w << 7 : w >> 1);
}

template <bool HALF, int TF>
__global__ __launch_bounds__(256, TF > 2 ? 1 : 2) void mx_back_kernel(Call c) {
    using T = BackTile<TF>;
    extern __shared__ __attribute__((aligned(16))) char lds[];
    const BackArgs& a = c.b;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int i32 = lane & 31, h = lane >> 5;
    // consecutive workgroups go to different dies: give each die a run of tiles
    // that share columns
    const uint32_t nt = (uint32_t)((a.n_tok + T::BT - 1) / T::BT), nn = (uint32_t)((a.d_in + BN - 1) / BN);
    const uint32_t n = gridDim.x, each = n / 8;
    const uint32_t id = blockIdx.x < each * 8 ? (blockIdx.x % 8) * each + blockIdx.x / 8 : blockIdx.x;
    const int part = (int)(id / (nt * nn));
    const int64_t n0 = (int64_t)(id / nt % nn) * BN, t0 = (int64_t)(id % nt) * T::BT;
    const int nw = 128 * (wave >> 1), tw = 32 * TF * (wave & 1);
    const int first = part * c.per, end = min(first + c.per, c.stages * a.matrices * c.planes), S = end - first;

    // this thread's pieces
    const int64_t tn = min((int64_t)T::BT, a.n_tok - t0);
    uint32_t xoff[T::X_DMA], woff[T::W_DMA], soff;
#pragma unroll
    for (int j = 0; j < T::X_DMA; ++j) {                  // eight tokens an instruction
        const int t = 8 * (wave + 4 * j) + (lane >> 3), ch = (lane & 7) ^ (t & 7);
        xoff[j] = (uint32_t)(min((int64_t)t, tn - 1) * c.ld * 2 + 16 * ch);
    }
#pragma unroll
    for (int j = 0; j < T::W_DMA; ++j) {                  // eight rows an instruction
        const int k = 8 * (wave + 4 * j) + (lane >> 3);
        const int64_t at = n0 / 2 + 16 * (lane & 7);
        woff[j] = at < c.w_row ? (uint32_t)(k * c.w_row + at) : 1u << 31;
    }
    {                                                     // 32 rows an instruction; waves 2, 3 as 0, 1
        const int k = 32 * (wave & 1) + (lane >> 1);
        const int64_t at = n0 / 32 + 4 * (lane & 1);
        soff = at < c.s_row ? (uint32_t)(k * c.s_row + at) : 1u << 31;
    }
    const uint32_t base = (uint32_t)(uintptr_t)lds;
    // segment and first row of a stage
    const auto place = [&](int f, int& seg, int64_t& k0) {
        const int st = first + min(f, S - 1);
        seg = __builtin_amdgcn_readfirstlane(st / c.stages);
        k0 = (int64_t)(st - seg * c.stages) * SK;
    };
    const auto fetch_x = [&](int f, int slot, int from, int to) {
        int seg;
        int64_t k0;
        place(f, seg, k0);
        const u32x4_t b = buffer_of(c.D + t0 * c.ld + seg * c.pad + k0, ((tn - 1) * c.ld + SK) * 2);
#pragma unroll
        for (int j = from; j < to; ++j) dma_16(base + slot * T::X + 1024 * (wave + 4 * j), xoff[j], b);
    };
    const auto fetch_w = [&](int f, int slot) {
        int seg;
        int64_t k0;
        place(f, seg, k0);
        const int m = seg / c.planes;
        const int64_t rows = min((int64_t)SK, a.rows - k0);
        const u32x4_t wb = buffer_of(a.codes[m] + k0 * c.w_row, rows * c.w_row);
        const u32x4_t sb = buffer_of(a.scales[m] + k0 * c.s_row, rows * c.s_row);
#pragma unroll
        for (int j = 0; j < T::W_DMA; ++j) dma_16(base + T::RAWS + slot * RAW + 1024 * (wave + 4 * j), woff[j], wb);
        dma_4(base + T::RAW_SCALES + slot * RAW_S + 256 * (wave & 1), soff, sb);
    };

    f16_t acc[4][TF];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < TF; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
    bool left = false;       // a block whose scale float16 lacks

    // turning: thread (q, o) has rows 8 q .. + 7 of column octet o
    const int q8 = threadIdx.x >> 5, o8 = threadIdx.x & 31;
    struct Turn {
        uint32_t w[8], s[8];
    };
    const auto turn_read = [&](int slot, Turn& r) {
        const char* w = lds + T::RAWS + slot * RAW + 8 * q8 * (BN / 2) + 4 * o8;
        const char* s = lds + T::RAW_SCALES + slot * RAW_S + 8 * q8 * (BN / 32) + (o8 >> 2);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            r.w[k] = *(const uint32_t*)(w + k * (BN / 2));
            r.s[k] = *(const uint8_t*)(s + k * (BN / 32));
        }
    };
    const auto turn_write = [&](int slot, const Turn& r) {
        if constexpr (HALF) {
#pragma unroll
            for (int k = 0; k < 8; ++k) left |= r.s[k] - 104u > 36u && (r.w[k] != 0u || r.s[k] == 255u);
        }
        // byte b of four words
        const auto four = [&](int k, auto b) {
            constexpr uint32_t B = decltype(b)::value;
            const uint32_t lo = __builtin_amdgcn_perm(r.w[k + 1], r.w[k], (4 + B) << 8 | B | 0x0C0C0000u);
            const uint32_t hi = __builtin_amdgcn_perm(r.w[k + 3], r.w[k + 2], (4 + B) << 24 | B << 16 | 0x0C0Cu);
            return lo | hi;
        };
        using B0 = std::integral_constant<uint32_t, 0>;
        using B1 = std::integral_constant<uint32_t, 1>;
        using B2 = std::integral_constant<uint32_t, 2>;
        using B3 = std::integral_constant<uint32_t, 3>;
        u32x4_t* to = (u32x4_t*)(lds + T::CODES + slot * RAW + q8 * (BN / 2 * 8) + 32 * o8);
        to[0] = u32x4_t{four(0, B0{}), four(4, B0{}), four(0, B1{}), four(4, B1{})};
        to[1] = u32x4_t{four(0, B2{}), four(4, B2{}), four(0, B3{}), four(4, B3{})};
        if ((o8 & 3) == 0) {
            u32x2_t v;
            v.x = r.s[0] | r.s[1] << 8 | r.s[2] << 16 | r.s[3] << 24;
            v.y = r.s[4] | r.s[5] << 8 | r.s[6] << 16 | r.s[7] << 24;
            *(u32x2_t*)(lds + T::SCALES + slot * RAW_S + q8 * (BN / 32 * 8) + 8 * (o8 >> 2)) = v;
        }
    };

    // a step's operands as LDS holds them
    struct Step {
        u32x4_t x[TF], w;
        u32x2_t s;
    };
    const auto read = [&](int xslot, int wslot, int ks, Step& r) {
        const int q = 2 * ks + h;
        r.w = *(const u32x4_t*)(lds + T::CODES + wslot * RAW + q * (BN / 2 * 8) + 4 * nw + 16 * i32);
        r.s = *(const u32x2_t*)(lds + T::SCALES + wslot * RAW_S + q * (BN / 32 * 8) + 8 * (nw / 32 + (i32 >> 3)));
        const char* xp = lds + xslot * T::X + (tw + i32) * (SK * 2) + 16 * (q ^ (i32 & 7));
#pragma unroll
        for (int j = 0; j < TF; ++j) r.x[j] = *(const u32x4_t*)(xp + 32 * SK * 2 * j);
    };
    // its weights: four columns of eight rows
    const auto convert = [](const Step& r, u32x4_t (&w)[4]) {
        const float s[8] = {scale_of<0>(r.s.x), scale_of<1>(r.s.x), scale_of<2>(r.s.x), scale_of<3>(r.s.x),
                            scale_of<0>(r.s.y), scale_of<1>(r.s.y), scale_of<2>(r.s.y), scale_of<3>(r.s.y)};
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int k = 0; k < 2; ++k) {                 // rows 4 k .. + 3 of a pair of columns
                const uint32_t v = r.w[2 * p + k];
                const uint32_t v0 = H16<!HALF>::template fp4<0>(v, s[4 * k]), v1 = H16<!HALF>::template fp4<1>(v, s[4 * k + 1]);
                const uint32_t v2 = H16<!HALF>::template fp4<2>(v, s[4 * k + 2]), v3 = H16<!HALF>::template fp4<3>(v, s[4 * k + 3]);
                w[2 * p][2 * k] = __builtin_amdgcn_perm(v1, v0, 0x05040100u);
                w[2 * p + 1][2 * k] = __builtin_amdgcn_perm(v1, v0, 0x07060302u);
                w[2 * p][2 * k + 1] = __builtin_amdgcn_perm(v3, v2, 0x05040100u);
                w[2 * p + 1][2 * k + 1] = __builtin_amdgcn_perm(v3, v2, 0x07060302u);
            }
    };

    fetch_w(0, 0);
    fetch_w(1, 1);
    fetch_x(0, 0, 0, T::X_DMA);
    fetch_w(2, 2);
    fetch_x(1, 1, 0, T::X_DMA);
    wait_vmem<T::DMA>();                                  // the last two are under way
    meet();
    {
        Turn r;
        turn_read(0, r);
        turn_write(0, r);
    }
    meet();
    Step d[2];
    u32x4_t w[2][4];
    read(0, 0, 0, d[0]);
    convert(d[0], w[0]);
    int xs = 0, rs = 1;          // s % 3, (s + 1) % 3
    for (int s = 0; s < S; ++s) {
        const int x1 = xs == 2 ? 0 : xs + 1, x2 = x1 == 2 ? 0 : x1 + 1;
        Turn r;
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
            if (ks == 3) {
                // before the last step, whose operands are here: the next stage's
                // gradients, and the codes after its own, have landed
                wait_vmem<T::DMA>();
                meet();
            }
            if (ks == 0) turn_read(rs, r);
            if (ks < 3) read(xs, s & 1, ks + 1, d[(ks + 1) & 1]);
            else read(x1, (s + 1) & 1, 0, d[0]);
            if (ks == 0) fetch_x(s + 2, x2, 0, T::X_DMA / 2);
            if (ks == 1) fetch_x(s + 2, x2, T::X_DMA / 2, T::X_DMA);
            if (ks == 2) fetch_w(s + 3, xs);
            if (ks == 1) turn_write((s + 1) & 1, r);
#pragma unroll
            for (int j = 0; j < TF; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[i][j] = H16<!HALF>::mfma32(w[ks & 1][i], d[ks & 1].x[j], acc[i][j]);
            convert(d[(ks + 1) & 1], w[(ks + 1) & 1]);
        }
        xs = x1;
        rs = rs == 2 ? 0 : rs + 1;
    }
    wait_vmem<0>();              // nothing lands in LDS that is another's by then

    if constexpr (HALF) {
        // again with the gradients in two bfloat16 parts, from memory directly
        if (__syncthreads_or(left)) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < TF; ++j)
#pragma unroll
                    for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
            const int64_t col = n0 + nw + 4 * i32;
            for (int st = 4 * first; st < 4 * end; ++st) {
                const int seg = st / (4 * c.stages), m = seg / c.planes;
                const int64_t k0 = (int64_t)(st - seg * 4 * c.stages) * 16 + 8 * h;
                u32x4_t v[4];
#pragma unroll
                for (int k = 0; k < 8; k += 2) {
                    uint32_t u[2][2] = {{0u, 0u}, {0u, 0u}};
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        if (k0 + k + e < a.rows && col < 2 * c.w_row) {
                            const uint32_t code = *(const uint16_t*)(a.codes[m] + (k0 + k + e) * c.w_row + col / 2);
                            const float sc = mx_scale(a.scales[m][(k0 + k + e) * c.s_row + col / 32]);
                            u[e][0] = H16<true>::fp4<0>(code, sc);
                            u[e][1] = H16<true>::fp4<1>(code, sc);
                        }
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
                        v[2 * p][k / 2] = __builtin_amdgcn_perm(u[1][p], u[0][p], 0x05040100u);
                        v[2 * p + 1][k / 2] = __builtin_amdgcn_perm(u[1][p], u[0][p], 0x07060302u);
                    }
                }
#pragma unroll
                for (int j = 0; j < TF; ++j) {
                    const int64_t t = min(t0 + tw + 32 * j + i32, a.n_tok - 1);
                    const u32x4_t x = *(const u32x4_t*)(c.D + t * c.ld + seg * c.pad + k0);
                    float f[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) f[e] = H16<false>::to_f32((uint16_t)(x[e >> 1] >> (16 * (e & 1))));
                    u32x4_t p[2];
                    cut(f, p);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        acc[i][j] = H16<true>::mfma32(v[i], p[0], acc[i][j]);
                        acc[i][j] = H16<true>::mfma32(v[i], p[1], acc[i][j]);
                    }
                }
            }
        }
    }

#pragma unroll
    for (int j = 0; j < TF; ++j) {
        const int64_t t = t0 + tw + 32 * j + i32;
        if (t >= a.n_tok) continue;
        const int e2 = a.exps && c.parts == 1 ? a.exps[t] : 0;
#pragma unroll
        for (int g = 0; g < 4; ++g)
#pragma unroll
            for (int o = 0; o < 2; ++o) {                 // eight of a group's sixteen columns
                const int64_t col = n0 + nw + 32 * g + 16 * h + 8 * o;
                if (col >= a.d_in) continue;
                const int m = (int)min((int64_t)8, a.d_in - col);
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = acc[e & 3][j][4 * g + 2 * o + (e >> 2)];
                if (c.parts > 1) {
                    store8(c.sums, GPTQ_F32, ((int64_t)part * a.n_tok + t) * a.d_in + col, m, m == 8 && a.d_in % 4 == 0, v);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] = ldexpf(v[e], e2);
                    store8(a.dX, a.dx_dt, t * a.ld_dx + col, m, c.out8 && m == 8, v);
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
    put4(a.dX, a.dx_dt, c.out8 && m == 4, t * a.ld_dx + n, m, v);
}

// The caller's gradients as planes: padded to whole stages, on 16 bytes, and
// float32 ones cut into three bfloat16 parts.
struct Planes {
    const void* D;
    gptq_dtype dt;
    int64_t n_tok, rows, ld, pad;
    uint16_t* out;             // [token][plane][pad]
    bool vec;
};
__global__ __launch_bounds__(256) void mx_planes_kernel(Planes c) {
    const int64_t k = 8 * ((int64_t)blockIdx.x * 256 + threadIdx.x);
    if (k >= c.pad) return;
    for (int64_t t = blockIdx.y; t < c.n_tok; t += gridDim.y) {
        const int n = (int)max((int64_t)0, min((int64_t)8, c.rows - k));
        if (c.dt == GPTQ_F32) {
            float v[8];
            load8_f32(c.D, GPTQ_F32, t * c.ld + k, n, c.vec && n == 8, v);
            u32x4_t p[3];
            cut(v, p);
#pragma unroll
            for (int j = 0; j < 3; ++j) *(u32x4_t*)(c.out + (t * 3 + j) * c.pad + k) = p[j];
        } else {
            const uint16_t* d = (const uint16_t*)c.D + t * c.ld + k;
            u32x4_t w;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = (2 * i < n ? d[2 * i] : 0u) | (2 * i + 1 < n ? (uint32_t)d[2 * i + 1] : 0u) << 16;
            *(u32x4_t*)(c.out + t * c.pad + k) = w;
        }
    }
}

// ---------------------------------------------------------------------------
// A token's dG and dU.  One workgroup a token, which looks for its largest
// finite value first and scales by a power of two; float32 ones are kept as
// they are.
// ---------------------------------------------------------------------------
struct Gates {
    GatedBackArgs a;
    uint16_t* D;               // [token][2][pad] float16, or [token][2][3][pad] bfloat16 parts of float32 ones
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
        if (c.exps) {
            store8(c.D, GPTQ_F16, t * 2 * c.pad + k, 8, true, g);
            store8(c.D, GPTQ_F16, (t * 2 + 1) * c.pad + k, 8, true, u);
        } else {
            u32x4_t p[3];
            cut(g, p);
#pragma unroll
            for (int j = 0; j < 3; ++j) *(u32x4_t*)(c.D + (t * 6 + j) * c.pad + k) = p[j];
            cut(u, p);
#pragma unroll
            for (int j = 0; j < 3; ++j) *(u32x4_t*)(c.D + (t * 6 + 3 + j) * c.pad + k) = p[j];
        }
    }
}

// How a call is computed: the tile's tokens, and the parts of the sum's stages.
struct Plan {
    int tf, stages, per, parts;
};
Plan plan_of(int segments, int64_t n_tok, int64_t d_in, int64_t rows) {
    Plan p;
    p.tf = n_tok <= 64 ? 1 : n_tok <= 128 ? 2 : 4;
    p.stages = (int)ceil_div(rows, SK);
    const int64_t tiles = ceil_div(d_in, BN) * ceil_div(n_tok, 64 * p.tf), all = (int64_t)p.stages * segments;
    const int64_t fill = p.tf < 4 ? 512 : 256;
    const int64_t want = std::max<int64_t>(1, std::min<int64_t>(fill / tiles, all / 4));
    p.per = (int)std::max<int64_t>(1, ceil_div(all, want));
    p.parts = (int)ceil_div(all, p.per);
    return p;
}

int64_t padded(int64_t rows) { return ceil_div(rows, SK) * SK; }
// bytes of the planes that a call makes of n_tok rows
size_t planes_bytes(int64_t n_tok, int64_t rows, int segments) {
    return align_up((size_t)n_tok * segments * padded(rows) * 2, 256);
}
size_t sums_bytes(int segments, int64_t n_tok, int64_t d_in, int64_t rows) {
    const Plan p = plan_of(segments, n_tok, d_in, rows);
    return p.parts > 1 ? (size_t)p.parts * n_tok * d_in * sizeof(float) : 0;
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

gptq_status launch_sum(Call& c, int segments, hipStream_t s) {
    const BackArgs& a = c.b;
    const Plan p = plan_of(segments, a.n_tok, a.d_in, a.rows);
    const int size = a.dx_dt == GPTQ_F32 ? 4 : 2;
    c.planes = segments / a.matrices;
    c.w_row = mx_code_bytes(a.d_in, GPTQ_MX_FP4);
    c.s_row = mx_scale_bytes(a.d_in);
    c.stages = p.stages;
    c.per = p.per;
    c.parts = p.parts;
    c.out8 = ((uintptr_t)a.dX | (uintptr_t)(a.ld_dx * size)) % 16 == 0;
    if (c.parts > 0) {
        const bool half = a.dt == GPTQ_F16;
        gptq_status st;
        if (p.tf == 1) st = half ? launch_tile<true, 1>(c, s) : launch_tile<false, 1>(c, s);
        else if (p.tf == 2) st = half ? launch_tile<true, 2>(c, s) : launch_tile<false, 2>(c, s);
        else st = half ? launch_tile<true, 4>(c, s) : launch_tile<false, 4>(c, s);
        if (st != GPTQ_OK) return st;
    }
    if (c.parts != 1) {
        for (int64_t t = 0; t < a.n_tok; t += 65535) {
            Call j = c;
            const int64_t n = std::min<int64_t>(65535, a.n_tok - t);
            j.b.dX = (char*)a.dX + t * a.ld_dx * size;
            if (j.sums) j.sums += t * a.d_in;
            if (a.exps) j.b.exps += t;
            mx_back_join_kernel<<<dim3((unsigned)ceil_div(a.d_in, 1024), (unsigned)n), 256, 0, s>>>(j);
            GPTQ_LAUNCH_CHECK();
        }
    }
    return GPTQ_OK;
}

}  // namespace

size_t mx_backward_ws(gptq_dtype dt, int64_t n_tok, int64_t d_in, int64_t rows) {
    const int planes = dt == GPTQ_F32 ? 3 : 1;
    return planes_bytes(n_tok, rows, planes) + sums_bytes(planes, n_tok, d_in, rows);
}

gptq_status mx_backward_launch(const BackArgs& a, const void* D, int64_t ld, void* ws, hipStream_t s) {
    Call c{};
    c.b = a;
    const int planes = a.dt == GPTQ_F32 ? 3 : 1, size = a.dt == GPTQ_F32 ? 4 : 2;
    c.pad = padded(a.rows);
    c.sums = (float*)((char*)ws + planes_bytes(a.n_tok, a.rows, planes));
    const bool on16 = ((uintptr_t)D | (uintptr_t)(ld * size)) % 16 == 0;
    if (planes == 1 && on16 && a.rows % SK == 0 && ld <= (int64_t(1) << 20)) {
        c.D = (const uint16_t*)D;
        c.ld = a.n_tok == 1 ? c.pad : ld;
    } else {
        c.D = (const uint16_t*)ws;
        c.ld = planes * c.pad;
        if (a.rows > 0) {
            Planes p{D, a.dt, a.n_tok, a.rows, ld, c.pad, (uint16_t*)ws, on16};
            mx_planes_kernel<<<dim3((unsigned)ceil_div(c.pad, 2048), (unsigned)std::min<int64_t>(a.n_tok, 65535)), 256, 0, s>>>(p);
            GPTQ_LAUNCH_CHECK();
        }
    }
    return launch_sum(c, planes, s);
}

size_t mx_gated_backward_ws(gptq_dtype dt, int64_t n_tok, int64_t d_in, int64_t d_ff) {
    const int segments = dt == GPTQ_F32 ? 6 : 2;
    return planes_bytes(n_tok, d_ff, segments) + align_up(4 * (size_t)n_tok, 256) + sums_bytes(segments, n_tok, d_in, d_ff);
}

gptq_status mx_gated_backward_launch(const GatedBackArgs& a, void* ws, hipStream_t s) {
    const bool wide = a.dt == GPTQ_F32;
    const int size = wide ? 4 : 2, segments = wide ? 6 : 2;
    Call c{};
    BackArgs& b = c.b;
    b.dt = wide ? GPTQ_F32 : GPTQ_F16;
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
    c.ld = segments * c.pad;
    char* exps = (char*)ws + planes_bytes(a.n_tok, a.d_ff, segments);
    c.sums = (float*)(exps + align_up(4 * (size_t)a.n_tok, 256));
    if (a.d_ff > 0) {
        Gates g{};
        g.a = a;
        g.D = (uint16_t*)ws;
        g.pad = c.pad;
        g.exps = wide ? nullptr : (int32_t*)exps;
        const auto fits = [&](const void* p, int64_t ld) { return ((uintptr_t)p | (uintptr_t)(ld * size)) % 16 == 0; };
        g.vec = fits(a.dY, a.ld_dy) && fits(a.G, a.ld_gu) && fits(a.U, a.ld_gu);
        g.vec_out = a.dG && fits(a.dG, a.ld_dgu) && fits(a.dU, a.ld_dgu);
        mx_gates_kernel<<<(unsigned)a.n_tok, 256, 0, s>>>(g);
        GPTQ_LAUNCH_CHECK();
        b.exps = g.exps;
    }
    return launch_sum(c, segments, s);
}

}  // namespace gptq
