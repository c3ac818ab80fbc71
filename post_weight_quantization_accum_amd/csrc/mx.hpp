// Microscaled values on gfx950: blocks of 32 e2m1 or e4m3 elements with a
// shared power of two (storage: include/gptq.h, "Microscaled values").
#pragma once

#include "internal.hpp"

namespace gptq {

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef _Float16 h16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef short s16x2_t __attribute__((ext_vector_type(2)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));

// columns of one padded storage unit, and of one block
constexpr int MX_PAD = 128, MX_BLOCK = 32;

__host__ __device__ __forceinline__ int64_t mx_code_bytes(int64_t n_cols, gptq_mx_format f) {
    return ceil_div(n_cols, MX_PAD) * (f == GPTQ_MX_FP4 ? MX_PAD / 2 : MX_PAD);
}
__host__ __device__ __forceinline__ int64_t mx_scale_bytes(int64_t n_cols) {
    return ceil_div(n_cols, MX_PAD) * (MX_PAD / MX_BLOCK);
}

// Scale byte as the float operand of the conversion instructions, which take
// its exponent field: byte 0 stands for 2^-127 although the float is 0, and
// byte 255 makes every converted value NaN.  (The tests check all codes and
// all bytes in float32, and all up to the largest that the quantiser writes in
// bfloat16 and float16.)
__device__ __forceinline__ float mx_scale(uint32_t byte) { return __uint_as_float(byte << 23); }

// One 16-bit type of activations and of the matrix cores.
template <bool BF>
struct H16;
template <>
struct H16<true> {
    static constexpr gptq_dtype DT = GPTQ_BF16;
    static constexpr uint32_t NAN2 = 0x7FC07FC0u;
    static __device__ __forceinline__ float to_f32(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
    static __device__ __forceinline__ uint32_t pack(float a, float b) {
        bf16x2_t v;
        v.x = (__bf16)a;
        v.y = (__bf16)b;
        return __builtin_bit_cast(uint32_t, v);
    }
    template <int S>
    static __device__ __forceinline__ uint32_t fp4(uint32_t w, float s) {
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, S));
    }
    template <bool HI>
    static __device__ __forceinline__ uint32_t fp8(uint32_t w, float s) {
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s, HI));
    }
    // c + the two values of w
    static __device__ __forceinline__ float add2(uint32_t w, float c) {
        return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(s16x2_t, w), __builtin_bit_cast(s16x2_t, 0x3F803F80u), c, false);
    }
    static __device__ __forceinline__ f32x4_t mfma16(u32x4_t a, u32x4_t b, f32x4_t c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                       __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
    }
    static __device__ __forceinline__ f16_t mfma32(u32x4_t a, u32x4_t b, f16_t c) {
        return mfma_32x32x16(a, b, c, (bf16x8_t*)nullptr);
    }
};
template <>
struct H16<false> {
    static constexpr gptq_dtype DT = GPTQ_F16;
    static constexpr uint32_t NAN2 = 0x7E007E00u;
    static __device__ __forceinline__ float to_f32(uint16_t b) { return (float)__builtin_bit_cast(_Float16, b); }
    static __device__ __forceinline__ uint32_t pack(float a, float b) {
        h16x2_t v;
        v.x = (_Float16)a;
        v.y = (_Float16)b;
        return __builtin_bit_cast(uint32_t, v);
    }
    template <int S>
    static __device__ __forceinline__ uint32_t fp4(uint32_t w, float s) {
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, S));
    }
    template <bool HI>
    static __device__ __forceinline__ uint32_t fp8(uint32_t w, float s) {
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, s, HI));
    }
    static __device__ __forceinline__ float add2(uint32_t w, float c) {
        return __builtin_amdgcn_fdot2(__builtin_bit_cast(h16x2_t, w), __builtin_bit_cast(h16x2_t, 0x3C003C00u), c, false);
    }
    static __device__ __forceinline__ f32x4_t mfma16(u32x4_t a, u32x4_t b, f32x4_t c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h16x8_t, a),
                                                      __builtin_bit_cast(h16x8_t, b), c, 0, 0, 0);
    }
    static __device__ __forceinline__ f16_t mfma32(u32x4_t a, u32x4_t b, f16_t c) {
        return mfma_32x32x16(a, b, c, (h16x8_t*)nullptr);
    }
};

// Eight e2m1 codes (one word, the first in the low bits) times 2^e as eight
// 16-bit values in order.
template <bool BF>
__device__ __forceinline__ u32x4_t fp4x8(uint32_t w, float s) {
    u32x4_t r;
    r.x = H16<BF>::template fp4<0>(w, s);
    r.y = H16<BF>::template fp4<1>(w, s);
    r.z = H16<BF>::template fp4<2>(w, s);
    r.w = H16<BF>::template fp4<3>(w, s);
    return r;
}
// Eight e4m3 codes (two words).
template <bool BF>
__device__ __forceinline__ u32x4_t fp8x8(uint32_t w0, uint32_t w1, float s) {
    u32x4_t r;
    r.x = H16<BF>::template fp8<false>(w0, s);
    r.y = H16<BF>::template fp8<true>(w0, s);
    r.z = H16<BF>::template fp8<false>(w1, s);
    r.w = H16<BF>::template fp8<true>(w1, s);
    return r;
}

// 16 and 8 bytes in memory that start where an element may: gfx950 takes wide
// accesses at any address (one row more of a cache for a wave of them; eight
// accesses by single elements cost five times as much).
typedef uint32_t u32x4_any_t __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2_any_t __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t u32_any_t __attribute__((aligned(2)));
typedef float f32x2_any_t __attribute__((ext_vector_type(2), aligned(4)));
typedef float f32x4_any_t __attribute__((ext_vector_type(4), aligned(4)));

// Eight consecutive elements of a row as float32; n of them exist (0..8),
// the others are 0.  vec: the whole 8 exist.
__device__ __forceinline__ void load8_f32(const void* X, gptq_dtype dt, int64_t at, int n, bool vec, float (&v)[8]) {
    if (dt == GPTQ_F32) {
        const float* p = (const float*)X + at;
        if (vec) {
            const f32x4_any_t a = *(const f32x4_any_t*)p, b = *(const f32x4_any_t*)(p + 4);
            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
            v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = i < n ? p[i] : 0.0f;
        }
        return;
    }
    const uint16_t* p = (const uint16_t*)X + at;
    uint32_t w[4];
    if (vec) {
        const u32x4_any_t a = *(const u32x4_any_t*)p;
        w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t lo = 2 * i < n ? p[2 * i] : 0, hi = 2 * i + 1 < n ? p[2 * i + 1] : 0;
            w[i] = lo | hi << 16;
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (dt == GPTQ_BF16) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        } else {
            v[2 * i] = H16<false>::to_f32((uint16_t)w[i]);
            v[2 * i + 1] = H16<false>::to_f32((uint16_t)(w[i] >> 16));
        }
    }
}

// Eight float32 values to a row of y's type, n of them (0..8).
__device__ __forceinline__ void store8(void* Y, gptq_dtype dt, int64_t at, int n, bool vec, const float (&v)[8]) {
    if (dt == GPTQ_F32) {
        float* p = (float*)Y + at;
        if (vec) {
            *(f32x4_any_t*)p = f32x4_any_t{v[0], v[1], v[2], v[3]};
            *(f32x4_any_t*)(p + 4) = f32x4_any_t{v[4], v[5], v[6], v[7]};
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < n) p[i] = v[i];
        }
        return;
    }
    uint16_t* p = (uint16_t*)Y + at;
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = dt == GPTQ_BF16 ? H16<true>::pack(v[2 * i], v[2 * i + 1]) : H16<false>::pack(v[2 * i], v[2 * i + 1]);
    if (vec) {
        *(u32x4_any_t*)p = u32x4_any_t{w[0], w[1], w[2], w[3]};
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
    }
}

// Quantises the 32-value block that four neighbouring lanes hold eight
// values of each.  All four lanes get the block's scale byte; codes: this
// lane's 4 (e2m1) or 8 (e4m3) bytes.
template <gptq_mx_format F>
__device__ __forceinline__ void quantize_block8(const float (&v)[8], uint32_t& byte, u32x2_t& codes) {
    // the bit pattern of |v| orders as |v| does, infinities and NaN on top
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    m = max(m, (uint32_t)__shfl_xor((int)m, 1, 64));
    m = max(m, (uint32_t)__shfl_xor((int)m, 2, 64));
    constexpr int TOP = F == GPTQ_MX_FP4 ? 2 : 8;
    // floor(log2 a) + 127 is a's exponent field; below 2^-126 (field 0) and
    // up to 2^(TOP - 127) the scale is at its least, 2^-127, all the same
    const int e = (int)(m >> 23);
    const bool bad = e == 255;
    byte = bad ? 255u : (uint32_t)max(e - TOP, 0);
    const float s = mx_scale(bad ? 127u : byte);
    codes = u32x2_t{0u, 0u};
    if constexpr (F == GPTQ_MX_FP4) {
        uint32_t w = 0;
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], s, 0);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], s, 1);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], s, 2);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], s, 3);
        codes.x = bad ? 0u : w;
    } else {
        // the conversion makes NaN of what rounds above 448: clamp first
        // (448 * 2^e: the exponent field moves by e, and stays in 8 .. 254)
        const float lim = __uint_as_float(__float_as_uint(448.0f) + ((byte - 127u) << 23));
        s16x2_t a = {0, 0}, b = {0, 0};
        float c[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) c[i] = __builtin_amdgcn_fmed3f(v[i], -lim, lim);
        a = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(a, c[0], c[1], s, false);
        a = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(a, c[2], c[3], s, true);
        b = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(b, c[4], c[5], s, false);
        b = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(b, c[6], c[7], s, true);
        codes.x = bad ? 0u : __builtin_bit_cast(uint32_t, a);
        codes.y = bad ? 0u : __builtin_bit_cast(uint32_t, b);
    }
}

// Eight values of codes (w0, and w1 for e4m3) and a scale byte in float32.
template <gptq_mx_format F>
__device__ __forceinline__ void values8(uint32_t w0, uint32_t w1, uint32_t byte, float (&v)[8]) {
    const float s = mx_scale(byte);
    f32x2_t p[4];
    if constexpr (F == GPTQ_MX_FP4) {
        p[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w0, s, 0);
        p[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w0, s, 1);
        p[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w0, s, 2);
        p[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w0, s, 3);
    } else {
        p[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w0, s, false);
        p[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w0, s, true);
        p[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w1, s, false);
        p[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w1, s, true);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = p[i].x;
        v[2 * i + 1] = p[i].y;
    }
}

// ---------------------------------------------------------------------------
// Memory to LDS without registers.
// ---------------------------------------------------------------------------
// Raw buffer over `bytes` bytes from p (wave-uniform); reads past them give 0.
__device__ __forceinline__ u32x4_t buffer_of(const void* p, int64_t bytes) {
    const uint64_t b = (uint64_t)(uintptr_t)p;
    u32x4_t r;
    r.x = __builtin_amdgcn_readfirstlane((uint32_t)b);
    r.y = __builtin_amdgcn_readfirstlane((uint32_t)(b >> 32) & 0xFFFFu);
    r.z = __builtin_amdgcn_readfirstlane((uint32_t)min(bytes, (int64_t)0xFFFFFFFF));
    r.w = 0x00020000u;
    asm volatile("s_nop 4" : "+s"(r));      // scalars written by the vector unit: five wait states before a load takes them
    return r;
}
// Lane l's 16 (4) bytes at buffer offset `off` land at LDS address `to` + 16 l
// (4 l).  Written as inline asm so that the compiler does not make every later
// LDS read wait for it; the kernel waits itself (wait_vmem, then a barrier).
// No register receives data; the wait state after m0 is this code's to keep.
__device__ __forceinline__ void dma_16(uint32_t to, uint32_t off, u32x4_t buf) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" : : "s"(to), "v"(off), "s"(buf) : "memory");
}
__device__ __forceinline__ void dma_4(uint32_t to, uint32_t off, u32x4_t buf) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds" : : "s"(to), "v"(off), "s"(buf) : "memory");
}
// At most N of this wave's memory loads still under way.
template <int N>
__device__ __forceinline__ void wait_vmem() {
    static_assert(N >= 0 && N < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (15 << 8) | ((N >> 4) << 14));
    asm volatile("" ::: "memory");
}
// All waves here, with their LDS reads done.
__device__ __forceinline__ void meet() {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// ---------------------------------------------------------------------------
// Launchers (arguments validated in mx_api.hip).
// ---------------------------------------------------------------------------
constexpr int64_t MAX_THREADS = (int64_t(1) << 32) - 1024;   // of a launch, its last workgroup included
gptq_status mx_quantize_launch(const void* X, gptq_dtype dt, int64_t n_rows, int64_t n_cols, int64_t ld_x,
                               gptq_mx_format f, uint8_t* codes, uint8_t* scales, hipStream_t s);
gptq_status mx_dequantize_launch(const uint8_t* codes, const uint8_t* scales, gptq_mx_format f, int64_t n_rows,
                                 int64_t n_cols, void* Y, gptq_dtype dt, int64_t ld_y, hipStream_t s);
gptq_status mx_matmul_launch(const void* X, gptq_dtype dt, int64_t n_tok, int64_t d_in, int64_t ld_x,
                             const uint8_t* codes, const uint8_t* scales, int64_t d_out, float* Y, int64_t ld_y,
                             hipStream_t s);
gptq_status mx_matmul_quantized_launch(const uint8_t* xc, const uint8_t* xs, gptq_mx_format xf, int64_t n_tok,
                                       int64_t d_in, const uint8_t* codes, const uint8_t* scales, int64_t d_out,
                                       float* Y, int64_t ld_y, hipStream_t s);
int mx_matmul_kernel(gptq_dtype dt, gptq_mx_format xf, int64_t n_tok, int64_t d_in, int64_t d_out, bool aligned);

// n / d for 32-bit n by a multiplication (d >= 1): division by invariant
// integers after Granlund and Montgomery (1994).
struct FastDiv {
    uint32_t d, mul, s1, s2;
};
inline FastDiv fast_div(uint32_t d) {
    uint32_t l = 0;
    while (l < 32 && ((uint64_t)1 << l) < d) ++l;
    FastDiv f;
    f.d = d;
    f.mul = (uint32_t)(((((uint64_t)1 << l) - d) << 32) / d + 1);
    f.s1 = l < 1 ? l : 1;
    f.s2 = l > 1 ? l - 1 : 0;
    return f;
}
__host__ __device__ __forceinline__ uint32_t div_by(uint32_t n, FastDiv f) {
    const uint32_t t = (uint32_t)(((uint64_t)n * f.mul) >> 32);
    return (t + ((n - t) >> f.s1)) >> f.s2;
}

gptq_status cache_write_launch(const gptq_kv_cache& c, const void* K, const void* V, gptq_dtype dt, int64_t n_tok,
                               int64_t ld_k, int64_t ld_v, const int64_t* slots, hipStream_t s);
gptq_status cache_read_launch(const gptq_kv_cache& c, const int32_t* table, int64_t max_pages, int64_t n_seq,
                              const int32_t* row_start, int64_t n_rows, void* K, void* V, gptq_dtype dt, int64_t ld_k,
                              int64_t ld_v, hipStream_t s);

struct AttentionShape {
    int64_t n_tok, n_heads, n_seq, max_pages, max_q, window;
};
size_t cache_attention_ws(const gptq_kv_cache& c, const AttentionShape& a);
gptq_status cache_attention_plan(const gptq_kv_cache& c, const AttentionShape& a, int64_t* plan);
gptq_status cache_attention_launch(const gptq_kv_cache& c, const AttentionShape& a, const void* Q, gptq_dtype dt,
                                   int64_t ld_q, const int32_t* q_start, const int32_t* kv_len, const int32_t* table,
                                   float scale, void* O, int64_t ld_o, void* ws, hipStream_t s);

}  // namespace gptq
