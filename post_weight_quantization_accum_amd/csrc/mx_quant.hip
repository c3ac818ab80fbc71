// Rows of values to microscaled blocks and back (include/gptq.h,
// "Microscaled values").
//
// A lane takes eight neighbouring values, four lanes a block: the largest
// magnitude of a block is two exchanges inside a quad, the scale its exponent
// field, and the elements come out of the conversion instructions, which
// round half to even on v * 2^-e.  Both kernels are bound by memory: 4096 x
// 11008 float32 to e2m1 and back to float32 take 46 and 33 us, 385 MB in 78 us
// together (4.9 TB/s; a copy of 1 GiB reaches 5.2); 64 x 4096 bf16 takes 4.2 us
// both ways, two launches.
#include "mx.hpp"

namespace gptq {
namespace {

struct QuantArgs {
    const void* X;
    gptq_dtype dt;
    int64_t n_units;       // rows * units per row (units of 8 columns)
    FastDiv upr;           // units per padded row
    int64_t n_cols, ld_x;
    bool aligned;          // every row starts on 16 bytes
    uint8_t* codes;
    uint8_t* scales;
};

template <gptq_mx_format F>
__global__ __launch_bounds__(256) void mx_quantize_kernel(QuantArgs a) {
    const uint32_t u = blockIdx.x * 256 + threadIdx.x;
    // units per row is a multiple of 16, so a quad is wholly in or out
    if (u >= a.n_units) return;
    const uint32_t r = div_by(u, a.upr);
    const int c = (int)(u - r * a.upr.d) * 8;
    const int n = (int)min((int64_t)8, max((int64_t)0, a.n_cols - c));
    float v[8];
    load8_f32(a.X, a.dt, r * a.ld_x + c, n, a.aligned && n == 8, v);
    uint32_t byte;
    u32x2_t w;
    quantize_block8<F>(v, byte, w);
    if constexpr (F == GPTQ_MX_FP4) ((uint32_t*)a.codes)[u] = w.x;
    else ((u32x2_t*)a.codes)[u] = w;
    if ((u & 3) == 0) a.scales[u >> 2] = (uint8_t)byte;
}

struct DequantArgs {
    const uint8_t* codes;
    const uint8_t* scales;
    int64_t n_units;       // rows * units per row (units of 8 columns that exist, the last one short)
    FastDiv upr;
    int64_t upr_pad;       // units per padded row
    int64_t n_cols, ld_y;
    bool aligned;
    void* Y;
    gptq_dtype dt;
};

template <gptq_mx_format F>
__global__ __launch_bounds__(256) void mx_dequantize_kernel(DequantArgs a) {
    const uint32_t u = blockIdx.x * 256 + threadIdx.x;
    if (u >= a.n_units) return;
    const uint32_t r = div_by(u, a.upr);
    const int64_t k = u - r * a.upr.d, at = r * a.upr_pad + k;
    const int n = (int)min((int64_t)8, a.n_cols - 8 * k);
    u32x2_t w = {0u, 0u};
    if constexpr (F == GPTQ_MX_FP4) w.x = ((const uint32_t*)a.codes)[at];
    else w = ((const u32x2_t*)a.codes)[at];
    float v[8];
    values8<F>(w.x, w.y, a.scales[at >> 2], v);
    store8(a.Y, a.dt, r * a.ld_y + 8 * k, n, a.aligned && n == 8, v);
}

int64_t elem_bytes(gptq_dtype dt) { return dt == GPTQ_F32 ? 4 : 2; }

}  // namespace

gptq_status mx_quantize_launch(const void* X, gptq_dtype dt, int64_t n_rows, int64_t n_cols, int64_t ld_x,
                               gptq_mx_format f, uint8_t* codes, uint8_t* scales, hipStream_t s) {
    QuantArgs a;
    a.X = X;
    a.dt = dt;
    const int64_t upr = ceil_div(n_cols, MX_PAD) * (MX_PAD / 8);
    a.n_units = n_rows * upr;
    a.upr = fast_div((uint32_t)upr);
    a.n_cols = n_cols;
    a.ld_x = ld_x;
    a.aligned = ((uintptr_t)X | (uintptr_t)(ld_x * elem_bytes(dt))) % 16 == 0;
    a.codes = codes;
    a.scales = scales;
    if (a.n_units > MAX_THREADS) return GPTQ_ERR_UNSUPPORTED;
    const dim3 grid((unsigned)ceil_div(a.n_units, 256)), block(256);
    if (f == GPTQ_MX_FP4) hipLaunchKernelGGL(mx_quantize_kernel<GPTQ_MX_FP4>, grid, block, 0, s, a);
    else hipLaunchKernelGGL(mx_quantize_kernel<GPTQ_MX_FP8>, grid, block, 0, s, a);
    GPTQ_LAUNCH_CHECK();
    return GPTQ_OK;
}

gptq_status mx_dequantize_launch(const uint8_t* codes, const uint8_t* scales, gptq_mx_format f, int64_t n_rows,
                                 int64_t n_cols, void* Y, gptq_dtype dt, int64_t ld_y, hipStream_t s) {
    DequantArgs a;
    a.codes = codes;
    a.scales = scales;
    const int64_t upr = ceil_div(n_cols, 8);
    a.n_units = n_rows * upr;
    a.upr = fast_div((uint32_t)upr);
    a.upr_pad = ceil_div(n_cols, MX_PAD) * (MX_PAD / 8);
    a.n_cols = n_cols;
    a.ld_y = ld_y;
    a.aligned = ((uintptr_t)Y | (uintptr_t)(ld_y * elem_bytes(dt))) % 16 == 0;
    a.Y = Y;
    a.dt = dt;
    if (a.n_units > MAX_THREADS) return GPTQ_ERR_UNSUPPORTED;
    const dim3 grid((unsigned)ceil_div(a.n_units, 256)), block(256);
    if (f == GPTQ_MX_FP4) hipLaunchKernelGGL(mx_dequantize_kernel<GPTQ_MX_FP4>, grid, block, 0, s, a);
    else hipLaunchKernelGGL(mx_dequantize_kernel<GPTQ_MX_FP8>, grid, block, 0, s, a);
    GPTQ_LAUNCH_CHECK();
    return GPTQ_OK;
}

}  // namespace gptq
