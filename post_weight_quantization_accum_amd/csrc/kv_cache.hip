// Writing keys and values into the pages of a cache, and reading sequences
// back (include/gptq.h, "A paged cache of keys and values").
//
// Both move rows of head_dim values in units of eight, a lane each, which
// takes its unit of the keys and of the values: they share the place, and the
// way to it (slot or table entry, loads that wait on each other) costs as much
// as the data.  A block of 32 channels is a quad of lanes (head_dim is a
// multiple of 32), quantised as by mx_quantize_kernel.  Both are bound by
// memory, or by their launch for a handful of tokens.  Measured: 10000 rows of
// 12 heads of 64, e4m3 to float16, read back in 12.3 us (47 MB, 3.8 TB/s) and
// 16 tokens written in 4.0 us; 5800 rows of 8 heads of 128, bf16 and e2m1,
// written in 9.0 us and read back in 9.0 us (30 MB each, 3.3 TB/s).
#include "mx.hpp"

namespace gptq {
namespace {

struct Store {
    uint8_t* rows[2];      // keys, values
    uint8_t* scales[2];
    int64_t n_pages;
    FastDiv page;          // page_size
    int n_kv, d;
};

// Row number of (page, head, offset).
__device__ __forceinline__ int64_t row_of(const Store& c, int64_t page, int head, int off) {
    return (page * c.n_kv + head) * c.page.d + off;
}

struct WriteArgs {
    Store c;
    const void* X[2];
    int64_t ld[2];
    bool aligned[2];
    gptq_dtype dt;
    const int64_t* slots;
    int64_t n_units;       // tokens * units per token
    FastDiv upt, uph;      // units per token, per head
};

template <gptq_mx_format F>
__global__ __launch_bounds__(256) void cache_write_kernel(WriteArgs a) {
    const uint32_t u = blockIdx.x * 256 + threadIdx.x;
    if (u >= a.n_units) return;
    const int64_t t = div_by(u, a.upt);
    const uint32_t k = u - (uint32_t)t * a.upt.d;
    const uint32_t head = div_by(k, a.uph), c = k - head * a.uph.d;
    const int64_t slot = a.slots[t];
    // the values do not wait for the slot
    uint32_t w[2][4];      // of 16-bit rows
    float v[2][8];
#pragma unroll
    for (int m = 0; m < 2; ++m) {
        if constexpr (F == GPTQ_MX_NONE) {
            const uint16_t* p = (const uint16_t*)a.X[m] + t * a.ld[m] + 8 * k;
            if (a.aligned[m]) {
                const uint4 x = *(const uint4*)p;
                w[m][0] = x.x; w[m][1] = x.y; w[m][2] = x.z; w[m][3] = x.w;
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) w[m][i] = p[2 * i] | (uint32_t)p[2 * i + 1] << 16;
            }
        } else {
            load8_f32(a.X[m], a.dt, t * a.ld[m] + 8 * k, 8, a.aligned[m], v[m]);
        }
    }
    // a quad shares its token: it leaves or stays as one
    if (slot < 0 || slot >= a.c.n_pages * a.c.page.d) return;
    const int64_t page = slot <= (int64_t)UINT32_MAX ? div_by((uint32_t)slot, a.c.page) : slot / a.c.page.d;
    const int64_t row = row_of(a.c, page, (int)head, (int)(slot - page * a.c.page.d));
    const int64_t at = row * (a.c.d / 8) + c;
#pragma unroll
    for (int m = 0; m < 2; ++m) {
        if constexpr (F == GPTQ_MX_NONE) {
            ((uint4*)a.c.rows[m])[at] = make_uint4(w[m][0], w[m][1], w[m][2], w[m][3]);
        } else {
            uint32_t byte;
            u32x2_t code;
            quantize_block8<F>(v[m], byte, code);
            if constexpr (F == GPTQ_MX_FP4) ((uint32_t*)a.c.rows[m])[at] = code.x;
            else ((u32x2_t*)a.c.rows[m])[at] = code;
            if ((c & 3) == 0) a.c.scales[m][at >> 2] = (uint8_t)byte;
        }
    }
}

struct ReadArgs {
    Store c;
    gptq_dtype held;       // of 16-bit rows
    const int32_t* table;
    const int32_t* row_start;
    int64_t max_pages;
    int n_seq;
    void* Y[2];
    int64_t ld[2];
    bool aligned[2];
    gptq_dtype dt;
    int64_t n_units;
    FastDiv upt, uph;
};

// The last of n sequences that starts at or before row t (the first if none
// does), with its start and the next one's; the same for the whole wave, whose
// lanes look at 64 starts at a time.
struct Place {
    int seq;
    int32_t start, next;
};
__device__ __forceinline__ Place sequence_of(const int32_t* start, int n, int32_t t) {
    const int lane = threadIdx.x & 63;
    int lo = 0, span = n;
    while (span > 63) {
        const int step = (span + 62) / 63, i = lane * step;
        const int found = __popcll(__ballot(i < span && start[lo + min(i, span - 1)] <= t));
        const int at = max(found - 1, 0) * step;
        lo += at;
        span = min(step, span - at);
    }
    const int32_t mine = start[lo + min(lane, span)];            // span <= 63: the one behind them is there too
    const int at = max((int)__popcll(__ballot(lane < span && mine <= t)) - 1, 0);
    return Place{__builtin_amdgcn_readfirstlane(lo + at), __builtin_amdgcn_readlane(mine, at),
                 __builtin_amdgcn_readlane(mine, at + 1)};
}

template <gptq_mx_format F>
__global__ __launch_bounds__(256) void cache_read_kernel(ReadArgs a) {
    const uint32_t id = blockIdx.x * 256 + threadIdx.x;
    const bool is = id < a.n_units;
    const uint32_t u = is ? id : (uint32_t)a.n_units - 1u;
    const int64_t t = div_by(u, a.upt);
    const uint32_t k = u - (uint32_t)t * a.upt.d;
    const uint32_t head = div_by(k, a.uph), c = k - head * a.uph.d;
    // the sequence of the wave's first row, or one behind it
    Place p = sequence_of(a.row_start, a.n_seq, __builtin_amdgcn_readfirstlane((int)t));
    if (p.next <= t) {
        int hi = a.n_seq;
        while (hi - p.seq > 1) {
            const int mid = (p.seq + hi) >> 1;
            if (a.row_start[mid] <= t) p.seq = mid;
            else hi = mid;
        }
        p.start = a.row_start[p.seq];
        p.next = a.row_start[p.seq + 1];
    }
    if (!is || t < p.start || t >= p.next) return;
    const uint32_t pos = (uint32_t)(t - p.start);
    const uint32_t slot = div_by(pos, a.c.page);
    const int64_t page = slot < a.max_pages ? a.table[(int64_t)p.seq * a.max_pages + slot] : -1;
    float v[2][8];
    if (page < 0 || page >= a.c.n_pages) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[0][i] = v[1][i] = __uint_as_float(0x7FC00000u);
    } else {
        const int64_t row = row_of(a.c, page, (int)head, (int)(pos - slot * a.c.page.d));
        const int64_t at = row * (a.c.d / 8) + c;
        if constexpr (F == GPTQ_MX_NONE) {
#pragma unroll
            for (int m = 0; m < 2; ++m) load8_f32(a.c.rows[m], a.held, 8 * at, 8, true, v[m]);
        } else {
            u32x2_t w[2] = {{0u, 0u}, {0u, 0u}};
            uint8_t byte[2];
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                if constexpr (F == GPTQ_MX_FP4) w[m].x = ((const uint32_t*)a.c.rows[m])[at];
                else w[m] = ((const u32x2_t*)a.c.rows[m])[at];
                byte[m] = a.c.scales[m][at >> 2];
            }
#pragma unroll
            for (int m = 0; m < 2; ++m) values8<F>(w[m].x, w[m].y, byte[m], v[m]);
        }
    }
#pragma unroll
    for (int m = 0; m < 2; ++m) store8(a.Y[m], a.dt, t * a.ld[m] + 8 * k, 8, a.aligned[m], v[m]);
}

Store store_of(const gptq_kv_cache& c) {
    Store s;
    s.rows[0] = (uint8_t*)c.k;
    s.rows[1] = (uint8_t*)c.v;
    s.scales[0] = c.k_scales;
    s.scales[1] = c.v_scales;
    s.n_pages = c.n_pages;
    s.page = fast_div((uint32_t)c.page_size);
    s.n_kv = c.n_kv_heads;
    s.d = c.head_dim;
    return s;
}

bool rows_aligned(const void* p, int64_t ld, gptq_dtype dt) {
    return ((uintptr_t)p | (uintptr_t)(ld * (dt == GPTQ_F32 ? 4 : 2))) % 16 == 0;
}

template <class A>
gptq_status units(A& a, const gptq_kv_cache& c, int64_t n_rows, dim3& grid) {
    const int uph = c.head_dim / 8;
    a.upt = fast_div((uint32_t)(uph * c.n_kv_heads));
    a.uph = fast_div((uint32_t)uph);
    a.n_units = n_rows * a.upt.d;
    if (a.n_units > MAX_THREADS) return GPTQ_ERR_UNSUPPORTED;
    grid = dim3((unsigned)ceil_div(a.n_units, 256));
    return GPTQ_OK;
}

}  // namespace

gptq_status cache_write_launch(const gptq_kv_cache& c, const void* K, const void* V, gptq_dtype dt, int64_t n_tok,
                               int64_t ld_k, int64_t ld_v, const int64_t* slots, hipStream_t s) {
    WriteArgs a;
    a.c = store_of(c);
    a.X[0] = K;
    a.X[1] = V;
    a.ld[0] = ld_k;
    a.ld[1] = ld_v;
    a.aligned[0] = rows_aligned(K, ld_k, dt);
    a.aligned[1] = rows_aligned(V, ld_v, dt);
    a.dt = dt;
    a.slots = slots;
    dim3 grid;
    const gptq_status st = units(a, c, n_tok, grid);
    if (st != GPTQ_OK) return st;
    const dim3 block(256);
    switch (c.format) {
        case GPTQ_MX_FP4: hipLaunchKernelGGL(cache_write_kernel<GPTQ_MX_FP4>, grid, block, 0, s, a); break;
        case GPTQ_MX_FP8: hipLaunchKernelGGL(cache_write_kernel<GPTQ_MX_FP8>, grid, block, 0, s, a); break;
        default: hipLaunchKernelGGL(cache_write_kernel<GPTQ_MX_NONE>, grid, block, 0, s, a); break;
    }
    GPTQ_LAUNCH_CHECK();
    return GPTQ_OK;
}

gptq_status cache_read_launch(const gptq_kv_cache& c, const int32_t* table, int64_t max_pages, int64_t n_seq,
                              const int32_t* row_start, int64_t n_rows, void* K, void* V, gptq_dtype dt, int64_t ld_k,
                              int64_t ld_v, hipStream_t s) {
    ReadArgs a;
    a.c = store_of(c);
    a.held = c.dtype;
    a.table = table;
    a.row_start = row_start;
    a.max_pages = max_pages;
    a.n_seq = (int)n_seq;
    a.Y[0] = K;
    a.Y[1] = V;
    a.ld[0] = ld_k;
    a.ld[1] = ld_v;
    a.aligned[0] = rows_aligned(K, ld_k, dt);
    a.aligned[1] = rows_aligned(V, ld_v, dt);
    a.dt = dt;
    dim3 grid;
    const gptq_status st = units(a, c, n_rows, grid);
    if (st != GPTQ_OK) return st;
    const dim3 block(256);
    switch (c.format) {
        case GPTQ_MX_FP4: hipLaunchKernelGGL(cache_read_kernel<GPTQ_MX_FP4>, grid, block, 0, s, a); break;
        case GPTQ_MX_FP8: hipLaunchKernelGGL(cache_read_kernel<GPTQ_MX_FP8>, grid, block, 0, s, a); break;
        default: hipLaunchKernelGGL(cache_read_kernel<GPTQ_MX_NONE>, grid, block, 0, s, a); break;
    }
    GPTQ_LAUNCH_CHECK();
    return GPTQ_OK;
}

}  // namespace gptq
