// Attention of new tokens over a paged cache (include/gptq.h,
// gptq_cache_attention).
//
// The rows of one sequence and key-value head are its tokens times the heads
// of the group, r = token * G + head, so that grouped heads share every key
// they read.  Scores are computed transposed, S^T = K Q^T: the matrix
// instruction then leaves each lane with one row's scores for a few keys,
// which is the layout in which the same lane supplies P^T to O^T = V^T P^T
// once the keys are taken in that order.  P never leaves the registers; V
// goes through LDS and comes back transposed by ds_read_b64_tr_b16.
//
// Two kernels.  cache_few_kernel: tiles of 16 rows, each wave with keys of
// its own, for sequences of few rows (decoding), which are bound by the
// cache's bytes.  cache_many_kernel: tiles of 128 rows that share tiles of 64
// keys in LDS, for chunks of a prompt, which are bound by the matrix cores
// and the exponentials.  Both can cut a tile's keys into parts (a float32
// output, a maximum and a sum per row and part) that cache_join_kernel joins.
//
// Softmax runs over the keys with a running maximum that is raised only when
// a score exceeds it by 2^8 (powers of two; raising late is a published idea):
// until then the weights are at most 2^8 (2^15 in float16, see lift()), below
// any overflow, and nothing has to be rescaled.
#include <algorithm>
#include <cmath>

#include "mx.hpp"

namespace gptq {
namespace {

constexpr int FEW_ROWS = 16, MANY_ROWS = 128;
constexpr int FEW_WAVES = 8;                      // of a few-row workgroup, each with steps of its own
// Sequences of at most this many rows go to the few-row kernel, which reads the
// cache once per 16 rows: the fewer bytes a key has, the longer that pays.
// Measured (8 kv heads of 128 channels, pages of 16; few-row / many-row kernel,
// us, for 8 x 4096, 1 x 32768 and 32 x 4096 positions; the limit is where the
// product of the three ratios passes 1):
//   16 bits 16 rows 35 / 35, 35 / 46, 103 / 123; 32 rows 44 / 36, 44 / 47, 142 / 133
//   e4m3    32 rows 31 / 34, 31 / 47,  87 / 114; 48 rows 42 / 38, 40 / 48, 126 / 96
//   e2m1    64 rows 28 / 38, 30 / 43, 106 /  91; 96 rows 52 / 43, 42 / 45, 156 / 123
constexpr int few_most(gptq_mx_format f) { return f == GPTQ_MX_FP4 ? 64 : f == GPTQ_MX_FP8 ? 32 : 16; }
constexpr int FEW_KEYS = 64, MANY_KEYS = 64;      // keys per step
constexpr int FEW_MIN = 4, MANY_MIN = 8;          // least steps per part
// Positions from here on count as past the table: keys are fetched up to two
// steps ahead of eight waves' (1100 positions), and those numbers must not pass
// 31 bits either.
constexpr int64_t POSITIONS = (int64_t(1) << 31) - 4096;
static_assert(4096 > 3 * FEW_WAVES * FEW_KEYS && 4096 > 4 * MANY_KEYS, "room for the steps ahead");
constexpr float RAISE = 8.0f;
// Float16 weights are 2^7 times as large (at most 2^15), so that those are not
// lost that are below 2^-25 of the largest, which thousands of keys of a long
// cache can be: from 2^-32 on they count.  bfloat16 has no such border.
template <bool BF>
constexpr float lift() { return BF ? 0.0f : 7.0f; }
constexpr float FAR = 256.0f;                     // an exponent of a maximum that is taken off the scores themselves
constexpr float NEG_INF = -__builtin_huge_valf();

struct AttnArgs {
    const uint8_t *K, *V, *KS, *VS;
    uint32_t n_pages;
    FastDiv page;
    int n_kv, d;
    const uint16_t* Q;
    uint16_t* O;
    int64_t ld_q, ld_o;
    bool q_aligned, o_aligned;     // rows of 16 bytes, of 8 bytes
    const int32_t *q_start, *kv_len, *table;
    int64_t max_pages;
    int cap;                       // positions that the table reaches (at most POSITIONS)
    int n_seq, n_tok;
    FastDiv group;                 // heads per key-value head
    float scale;                   // times log2(e)
    float raise;                   // 2^8 in scores before scaling
    int window;                    // 0: none
    uint32_t span;                 // keys that a token sees, itself the last
    int n_slots;                   // of the many-row kernel's tiles
    int per_seq;                   // of the few-row kernel's workgroups per sequence
    int n_split;
    int64_t rows_min, rows_max;    // of the sequences this launch takes
    float* part_o;                 // [part][part_rows][D]
    float* part_ml;                // [part][part_rows][2]
    int64_t part_rows;             // per_seq_head > 0: sequences * kv heads * per_seq_head, else tokens * heads
    int per_seq_head;              // rows that a sequence and kv head has room for
};

// A tile of rows of one sequence, and the keys that any of them attends to.
struct Tile {
    int seq, q0, row0, rows;       // first token; first row of the tile; rows of the sequence
    int first;                     // position of the sequence's first new token
    int lo, hi;                    // keys
};

__device__ __forceinline__ int clampi(int v, int lo, int hi) { return min(max(v, lo), hi); }

__device__ __forceinline__ int first_slot(const AttnArgs& a, int s, int rt) {
    const int64_t q0 = clampi(a.q_start[s], 0, a.n_tok);
    return (int)(q0 * a.group.d / rt) + s;
}

// The last of n ascending values f(i) that is at most x (-1: none), by the
// 64 lanes of a wave.
template <class Fn>
__device__ __forceinline__ int last_at_most(int n, int x, Fn f) {
    const int lane = threadIdx.x & 63;
    int lo = 0;
    while (true) {
        const int step = (n + 63) >> 6, i = lane * step;
        const uint64_t ok = __ballot(i < n && f(lo + min(i, n - 1)) <= x);
        const int c = __popcll(ok);
        if (c == 0) return -1;       // only at the first step
        lo += (c - 1) * step;
        n = min(step, n - (c - 1) * step);
        if (step == 1) return lo;
    }
}

__device__ __forceinline__ void tile_keys(const AttnArgs& a, Tile& t, int rt) {
    const int last = t.first + (int)div_by((uint32_t)min(t.row0 + rt, t.rows) - 1u, a.group);
    const int from = t.first + (int)div_by((uint32_t)t.row0, a.group);
    t.hi = clampi(last + 1, 0, a.cap);
    t.lo = a.window ? clampi(from - a.window + 1, 0, t.hi) : 0;
}

// Fills in sequence s; false where it is not this launch's.
__device__ __forceinline__ bool sequence(const AttnArgs& a, int s, Tile& t) {
    t.seq = s;
    t.q0 = clampi(a.q_start[s], 0, a.n_tok);
    const int n = clampi(a.q_start[s + 1], t.q0, a.n_tok) - t.q0;
    const int64_t rows = (int64_t)n * a.group.d;
    t.rows = (int)rows;
    t.first = max(a.kv_len[s], 0) - n;
    return rows > a.rows_min && rows <= a.rows_max;
}

// Tile of the many-row kernel's slot.
__device__ __forceinline__ bool find_tile(const AttnArgs& a, int slot, int rt, Tile& t) {
    const int s = __builtin_amdgcn_readfirstlane(last_at_most(a.n_seq, slot, [&](int i) { return first_slot(a, i, rt); }));
    if (s < 0) return false;
    const int k = __builtin_amdgcn_readfirstlane(slot - first_slot(a, s, rt));
    // (k < 0 only where q_start does not ascend: such a tile has no rows)
    if (k < 0 || !sequence(a, s, t) || (int64_t)k * rt >= t.rows) return false;
    t.row0 = k * rt;
    tile_keys(a, t, rt);
    return true;
}

// Steps in one part: the longest sequence's over the number of parts that the
// grid has room for, so that all parts of a ragged batch are equally long and
// a shorter sequence has fewer.
__device__ __forceinline__ int part_steps(const AttnArgs& a, int rt, int keys, int least, int n_split) {
    if (n_split == 1) return INT32_MAX;
    int most = 0;
    for (int i = threadIdx.x & 63; i < a.n_seq; i += 64) most = max(most, a.kv_len[i]);
#pragma unroll
    for (int i = 1; i < 64; i <<= 1) most = max(most, __shfl_xor(most, i, 64));
    most = min(most, a.cap);
    if (a.window) most = min(most, a.window + rt);      // a tile has at most rt tokens
    const int steps = most / keys + 2;                  // at least any tile's
    return max(least, (steps + n_split - 1) / n_split);
}

// Parts of a tile.
__device__ __forceinline__ int parts_of(const Tile& t, int keys, int per, int& first, int& steps) {
    first = t.lo / keys;
    steps = t.hi > t.lo ? (t.hi + keys - 1) / keys - first : 0;
    return steps > per ? (steps - 1) / per + 1 : 1;
}
__device__ __forceinline__ int part_begin(int first, int steps, int per, int part) {
    return per > steps ? first : first + part * per;
}
__device__ __forceinline__ int part_end(int first, int steps, int per, int part) {
    return per > steps || (part + 1) * per > steps ? first + steps : first + (part + 1) * per;
}

// The table's entry for a position, as it is: what it says is looked at a
// step later, when it has arrived.  (Only where the tile has keys at all.)
__device__ __forceinline__ int table_entry(const AttnArgs& a, const Tile& t, int key) {
    const uint32_t n = div_by((uint32_t)clampi(key, 0, a.cap - 1), a.page);
    return a.table[t.seq * a.max_pages + n];
}

// Row of the cache that holds a position, given its entry: -1 outside
// [lo, hi), -2 on a bad page.
__device__ __forceinline__ int cache_row(const AttnArgs& a, const Tile& t, int head, int key, int entry) {
    const uint32_t off = (uint32_t)key - div_by((uint32_t)key, a.page) * a.page.d;
    const int row = (entry * a.n_kv + head) * (int)a.page.d + (int)off;
    return key < t.lo || key >= t.hi ? -1 : (uint32_t)entry >= a.n_pages ? -2 : row;
}

// Eight elements of Q from channel c of a row of head_dim d.
__device__ __forceinline__ u32x4_t load_q(const AttnArgs& a, int64_t at, int c) {
    u32x4_t v = {0u, 0u, 0u, 0u};
    if (c < a.d) {
        const uint16_t* p = a.Q + at + c;
        if (a.q_aligned) {
            v = *(const u32x4_t*)p;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = p[2 * i] | (uint32_t)p[2 * i + 1] << 16;
        }
    }
    return v;
}

// 16 bytes of a row of values, and the scale of its block.
template <gptq_mx_format F>
struct Chunk {
    u32x4_t w;
    uint32_t s;
    // i-th group of eight as 16-bit values
    template <bool BF>
    __device__ __forceinline__ u32x4_t eight(int i) const {
        if constexpr (F == GPTQ_MX_FP4) return fp4x8<BF>(w[i], mx_scale(s));
        else if constexpr (F == GPTQ_MX_FP8) return fp8x8<BF>(w[2 * i], w[2 * i + 1], mx_scale(s));
        else return w;
    }
};

// Chunk ci of cache row `row`.  Always reads: row 0 for a negative row, the
// row's first chunk where it has none of that number.  Such a chunk is put
// right by mend() when it is used, so that nothing waits for it before.
template <gptq_mx_format F>
__device__ __forceinline__ void load_chunk(const AttnArgs& a, Chunk<F>& c, const uint8_t* rows, const uint8_t* scales,
                                           int row, int ci) {
    const int bytes = F == GPTQ_MX_FP4 ? a.d / 2 : F == GPTQ_MX_FP8 ? a.d : 2 * a.d;
    const uint32_t r = (uint32_t)max(row, 0), at = 16 * ci < bytes ? 16 * ci : 0;
    c.w = *(const u32x4_t*)(rows + (uint64_t)r * (uint32_t)bytes + at);
    if constexpr (F != GPTQ_MX_NONE) c.s = scales[(uint64_t)r * (uint32_t)(a.d >> 5) + (at >> (F == GPTQ_MX_FP4 ? 4 : 5))];
    else c.s = 0;
}

// Zeros for a chunk that is not there; for K (`nan`) NaN on a bad page.
template <gptq_mx_format F, bool BF>
__device__ __forceinline__ void mend(const AttnArgs& a, Chunk<F>& c, int row, int ci, bool nan) {
    const int bytes = F == GPTQ_MX_FP4 ? a.d / 2 : F == GPTQ_MX_FP8 ? a.d : 2 * a.d;
    if (row < 0 || 16 * ci >= bytes) {
        const bool bad = nan && row == -2;
        const uint32_t w = F == GPTQ_MX_NONE && bad ? H16<BF>::NAN2 : 0u;
        c.w = u32x4_t{w, w, w, w};
        c.s = bad ? 255u : 0u;
    }
}

template <gptq_mx_format F>
constexpr int chunks_of(int D) { return F == GPTQ_MX_FP4 ? D / 32 : F == GPTQ_MX_FP8 ? D / 16 : D / 8; }
// groups of eight per chunk
template <gptq_mx_format F>
constexpr int eights() { return F == GPTQ_MX_FP4 ? 4 : F == GPTQ_MX_FP8 ? 2 : 1; }

__device__ __forceinline__ s16x4_t tr_read(const char* p) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4_t*)(void*)p);
}

// Two transposed reads as one operand.
__device__ __forceinline__ u32x4_t tr_pair(const char* p, const char* q) {
    const u32x2_t x = __builtin_bit_cast(u32x2_t, tr_read(p)), y = __builtin_bit_cast(u32x2_t, tr_read(q));
    return u32x4_t{x.x, x.y, y.x, y.y};
}

// LDS written by some lanes of a wave and read by others of the same wave:
// the LDS unit keeps a wave's order, the compiler must too.
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// What the weights of a row lose in their exponents, exp2(x * scale - base),
// from the row's maximum m on.  Where m * scale is so large in some row that
// its rounding would show in the weights (2^-16 of them at FAR; from 2^27 on
// they would all be 0 or infinite), the wave is "far": its scores lose m before
// they are scaled, which is exact near the maximum, and base is only the lift.
template <bool BF>
__device__ __forceinline__ bool set_base(const AttnArgs& a, float m, float& base) {
    base = (m == NEG_INF ? 0.0f : m) * a.scale;
    const bool far = __any(fabsf(base) > FAR);
    base = (far ? 0.0f : base) - lift<BF>();
    return far;
}
template <int N>
__device__ __forceinline__ void near_zero(float (&x)[N], float m) {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] -= m == NEG_INF ? 0.0f : m;
}

// Infinities and NaN in V.  A weight of 0 does not keep them from a token
// that must not see their key (0 * inf).  So in the steps whose keys some
// tokens of a tile see and others do not ("mixed": at the diagonal, and at
// the window's far edge) they are taken out of V on its way to LDS, and where
// that happened patch() adds them to the outputs of the tokens that do see
// them, after those are written.
template <bool BF>
__device__ __forceinline__ bool take_out(u32x4_t& v) {
    constexpr uint32_t LO = BF ? 0x7F80u : 0x7C00u, HI = LO << 16;
    bool any = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bool lo = (v[i] & LO) == LO, hi = (v[i] & HI) == HI;
        any |= lo || hi;
        v[i] = (lo ? 0u : v[i] & 0xFFFFu) | (hi ? 0u : v[i] & 0xFFFF0000u);
    }
    return any;
}

__device__ __forceinline__ bool mixed_step(const AttnArgs& a, int key0, int keys, int pos0, int pos1) {
    return pos1 > pos0 && (key0 + keys > pos0 + 1 || (a.window != 0 && key0 <= pos1 - a.window));
}

template <gptq_mx_format F, bool BF>
__device__ float v_value(const AttnArgs& a, int row, int ch) {
    if constexpr (F == GPTQ_MX_NONE) {
        return H16<BF>::to_f32(((const uint16_t*)a.V)[(int64_t)row * a.d + ch]);
    } else {
        const float s = mx_scale(a.VS[(int64_t)row * (a.d >> 5) + (ch >> 5)]);
        uint32_t w;
        if constexpr (F == GPTQ_MX_FP8) w = H16<BF>::template fp8<false>(a.V[(int64_t)row * a.d + ch], s);
        else w = H16<BF>::template fp4<0>(a.V[(int64_t)row * (a.d >> 1) + (ch >> 1)] >> (4 * (ch & 1)), s);
        return H16<BF>::to_f32((uint16_t)w);
    }
}

template <bool BF>
__device__ __forceinline__ void store_pair(const AttnArgs& a, uint16_t* p, float v0, float v1) {
    const uint32_t x = H16<BF>::pack(v0, v1);
    if (a.o_aligned) {
        *(uint32_t*)p = x;
    } else {
        p[0] = (uint16_t)x;
        p[1] = (uint16_t)(x >> 16);
    }
}
template <bool BF>
__device__ __forceinline__ void store_out(const AttnArgs& a, uint16_t* p, float v0, float v1, float v2, float v3) {
    const uint32_t x = H16<BF>::pack(v0, v1), y = H16<BF>::pack(v2, v3);
    if (a.o_aligned) {
        *(u32x2_t*)p = u32x2_t{x, y};
    } else {
        p[0] = (uint16_t)x;
        p[1] = (uint16_t)(x >> 16);
        p[2] = (uint16_t)y;
        p[3] = (uint16_t)(y >> 16);
    }
}

// Number of a row among those that can have parts.
__device__ __forceinline__ int64_t part_row(const AttnArgs& a, const Tile& t, int head, int row, int tok, int hd) {
    return a.per_seq_head ? ((int64_t)t.seq * a.n_kv + head) * a.per_seq_head + row
                          : (int64_t)(t.q0 + tok) * (a.n_kv * (int)a.group.d) + hd;
}

// Where a row's outputs are: in O, or in the part's float32 rows.
struct Out {
    uint16_t* o;
    float* f;
};
__device__ __forceinline__ Out out_of(const AttnArgs& a, const Tile& t, int head, int row, int part, bool direct, int D) {
    const int tok = (int)div_by((uint32_t)row, a.group), g = (int)a.group.d, hd = head * g + row - tok * g;
    Out r = {nullptr, nullptr};
    if (direct) r.o = a.O + (int64_t)(t.q0 + tok) * a.ld_o + (int64_t)hd * a.d;
    else r.f = a.part_o + (part * a.part_rows + part_row(a, t, head, row, tok, hd)) * D;
    return r;
}

// The workgroup's rows rt from row0 on, steps [begin, end).
template <gptq_mx_format F, bool BF, int D>
__device__ __forceinline__ void patch(const AttnArgs& a, const Tile& t, int head, int part, bool direct, int rt, int keys,
                                   int begin, int end, int pos0, int pos1) {
    __threadfence_block();
    __syncthreads();
    for (int e = threadIdx.x; e < rt * D; e += blockDim.x) {
        const int row = t.row0 + e / D, ch = e % D;
        if (row >= t.rows || ch >= a.d) continue;
        const int pos = t.first + (int)div_by((uint32_t)row, a.group);
        float add = 0.0f;
        for (int step = begin; step < end; ++step) {
            if (!mixed_step(a, step * keys, keys, pos0, pos1)) continue;
            for (int key = step * keys; key < (step + 1) * keys; ++key) {
                if ((uint32_t)(pos - key) >= a.span || key < t.lo || key >= t.hi) continue;
                const int r = cache_row(a, t, head, key, table_entry(a, t, key));
                const float v = r >= 0 ? v_value<F, BF>(a, r, ch) : 0.0f;
                if (!__builtin_isfinite(v)) add += v;
            }
        }
        if (add != 0.0f) {       // an infinity or NaN
            const Out o = out_of(a, t, head, row, part, direct, D);
            if (direct) o.o[ch] = (uint16_t)H16<BF>::pack(H16<BF>::to_f32(o.o[ch]) + add, 0.0f);
            else o.f[ch] += add;
        }
    }
}

// ---------------------------------------------------------------------------
// Few rows: a workgroup of eight waves, each with every eighth step of 64 keys.
// A lane reads its part of a key's channels straight into the matrix operand;
// V passes through the wave's own LDS to be transposed, half a step at a time,
// so that the waves never wait for each other before the join at the end.
// Bound by the cache's bytes: 32 sequences of up to 4096 e2m1 positions, 8 kv
// heads of 128 with 4 heads each, 27.3 us (90 MB, 3.3 TB/s: the longest of the
// 256 workgroups has 1.5 times the mean); with 16 bits 85 us (4.0 TB/s); one
// sequence of 65536 e4m3 positions 31 us in 32 parts (4.5 TB/s) and 4.5 us for
// their join.  Steps of 32 keys on four waves took 43 and 77 us.
// ---------------------------------------------------------------------------
// Waves per SIMD that the registers are kept for: 16-bit rows take four times
// those of e2m1.
template <gptq_mx_format F, int D>
constexpr int few_waves() { return D == 128 || F == GPTQ_MX_NONE ? 2 : 3; }

template <gptq_mx_format F, bool BF, int D>
__global__ __launch_bounds__(64 * FEW_WAVES, (few_waves<F, D>())) void cache_few_kernel(AttnArgs a) {
    constexpr int NC = chunks_of<F>(D), E8 = eights<F>();
    constexpr int KC = NC > 4 ? NC / 4 : 1;         // 16-byte chunks per lane and key (D = 64, e2m1: half of one)
    constexpr int QC = D / 32;                      // k-steps of 32 channels
    constexpr int CT = D / 16;
    constexpr int V_ROW = 2 * D + 32;               // rows 32 bytes further in the banks: transposed reads hit all
    constexpr int WAVE_B = 32 * V_ROW;              // half a step's values at a time
    constexpr int O_ROW = D + 4;
    static_assert(FEW_ROWS * O_ROW * 4 <= WAVE_B, "a wave's outputs fit where its V tile was");
    __shared__ __attribute__((aligned(16))) char lds[FEW_WAVES * WAVE_B];
    __shared__ float ml[FEW_WAVES][FEW_ROWS][2];

    const int head = blockIdx.x % a.n_kv, rest = blockIdx.x / a.n_kv;
    const int part = rest % a.n_split, slot = rest / a.n_split;
    Tile t;
    const int per = part_steps(a, FEW_ROWS, FEW_KEYS, FEW_MIN, a.n_split);
    if (!sequence(a, slot / a.per_seq, t)) return;
    // a sequence of more rows than the caller's hint said has several tiles to a workgroup
    for (t.row0 = slot % a.per_seq * FEW_ROWS; t.row0 < t.rows; t.row0 += a.per_seq * FEW_ROWS) {
    tile_keys(a, t, FEW_ROWS);
    int step0, steps;
    const int n_parts = parts_of(t, FEW_KEYS, per, step0, steps);
    if (part >= n_parts) continue;
    const int begin = part_begin(step0, steps, per, part), end = part_end(step0, steps, per, part);

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int n = lane & 15, g = lane >> 4;
    const int row = t.row0 + n;
    const bool live = row < t.rows;
    const int tok = (int)div_by((uint32_t)row, a.group);
    const int pos = live ? t.first + tok : -1;
    const int pos0 = t.first + (int)div_by((uint32_t)t.row0, a.group);
    const int pos1 = t.first + (int)div_by((uint32_t)min(t.row0 + FEW_ROWS, t.rows) - 1u, a.group);

    // A lane holds, of keys n, 16 + n, 32 + n and 48 + n of a step, D / 4
    // channels of K and of V: element j of k-step c is channel chan(c) + j.
    const auto chan = [&](int c) {
        if constexpr (F == GPTQ_MX_NONE) return 32 * c + 8 * g;
        else return D == 128 ? 32 * g + 8 * c : 16 * g + 8 * c;
    };
    const auto chunk = [&](int i) {                 // its i-th 16 bytes
        if constexpr (F == GPTQ_MX_NONE) return 4 * i + g;
        else if constexpr (D == 64 && F == GPTQ_MX_FP4) return g >> 1;
        else return KC * g + i;
    };
    const auto piece = [&](const Chunk<F>(&x)[KC], int c) {
        if constexpr (D == 64 && F == GPTQ_MX_FP4) return fp4x8<BF>((g & 1) ? x[0].w[2 + c] : x[0].w[c], mx_scale(x[0].s));
        else return x[c / E8].template eight<BF>(c % E8);
    };
    u32x4_t q[QC];
    {
        const int64_t at = (int64_t)(t.q0 + tok) * a.ld_q + (int64_t)(head * (int)a.group.d + row - tok * (int)a.group.d) * a.d;
#pragma unroll
        for (int c = 0; c < QC; ++c) q[c] = live ? load_q(a, at, chan(c)) : u32x4_t{0u, 0u, 0u, 0u};
    }

    f32x4_t acc[CT];
#pragma unroll
    for (int i = 0; i < CT; ++i) acc[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    float m = NEG_INF, l = 0.0f, base = -lift<BF>();
    bool far = false, taken = false;
    char* const vt = lds + wave * WAVE_B;

    // Keys and values of a step, fetched while the one before is worked on: K
    // again as soon as the scores are there, V as soon as it is in LDS.
    Chunk<F> kc[4][KC], vc[4][KC];
    int row4[4];
    bool edge = false;                              // some of it is not there
    const auto entry_of = [&](int step) { return table_entry(a, t, step * FEW_KEYS + lane); };
    const auto rows_of = [&](int (&r)[4], int step, int entry) {
        const int mine = step < end ? cache_row(a, t, head, step * FEW_KEYS + lane, entry) : -1;
#pragma unroll
        for (int h = 0; h < 4; ++h) r[h] = __shfl(mine, 16 * h + n, 64);
        return a.d != D || __any(mine < 0);
    };
    const auto load = [&](Chunk<F>(&c)[KC], const uint8_t* rows, const uint8_t* scales, int r) {
#pragma unroll
        for (int i = 0; i < KC; ++i) {
            load_chunk<F>(a, c[i], rows, scales, r, chunk(i));
            if (F == GPTQ_MX_FP8 && i > 0) c[i].s = c[0].s;   // the lane's channels lie in one block
        }
    };

    int step = begin + wave, entry = 0;
    if (begin < end) {
        const int e = entry_of(step);
        entry = entry_of(step + FEW_WAVES);
        edge = rows_of(row4, step, e);
#pragma unroll
        for (int h = 0; h < 4; ++h) load(kc[h], a.K, a.KS, row4[h]);
#pragma unroll
        for (int h = 0; h < 4; ++h) load(vc[h], a.V, a.VS, row4[h]);
    }
    for (; step < end; step += FEW_WAVES) {
        const int key0 = step * FEW_KEYS;
        // the next step's rows; the table's entries for the one after it are
        // asked for first, since loads arrive in order
        int rown[4];
        const int e = entry;
        entry = entry_of(step + 2 * FEW_WAVES);
        const bool edgen = rows_of(rown, step + FEW_WAVES, e);
        if (edge) {
#pragma unroll
            for (int h = 0; h < 4; ++h)
#pragma unroll
                for (int i = 0; i < KC; ++i) mend<F, BF>(a, kc[h][i], row4[h], chunk(i), true);
        }
        // S^T: this lane gets row n, keys key0 + 16 h + 4 g + r
        f32x4_t s[4];
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            s[h] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = 0; c < QC; ++c) s[h] = H16<BF>::mfma16(piece(kc[h], c), q[c], s[h]);
        }
#pragma unroll
        for (int h = 0; h < 4; ++h) load(kc[h], a.K, a.KS, rown[h]);

        float x[16], mx = NEG_INF;
#pragma unroll
        for (int e2 = 0; e2 < 16; ++e2) x[e2] = s[e2 >> 2][e2 & 3];
        if (key0 < t.lo || key0 + FEW_KEYS > pos0 + 1 || (a.window != 0 && key0 <= pos1 - a.window)) {
            const int rel = pos - key0 - 4 * g;
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = (uint32_t)(rel - (16 * (i >> 2) + (i & 3))) < a.span ? x[i] : NEG_INF;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) mx = fmaxf(mx, x[i]);
        if (__any(mx - m > a.raise)) {
            mx = fmaxf(mx, m);
            mx = fmaxf(mx, __shfl_xor(mx, 16, 64));
            mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
            const float f = mx == NEG_INF ? 1.0f : __builtin_amdgcn_exp2f((m - mx) * a.scale);
#pragma unroll
            for (int i = 0; i < CT; ++i) acc[i] *= f;
            l *= f;
            m = mx;
            far = set_base<BF>(a, m, base);
        }
        if (far) near_zero(x, m);
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = __builtin_amdgcn_exp2f(fmaf(x[i], a.scale, -base));
        float sum = 0.0f;
        const bool mixed = mixed_step(a, key0, FEW_KEYS, pos0, pos1);
        const char* vr = vt + (4 * g + (n >> 2)) * V_ROW + 8 * (n & 3);
#pragma unroll
        for (int f = 0; f < 2; ++f) {
            // V to LDS, rows of keys
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                auto& c4 = vc[2 * f + h];
                if (edge) {
#pragma unroll
                    for (int i = 0; i < KC; ++i) mend<F, BF>(a, c4[i], row4[2 * f + h], chunk(i), false);
                }
#pragma unroll
                for (int c = 0; c < QC; ++c) {
                    u32x4_t y = piece(c4, c);
                    if (mixed) taken |= take_out<BF>(y);
                    *(u32x4_t*)(vt + (16 * h + n) * V_ROW + 2 * chan(c)) = y;
                }
                load(c4, a.V, a.VS, rown[2 * f + h]);
            }
            wave_sync();
            // the weights as the matrix operand: rounded to the 16-bit type, as V is held in it,
            // and so rounded in their sum, which gets those of a step at once (a long cache's
            // small weights one by one would not change a large sum)
            const float* w = x + 8 * f;
            const u32x4_t p = {H16<BF>::pack(w[0], w[1]), H16<BF>::pack(w[2], w[3]), H16<BF>::pack(w[4], w[5]),
                               H16<BF>::pack(w[6], w[7])};
#pragma unroll
            for (int i = 0; i < 4; ++i) sum = H16<BF>::add2(p[i], sum);
#pragma unroll
            for (int i = 0; i < CT; ++i)
                acc[i] = H16<BF>::mfma16(tr_pair(vr + 32 * i, vr + 16 * V_ROW + 32 * i), p, acc[i]);
            wave_sync();
        }
        l += sum;
        edge = edgen;
#pragma unroll
        for (int h = 0; h < 4; ++h) row4[h] = rown[h];
    }

    // join the waves
    l += __shfl_xor(l, 16, 64);
    l += __shfl_xor(l, 32, 64);
    float* const ow = (float*)vt;
#pragma unroll
    for (int i = 0; i < CT; ++i) *(f32x4_t*)(ow + n * O_ROW + 16 * i + 4 * g) = acc[i];
    if (g == 0) {
        ml[wave][n][0] = m;
        ml[wave][n][1] = l;
    }
    taken = __syncthreads_or(taken);
    constexpr int TPR = 64 * FEW_WAVES / FEW_ROWS, CH = D / TPR;   // threads of a row, channels of a thread
    const int r = threadIdx.x / TPR, c0 = (threadIdx.x % TPR) * CH;
    float mj = NEG_INF;
#pragma unroll
    for (int w = 0; w < FEW_WAVES; ++w) mj = fmaxf(mj, ml[w][r][0]);
    const float bj = mj == NEG_INF ? 0.0f : mj;
    float lj = 0.0f, o[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) o[i] = 0.0f;
#pragma unroll
    for (int w = 0; w < FEW_WAVES; ++w) {
        const float f = __builtin_amdgcn_exp2f((ml[w][r][0] - bj) * a.scale);
        lj += f * ml[w][r][1];
        const float* p = (const float*)(lds + w * WAVE_B) + r * O_ROW + c0;
#pragma unroll
        for (int i = 0; i < CH; ++i) o[i] += f * p[i];
    }
    if (t.row0 + r < t.rows) {
        const int tk = (int)div_by((uint32_t)(t.row0 + r), a.group);
        if (t.first + tk >= a.cap) {                // the table does not reach this token
            lj = __builtin_nanf("");
            mj = 0.0f;
        }
        const Out out = out_of(a, t, head, t.row0 + r, part, n_parts == 1, D);
        if (n_parts == 1) {
            const float inv = lj == 0.0f ? 0.0f : 1.0f / lj;
#pragma unroll
            for (int i = 0; i < CH; i += 2)
                if (c0 + i < a.d) store_pair<BF>(a, out.o + c0 + i, o[i] * inv, o[i + 1] * inv);
        } else {
#pragma unroll
            for (int i = 0; i < CH; i += 2) *(float2*)(out.f + c0 + i) = make_float2(o[i], o[i + 1]);
            if (threadIdx.x % TPR == 0) {
                const int64_t at = (out.f - a.part_o) / D;
                a.part_ml[2 * at] = mj;
                a.part_ml[2 * at + 1] = lj;
            }
        }
    }
    if (taken) patch<F, BF, D>(a, t, head, part, n_parts == 1, FEW_ROWS, FEW_KEYS, begin, end, pos0, pos1);
    __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// Many rows: a workgroup of four waves, each with 32 rows, over tiles of 64 keys
// that all of them share, in two LDS buffers (the next tile's keys and values
// arrive in registers while this one is worked on, and are converted once for
// 128 rows).  Bound by the matrix instructions and the weights' arithmetic,
// which overlap only between the two waves of a SIMD: the matrix cores are busy
// for 40 % of the time, LDS for 33 %, and the waves wait for 47 % of it.  2048
// tokens over 16384 16-bit positions, 8 kv heads of 128 with 4 heads each, 560
// to 610 us by card (845 to 920 TFLOP/s); e2m1 539 to 570.  Keys fetched two
// tiles ahead (no faster), and softmax of one half of a tile beside the
// products of the other (765 us: its registers spill), were tried and not kept.
// Head sizes below D run in its tiles: 32 takes as long as 64 (384 and 375 us),
// 96 as long as 128 (587 and 597), and every step of theirs mends its chunks.
// ---------------------------------------------------------------------------
template <gptq_mx_format F, bool BF, int D>
__global__ __launch_bounds__(256, 2) void cache_many_kernel(AttnArgs a) {
    constexpr int NC = chunks_of<F>(D), E8 = eights<F>();
    constexpr int PER = MANY_KEYS * NC;             // chunks of a tile of keys
    constexpr int CPT = 2 * PER / 256;              // chunks of K and V per thread
    constexpr int KPT = CPT > 1 ? CPT / 2 : 1;      // keys per thread
    constexpr int QC = D / 16, CT = D / 32;
    constexpr int K_ROW = 2 * D + 16, V_ROW = 2 * D + 64;
    constexpr int BUF = MANY_KEYS * (K_ROW + V_ROW);
    __shared__ __attribute__((aligned(16))) char lds[2 * BUF];

    const int head = blockIdx.x % a.n_kv, rest = blockIdx.x / a.n_kv;
    const int part = rest % a.n_split, slot = a.n_slots - 1 - rest / a.n_split;   // the longest tiles first
    Tile t;
    if (!find_tile(a, slot, MANY_ROWS, t)) return;
    const int per = part_steps(a, MANY_ROWS, MANY_KEYS, MANY_MIN, a.n_split);
    int step0, steps;
    const int n_parts = parts_of(t, MANY_KEYS, per, step0, steps);
    if (part >= n_parts) return;
    const int begin = part_begin(step0, steps, per, part), end = part_end(step0, steps, per, part);

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n = lane & 31, h = lane >> 5;
    const int w0 = t.row0 + 32 * wave, row = w0 + n;
    const bool live = row < t.rows;
    const int tok = (int)div_by((uint32_t)row, a.group);
    const int hd = head * (int)a.group.d + row - tok * (int)a.group.d;
    const int pos = live ? t.first + tok : -1;
    const int tile0 = t.first + (int)div_by((uint32_t)t.row0, a.group);
    const int tile1 = t.first + (int)div_by((uint32_t)min(t.row0 + MANY_ROWS, t.rows) - 1u, a.group);
    bool taken = false;
    // positions of the wave's first and last row (none: pos1 < pos0)
    const int pos0 = t.first + (int)div_by((uint32_t)w0, a.group);
    const int pos1 = w0 < t.rows ? t.first + (int)div_by((uint32_t)min(w0 + 32, t.rows) - 1u, a.group) : -1;

    u32x4_t q[QC];
    {
        const int64_t at = (int64_t)(t.q0 + tok) * a.ld_q + (int64_t)hd * a.d;
#pragma unroll
        for (int c = 0; c < QC; ++c) q[c] = live ? load_q(a, at, 16 * c + 8 * h) : u32x4_t{0u, 0u, 0u, 0u};
    }
    f16_t acc[CT];
#pragma unroll
    for (int i = 0; i < CT; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[i][e] = 0.0f;
    float m = NEG_INF, l = 0.0f, base = -lift<BF>();
    bool far = false;

    // lane l looks after key l of a step
    const auto entry_of = [&](int step) { return table_entry(a, t, step * MANY_KEYS + lane); };
    Chunk<F> c[CPT];
    int rows[KPT];
    bool edge = false;
    const auto load = [&](int step, int entry) {
        const int mine = step < end ? cache_row(a, t, head, step * MANY_KEYS + lane, entry) : -1;
        edge = a.d != D || __any(mine < 0);
#pragma unroll
        for (int i = 0; i < KPT; ++i) rows[i] = __shfl(mine, (tid + 256 * i) % PER / NC, 64);
#pragma unroll
        for (int i = 0; i < CPT; ++i) {
            const bool v = tid + 256 * i >= PER;
            load_chunk<F>(a, c[i], v ? a.V : a.K, v ? a.VS : a.KS, rows[i % KPT], (tid + 256 * i) % NC);
        }
    };
    const auto store = [&](int b, int step) {
        if (edge) {
#pragma unroll
            for (int i = 0; i < CPT; ++i)
                mend<F, BF>(a, c[i], rows[i % KPT], (tid + 256 * i) % NC, tid + 256 * i < PER);
        }
        const bool mixed = mixed_step(a, step * MANY_KEYS, MANY_KEYS, tile0, tile1);
#pragma unroll
        for (int i = 0; i < CPT; ++i) {
            const int e = tid + 256 * i, key = e % PER / NC, ci = e % NC;
            const bool v = e >= PER;
            char* p = lds + b * BUF + (v ? MANY_KEYS * K_ROW + key * V_ROW : key * K_ROW) + ci * (16 * E8);
#pragma unroll
            for (int j = 0; j < E8; ++j) {
                u32x4_t x = c[i].template eight<BF>(j);
                if (mixed && v) taken |= take_out<BF>(x);
                *(u32x4_t*)(p + 16 * j) = x;
            }
        }
    };

    int entry = 0;
    if (begin < end) {
        const int first = entry_of(begin);
        entry = entry_of(begin + 1);
        load(begin, first);
        store(0, begin);
    }
    __syncthreads();
    for (int step = begin; step < end; ++step) {
        const int b = (step - begin) & 1, key0 = step * MANY_KEYS;
        // the table's entries first: loads arrive in order, and they are wanted before the rest
        const int next = entry;
        entry = entry_of(step + 2);
        load(step + 1, next);
        const bool none = key0 > pos1 || (a.window && key0 + MANY_KEYS - 1 <= pos0 - a.window);
        if (!none) {
            const char* kt = lds + b * BUF;
            const char* vt = kt + MANY_KEYS * K_ROW;
            // S^T: this lane gets row n, keys key0 + 32 i + 8 (e / 4) + 4 h + e % 4
            __builtin_amdgcn_s_setprio(1);                  // of the two waves of a SIMD, the one with products first (573 -> 555 us)
            f16_t s[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int e = 0; e < 16; ++e) s[i][e] = 0.0f;
#pragma unroll
                for (int k = 0; k < QC; ++k)
                    s[i] = H16<BF>::mfma32(*(const u32x4_t*)(kt + (32 * i + n) * K_ROW + 32 * k + 16 * h), q[k], s[i]);
            }
            __builtin_amdgcn_s_setprio(0);
            const bool whole = key0 + MANY_KEYS <= pos0 + 1 && (a.window == 0 || key0 > pos1 - a.window);
            float x[32], mx = NEG_INF;
#pragma unroll
            for (int e = 0; e < 32; ++e) x[e] = s[e >> 4][e & 15];
            if (!whole) {
                const int rel = pos - key0 - 4 * h;
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    // selected, not assigned under a condition: hipcc (ROCm 7.2) loses the other
                    // elements of a matrix result when one of them is set in a divergent branch
                    const int o = 8 * (e >> 2) + (e & 3);
                    x[e] = (uint32_t)(rel - o) < a.span ? x[e] : NEG_INF;
                }
            }
#pragma unroll
            for (int e = 0; e < 32; ++e) mx = fmaxf(mx, x[e]);
            if (__any(mx - m > a.raise)) {
                mx = fmaxf(mx, m);
                mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
                const float f = mx == NEG_INF ? 1.0f : __builtin_amdgcn_exp2f((m - mx) * a.scale);
#pragma unroll
                for (int i = 0; i < CT; ++i)
#pragma unroll
                    for (int e = 0; e < 16; ++e) acc[i][e] *= f;
                l *= f;
                m = mx;
                far = set_base<BF>(a, m, base);
            }
            if (far) near_zero(x, m);
#pragma unroll
            for (int e = 0; e < 32; ++e) x[e] = __builtin_amdgcn_exp2f(fmaf(x[e], a.scale, -base));
            // the weights as the matrix operand: rounded to the 16-bit type, as V is held in it, and
            // so rounded in their sum (two at a time; a step's at once: a long cache's small weights
            // one by one would not change a large sum)
            u32x4_t p[4];
            float sum = 0.0f;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                p[e >> 2][e & 3] = H16<BF>::pack(x[2 * e], x[2 * e + 1]);
                sum = H16<BF>::add2(p[e >> 2][e & 3], sum);
            }
            l += sum;
            __builtin_amdgcn_s_setprio(1);
            const char* vr = vt + (4 * h + ((lane & 15) >> 2)) * V_ROW + 32 * ((lane >> 4) & 1) + 8 * (lane & 3);
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int i = 0; i < CT; ++i) {
                    const char* v = vr + 16 * k * V_ROW + 64 * i;
                    acc[i] = H16<BF>::mfma32(tr_pair(v, v + 8 * V_ROW), p[k], acc[i]);
                }
            __builtin_amdgcn_s_setprio(0);
        }
        store(b ^ 1, step + 1);
        __syncthreads();
    }
    taken = __syncthreads_or(taken);
    l += __shfl_xor(l, 32, 64);
    if (live) {
        if (pos >= a.cap) {                         // the table does not reach this token
            l = __builtin_nanf("");
            m = 0.0f;
        }
        const Out out = out_of(a, t, head, row, part, n_parts == 1, D);
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
        for (int i = 0; i < CT; ++i)
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
                const int ch = 32 * i + 2 * e + 4 * h;
                if (n_parts != 1)
                    *(float4*)(out.f + ch) = make_float4(acc[i][e], acc[i][e + 1], acc[i][e + 2], acc[i][e + 3]);
                else if (ch < a.d)
                    store_out<BF>(a, out.o + ch, acc[i][e] * inv, acc[i][e + 1] * inv, acc[i][e + 2] * inv, acc[i][e + 3] * inv);
            }
        if (n_parts != 1 && h == 0) {
            const int64_t at = (out.f - a.part_o) / D;
            a.part_ml[2 * at] = m;
            a.part_ml[2 * at + 1] = l;
        }
    }
    if (taken) patch<F, BF, D>(a, t, head, part, n_parts == 1, MANY_ROWS, MANY_KEYS, begin, end, tile0, tile1);
}

// ---------------------------------------------------------------------------
// The parts of a row joined: a workgroup per token and head, O = sum_p
// 2^((m_p - m) scale) O_p / sum_p 2^((m_p - m) scale) l_p, each wave with every
// fourth part.
// 32 rows of 32 parts take 4.5 us, most of it the launch.
// ---------------------------------------------------------------------------
struct JoinArgs {
    AttnArgs a;
    int64_t few_max;               // sequences of at most this many rows were the few-row kernel's
    int few_split, many_split;
};

// WAVES waves to a row, 4 / WAVES rows to a workgroup.
template <bool BF, int D, int WAVES>
__global__ __launch_bounds__(256) void cache_join_kernel(JoinArgs j) {
    const AttnArgs& a = j.a;
    constexpr int CH = D / 64;
    __shared__ float ow[4][D + 1];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int64_t id = (int64_t)blockIdx.x * (4 / WAVES) + wave / WAVES;
    const int heads = a.n_kv * (int)a.group.d;
    Tile t;
    int row = -1, tok = 0, hd = 0;
    if (a.per_seq_head) {          // none of the sequences of more rows has parts
        const int64_t sh = id / a.per_seq_head;
        row = (int)(id - sh * a.per_seq_head);
        const int s = (int)(sh / a.n_kv), kv = (int)(sh - (int64_t)s * a.n_kv);
        if (s >= a.n_seq) row = -1;
        else {
            sequence(a, s, t);
            if (t.rows > a.per_seq_head || row >= t.rows) row = -1;
            else {
                const int i = (int)div_by((uint32_t)row, a.group);
                tok = t.q0 + i;
                hd = kv * (int)a.group.d + row - i * (int)a.group.d;
            }
        }
    } else if (id < a.part_rows) {
        tok = (int)(id / heads);
        hd = (int)(id - (int64_t)tok * heads);
        const int s = __builtin_amdgcn_readfirstlane(last_at_most(a.n_seq, tok, [&](int i) { return a.q_start[i]; }));
        if (s >= 0) {
            sequence(a, s, t);
            const int64_t r = (int64_t)(tok - t.q0) * a.group.d + hd % a.group.d;
            if (tok >= t.q0 && r < t.rows) row = (int)r;
        }
    }
    int n = 1;
    if (row >= 0) {
        const bool few = t.rows <= j.few_max;
        const int rt = few ? FEW_ROWS : MANY_ROWS, keys = few ? FEW_KEYS : MANY_KEYS;
        t.row0 = row / rt * rt;
        tile_keys(a, t, rt);
        int first, steps;
        n = parts_of(t, keys, part_steps(a, rt, keys, few ? FEW_MIN : MANY_MIN, few ? j.few_split : j.many_split), first, steps);
    }
    // the same for all waves of a row, and of the workgroup where they meet
    if (n == 1) return;
    const float2* ml = (const float2*)a.part_ml + id;      // parts are kept in the order of the ids
    float m = NEG_INF;
    for (int p = lane; p < n; p += 64) m = fmaxf(m, ml[p * a.part_rows].x);
#pragma unroll
    for (int i = 1; i < 64; i <<= 1) m = fmaxf(m, __shfl_xor(m, i, 64));
    const float base = m == NEG_INF ? 0.0f : m;
    float l = 0.0f, o[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) o[i] = 0.0f;
#pragma unroll 8
    for (int p = wave % WAVES; p < n; p += WAVES) {
        const int64_t at = p * a.part_rows;
        const float2 v = ml[at];
        const float f = __builtin_amdgcn_exp2f((v.x - base) * a.scale);
        l += f * v.y;
#pragma unroll
        for (int i = 0; i < CH; ++i) o[i] += f * a.part_o[(at + id) * D + CH * lane + i];
    }
    if constexpr (WAVES > 1) {
#pragma unroll
        for (int i = 0; i < CH; ++i) ow[wave][CH * lane + i] = o[i];
        if (lane == 0) ow[wave][D] = l;
        __syncthreads();
        if (wave) return;
        l = ow[0][D] + ow[1][D] + ow[2][D] + ow[3][D];
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int c = CH * lane + i;
            o[i] = ow[0][c] + ow[1][c] + ow[2][c] + ow[3][c];
        }
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    uint16_t* out = a.O + (int64_t)tok * a.ld_o + (int64_t)hd * a.d + CH * lane;
#pragma unroll
    for (int i = 0; i < CH; ++i)
        if (CH * lane + i < a.d) out[i] = (uint16_t)H16<BF>::pack(o[i] * inv, 0.0f);
}

// What is launched: which sequences go to which kernel, and in how many parts.
struct Plan {
    bool few, many;
    int64_t few_most, few_max;     // rows that the few-row kernel is best at; that it takes
    int64_t few_slots, many_slots;
    int per_seq, few_split, many_split;
    int D;
    int64_t part_rows;             // as in AttnArgs; 0: no parts
    int per_seq_head;
    int join_waves;                // per row
    bool fits;                     // what is counted in 32 bits stays there
};

Plan plan_of(const gptq_kv_cache& c, const AttentionShape& s) {
    Plan p;
    const int64_t g = s.n_heads / c.n_kv_heads, rows = s.n_tok * g, most = std::max<int64_t>(1, s.max_q * g);
    p.D = c.head_dim <= 64 ? 64 : 128;
    // The hint decides only between kernels: each launch takes every sequence
    // that no other one does, however many rows it has.
    p.few_most = few_most(c.format);
    p.many = most > p.few_most;
    p.few = !(p.many && s.n_seq == 1);
    p.few_max = !p.many ? INT64_MAX : p.few ? p.few_most : -1;
    p.per_seq = (int)ceil_div(std::min(most, p.few_most), FEW_ROWS);
    p.few_slots = p.few ? s.n_seq * p.per_seq : 0;
    p.many_slots = p.many ? rows / MANY_ROWS + s.n_seq : 0;
    // Parts of the keys: as many as make the least of the time, in us, of the
    // workgroups (all taken as long as the table allows) in rounds over the
    // chip, and of joining (10, and the parts written and read).  A few-row
    // workgroup has a compute unit to itself and takes 20 bytes of the cache
    // per ns; of the other kernel two share one, 2 us a step, and one alone
    // takes 0.84 of that.  (One sequence of 16384 16-bit positions, 8 x 4
    // heads of 128: 1024 tokens in 1 part 477 us, 2 313, 3 391; 512 tokens in
    // 3 198, 4 170, 7 192; 2048 tokens in 1 567, 2 615.)  More than fill the chip
    // once are left whole, and the few-row kernel's parts fill it at most once:
    // that suits sequences of like lengths (33 of up to 4096 e2m1 positions, 8 kv
    // heads: 1 part 37 us, 4 70), not one long one among many short ones (65536
    // e4m3 positions beside 31 of 300: 522 us, alone 32).
    int64_t keys = (int64_t)c.page_size * s.max_pages;
    if (s.window) keys = std::min(keys, s.window + s.max_q);
    const int64_t key_bytes = 2 * c.head_dim * (c.format == GPTQ_MX_NONE ? 32 : c.format == GPTQ_MX_FP8 ? 17 : 9) / 16;
    const auto split = [&](double wgs, int64_t limit, int64_t least, double us, bool pairs, int64_t joined) {
        int best = 1;
        double cost = 1e300;
        if (wgs >= (pairs ? 512.0 : 256.0)) limit = 1;
        if (!pairs) limit = std::min(limit, (int64_t)(256.0 / wgs));
        for (int64_t n = 1; n <= std::max<int64_t>(1, std::min(limit, keys / least)); ++n) {
            double rounds = std::ceil(wgs * (double)n / 256.0);
            if (pairs) rounds = std::floor(rounds / 2) + (std::fmod(rounds, 2.0) != 0.0 ? 0.84 : 0.0);
            const double join = n > 1 ? 10.0 + (double)n * (double)joined * p.D * 8.0 / 4e6 : 0.0;
            const double total = us * rounds / (double)n + join;
            if (total < cost) {
                cost = total;
                best = (int)n;
            }
        }
        return best;
    };
    p.few_split = p.many_split = 1;
    const int64_t all = rows * c.n_kv_heads, few_rows = s.n_seq * c.n_kv_heads * p.few_most;
    if (p.many)
        p.many_split = split((double)((ceil_div(rows, MANY_ROWS) + (s.n_seq - 1) / 2) * c.n_kv_heads), 32,
                             MANY_KEYS * MANY_MIN, (double)keys * 2.0 / MANY_KEYS, true, all);
    // Where only the few-row kernel makes parts, and its sequences can have
    // fewer rows than there are in all, only those rows have room for them and
    // are joined (a chunk of 2048 tokens beside one decoded token, 8 x 4 heads of
    // 128, e2m1: 2 MB instead of 136 MB).
    const bool only_few = p.many && p.many_split == 1 && few_rows < all;
    if (p.few)
        p.few_split = split((double)(p.few_slots * c.n_kv_heads), 64, FEW_KEYS * FEW_MIN, (double)(keys * key_bytes) / 20e3, false,
                            only_few ? few_rows : all);
    const int parts = std::max(p.few_split, p.many_split);
    p.per_seq_head = parts > 1 && only_few ? (int)p.few_most : 0;
    p.part_rows = parts == 1 ? 0 : only_few ? few_rows : all;
    // one wave walks a few parts as fast as four do, and four rows share its workgroup
    p.join_waves = parts > 8 ? 4 : 1;
    // rows, and the threads of a launch, are counted in 32 bits
    p.fits = all <= INT32_MAX && ceil_div(p.part_rows * p.join_waves, 4) * 256 <= MAX_THREADS &&
             p.few_slots * c.n_kv_heads * p.few_split * 64 * FEW_WAVES <= MAX_THREADS &&
             p.many_slots * c.n_kv_heads * p.many_split * 256 <= MAX_THREADS;
    return p;
}

template <gptq_mx_format F, bool BF, int D>
void launch(AttnArgs& a, const Plan& p, hipStream_t s) {
    if (p.many) {
        a.n_slots = (int)p.many_slots;
        a.n_split = p.many_split;
        a.rows_min = p.few ? p.few_most : 0;
        a.rows_max = INT64_MAX;
        hipLaunchKernelGGL((cache_many_kernel<F, BF, D>), dim3((unsigned)(p.many_slots * a.n_kv * p.many_split)),
                           dim3(256), 0, s, a);
    }
    if (p.few) {
        a.per_seq = p.per_seq;
        a.n_split = p.few_split;
        a.rows_min = 0;
        a.rows_max = p.few_max;
        hipLaunchKernelGGL((cache_few_kernel<F, BF, D>), dim3((unsigned)(p.few_slots * a.n_kv * p.few_split)),
                           dim3(64 * FEW_WAVES), 0, s, a);
    }
}

template <bool BF, int D>
void launch_format(AttnArgs& a, const Plan& p, gptq_mx_format f, hipStream_t s) {
    switch (f) {
        case GPTQ_MX_FP4: launch<GPTQ_MX_FP4, BF, D>(a, p, s); break;
        case GPTQ_MX_FP8: launch<GPTQ_MX_FP8, BF, D>(a, p, s); break;
        default: launch<GPTQ_MX_NONE, BF, D>(a, p, s); break;
    }
    if (p.part_rows) {
        const JoinArgs j{a, p.few_max, p.few_split, p.many_split};
        const dim3 grid((unsigned)ceil_div(p.part_rows * p.join_waves, 4));
        if (p.join_waves == 4) hipLaunchKernelGGL((cache_join_kernel<BF, D, 4>), grid, dim3(256), 0, s, j);
        else hipLaunchKernelGGL((cache_join_kernel<BF, D, 1>), grid, dim3(256), 0, s, j);
    }
}

}  // namespace

size_t cache_attention_ws(const gptq_kv_cache& c, const AttentionShape& s) {
    const Plan p = plan_of(c, s);
    return (size_t)std::max(p.few_split, p.many_split) * (size_t)p.part_rows * (size_t)(p.D + 2) * sizeof(float);
}

gptq_status cache_attention_plan(const gptq_kv_cache& c, const AttentionShape& s, int64_t* plan) {
    const Plan p = plan_of(c, s);
    plan[0] = p.few ? p.few_split : 0;
    plan[1] = p.many ? p.many_split : 0;
    plan[2] = p.part_rows;
    return p.fits ? GPTQ_OK : GPTQ_ERR_UNSUPPORTED;
}

gptq_status cache_attention_launch(const gptq_kv_cache& c, const AttentionShape& s, const void* Q, gptq_dtype dt,
                                   int64_t ld_q, const int32_t* q_start, const int32_t* kv_len, const int32_t* table,
                                   float scale, void* O, int64_t ld_o, void* ws, hipStream_t stream) {
    const Plan p = plan_of(c, s);
    if (!p.fits) return GPTQ_ERR_UNSUPPORTED;
    AttnArgs a;
    a.K = (const uint8_t*)c.k;
    a.V = (const uint8_t*)c.v;
    a.KS = c.k_scales;
    a.VS = c.v_scales;
    a.n_pages = (uint32_t)c.n_pages;
    a.page = fast_div((uint32_t)c.page_size);
    a.n_kv = c.n_kv_heads;
    a.d = c.head_dim;
    a.Q = (const uint16_t*)Q;
    a.O = (uint16_t*)O;
    a.ld_q = ld_q;
    a.ld_o = ld_o;
    a.q_aligned = ((uintptr_t)Q | (uintptr_t)(2 * ld_q)) % 16 == 0;
    a.o_aligned = ((uintptr_t)O | (uintptr_t)(2 * ld_o)) % 8 == 0;
    a.q_start = q_start;
    a.kv_len = kv_len;
    a.table = table;
    a.max_pages = s.max_pages;
    a.cap = (int)std::min<int64_t>((int64_t)c.page_size * s.max_pages, POSITIONS);
    a.n_seq = (int)s.n_seq;
    a.n_tok = (int)s.n_tok;
    a.group = fast_div((uint32_t)(s.n_heads / c.n_kv_heads));
    a.scale = scale * 1.44269504088896340736f;
    a.raise = RAISE / a.scale;
    a.window = (int)s.window;
    a.span = s.window ? (uint32_t)s.window : 0x80000000u;
    a.part_rows = p.part_rows;
    a.per_seq_head = p.per_seq_head;
    a.part_o = (float*)ws;
    a.part_ml = p.part_rows ? a.part_o + std::max(p.few_split, p.many_split) * p.part_rows * p.D : nullptr;
    a.n_slots = a.per_seq = a.n_split = 1;
    a.rows_min = a.rows_max = 0;
    const bool bf = dt == GPTQ_BF16;
    if (p.D == 64) {
        if (bf) launch_format<true, 64>(a, p, c.format, stream);
        else launch_format<false, 64>(a, p, c.format, stream);
    } else {
        if (bf) launch_format<true, 128>(a, p, c.format, stream);
        else launch_format<false, 128>(a, p, c.format, stream);
    }
    GPTQ_LAUNCH_CHECK();
    return GPTQ_OK;
}

}  // namespace gptq
