// Writing context rows into the 4-bit cache and reading them back.
//
// Append, per 16 dimensions x of one token and K/V head (a group):
//   s = max(2^-9, e4m3(min(448, max|x| 2^-e / 6))),   c = e2m1(x / (s 2^e)).
// The rounding of c is decided by comparing |x| with the seven borders between
// neighbouring magnitudes times s 2^e: border (3 bits) x s (4 bits) x a power
// of two is exact in fp32, so a value on a border goes to the even code as the
// definition has it; a quotient or a reciprocal would round first.  The
// quotient max|x| / 6 may round: e4m3's own borders have 5 bits and a bf16 max
// 8, so an unequal pair differs by more than 2^-13, far above fp32's rounding.
// A group with an infinity or a NaN stores the scale NaN: all of it reads back
// as NaN, and attention to it gives NaN, as a bf16 cache would.
//
// Both calls move bytes: 2 B in and 9/16 B out per element (append), the
// reverse (read).  One thread per group of K and of V: 64 B of loads in flight
// per thread, 32-byte sectors whole on the bf16 side and 8-byte pieces that
// neighbouring lanes complete to whole rows on the 4-bit side.
#include "internal.h"
#include "kv4.cuh"
#include "paged.h"

namespace dfl {

namespace {

struct Kv4Rows {
    Kv4Slab slab;
    const int32_t* table;   // [N][max_pages]
    int max_pages;
    const int32_t* start;   // [N] position of row 0 (negative: the sequence is skipped)
    const int32_t* count;   // [N] rows of each sequence
    int N, R;
    int k_exp, v_exp;
};

// Position of row i of sequence n -> its cell, or nullptr (row past the
// count, sequence skipped, or, recorded, a length or page out of range).
template <int HD>
__device__ __forceinline__ uint8_t* row_cell(const Kv4Rows& a, int n, int i, int head, const DevErr& err, int& tok) {
    const int s = a.start[n], m = a.count[n];
    if (s < 0 && m >= 0 && m <= a.R) return nullptr;
    if (m < 0 || m > a.R || s > a.max_pages * a.slab.page - m) {
        if (i == 0 && head == 0) record_error(err, DFL_ERR_INVALID_ARG);
        return nullptr;
    }
    if (i >= m) return nullptr;
    const int pos = s + i, j = pos / a.slab.page, in = pos - j * a.slab.page;
    const int p = a.table[(int64_t)n * a.max_pages + j];
    if (p < 0 || p >= a.slab.num_pages) {
        record_error(err, DFL_ERR_INVALID_ARG);
        return nullptr;
    }
    tok = in & (KV4_CELL_TOKENS - 1);
    return a.slab.data + (((int64_t)p * a.slab.Hkv + head) * a.slab.cells + in / KV4_CELL_TOKENS) * Kv4Cell<HD>::BYTES;
}

__device__ __forceinline__ void quantise16(const uint4 lo, const uint4 hi, int e, uint2& codes, uint8_t& scale) {
    const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    uint32_t mx = 0;   // magnitudes of bf16 order as integers
    #pragma unroll
    for (int i = 0; i < 8; ++i) mx = max(mx, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
    codes = make_uint2(0, 0);
    if (mx >= 0x7F80u) { scale = 0x7F; return; }
    const float q = __fdiv_rn(__uint_as_float(mx << 16) * kv4_exp2i(-e), 6.f);
    uint16_t sb;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(sb) : "f"(0.f), "f"(q));
    scale = max((int)(sb & 0xFF), 1);   // code 1 is 2^-9, the smallest scale
    const float t = half2_to_float2(e4m3x2_to_half(scale)).x * kv4_exp2i(e);
    uint32_t c[2] = {0, 0};
    #pragma unroll
    for (int i = 0; i < 16; ++i) {
        const uint32_t b = i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16;
        const float a = fabsf(__uint_as_float(b));
        uint32_t k = (a > 0.25f * t) + (a >= 0.75f * t) + (a > 1.25f * t) + (a >= 1.75f * t) + (a > 2.5f * t) +
                     (a >= 3.5f * t) + (a > 5.f * t);
        k |= (b >> 28) & 8u;
        c[i / 8] |= k << (4 * (i % 8));
    }
    codes = make_uint2(c[0], c[1]);
}

template <int HD>
__global__ void __launch_bounds__(256) kv4_append_kernel(const Kv4Rows a, const uint4* K, const uint4* V, const DevErr err) {
    grid_dep_begin();
    using Cell = Kv4Cell<HD>;
    const int64_t total = (int64_t)a.N * a.R * a.slab.Hkv * Cell::GROUPS;
    for (int64_t x = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; x < total; x += (int64_t)gridDim.x * blockDim.x) {
        const int group = (int)(x % Cell::GROUPS);
        const int64_t rh = x / Cell::GROUPS;
        const int head = (int)(rh % a.slab.Hkv);
        const int64_t row = rh / a.slab.Hkv;
        const int n = (int)(row / a.R), i = (int)(row - (int64_t)n * a.R);
        int tok;
        uint8_t* cell = row_cell<HD>(a, n, i, head, err, tok);
        if (!cell) continue;
        const uint4 k0 = K[2 * x], k1 = K[2 * x + 1], v0 = V[2 * x], v1 = V[2 * x + 1];
        if (!DFL_IN_BOUNDS(err.word, cell - a.slab.data,
                           (int64_t)a.slab.num_pages * a.slab.Hkv * a.slab.cells * Cell::BYTES))
            continue;
        uint2 c;
        uint8_t s;
        quantise16(k0, k1, a.k_exp, c, s);
        *reinterpret_cast<uint2*>(cell + Cell::k_code(tok, group)) = c;
        cell[Cell::k_scale(tok, group)] = s;
        quantise16(v0, v1, a.v_exp, c, s);
        *reinterpret_cast<uint2*>(cell + Cell::v_code(tok, group)) = c;
        cell[Cell::v_scale(tok, group)] = s;
    }
}

__device__ __forceinline__ void expand16(uint2 codes, uint8_t scale, float pow2, uint4& lo, uint4& hi) {
    const uint32_t s = e4m3x2_to_half(scale * 0x101u);
    uint32_t o[8];
    #pragma unroll
    for (int j = 0; j < 2; ++j) {
        uint32_t h[4];
        e2m1x8_to_half(j ? codes.y : codes.x, h);
        #pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = half2_to_float2(hmul2u(h[i], s));
            o[4 * j + i] = pack_bf16(f.x * pow2, f.y * pow2);
        }
    }
    lo = make_uint4(o[0], o[1], o[2], o[3]);
    hi = make_uint4(o[4], o[5], o[6], o[7]);
}

template <int HD>
__global__ void __launch_bounds__(256) kv4_read_kernel(const Kv4Rows a, uint4* K, uint4* V, const DevErr err) {
    grid_dep_begin();
    using Cell = Kv4Cell<HD>;
    const float pk = kv4_exp2i(a.k_exp), pv = kv4_exp2i(a.v_exp);
    const int64_t total = (int64_t)a.N * a.R * a.slab.Hkv * Cell::GROUPS;
    for (int64_t x = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; x < total; x += (int64_t)gridDim.x * blockDim.x) {
        const int group = (int)(x % Cell::GROUPS);
        const int64_t rh = x / Cell::GROUPS;
        const int head = (int)(rh % a.slab.Hkv);
        const int64_t row = rh / a.slab.Hkv;
        const int n = (int)(row / a.R), i = (int)(row - (int64_t)n * a.R);
        int tok;
        const uint8_t* cell = row_cell<HD>(a, n, i, head, err, tok);
        if (!cell) continue;
        const uint2 kc = *reinterpret_cast<const uint2*>(cell + Cell::k_code(tok, group));
        const uint2 vc = *reinterpret_cast<const uint2*>(cell + Cell::v_code(tok, group));
        uint4 lo, hi;
        expand16(kc, cell[Cell::k_scale(tok, group)], pk, lo, hi);
        K[2 * x] = lo;
        K[2 * x + 1] = hi;
        expand16(vc, cell[Cell::v_scale(tok, group)], pv, lo, hi);
        V[2 * x] = lo;
        V[2 * x + 1] = hi;
    }
}

Kv4Rows rows_args(const dfl_kv4_pool& pool, int layer, const dfl_pages& pg, const int32_t* start, const int32_t* count,
                  int R) {
    return Kv4Rows{kv4_slab(pool, layer), pg.table, pg.max_pages, start, count, pg.N, R, pool.k_exp, pool.v_exp};
}

unsigned rows_grid(const DeviceCtx* ctx, const Kv4Rows& a, int hd) {
    const int64_t total = (int64_t)a.N * a.R * a.slab.Hkv * (hd / 16);
    return (unsigned)std::min<int64_t>((total + 255) / 256, (int64_t)ctx->sm_count * 64);
}

}  // namespace

dfl_status kv4_append_run(DeviceCtx* ctx, const dfl_kv4_pool& pool, int layer, const dfl_pages& pg,
                          const int32_t* start, const int32_t* n_new, int R, const void* K, const void* V,
                          cudaStream_t st) {
    ProfScope ps("kv4_append", st);
    const Kv4Rows a = rows_args(pool, layer, pg, start, n_new, R);
    auto kern = pool.hd == 128 ? kv4_append_kernel<128> : kv4_append_kernel<64>;
    return launch_pdl(kern, rows_grid(ctx, a, pool.hd), 256, 0, st, a, static_cast<const uint4*>(K),
                      static_cast<const uint4*>(V), dev_err(ctx));
}

dfl_status kv4_read_run(DeviceCtx* ctx, const dfl_kv4_pool& pool, int layer, const dfl_pages& pg, const int32_t* start,
                        const int32_t* count, int R, void* K, void* V, cudaStream_t st) {
    ProfScope ps("kv4_read", st);
    const Kv4Rows a = rows_args(pool, layer, pg, start, count, R);
    auto kern = pool.hd == 128 ? kv4_read_kernel<128> : kv4_read_kernel<64>;
    return launch_pdl(kern, rows_grid(ctx, a, pool.hd), 256, 0, st, a, static_cast<uint4*>(K), static_cast<uint4*>(V),
                      dev_err(ctx));
}

}  // namespace dfl
