// Writing context rows into the 4-bit cache and reading them back.
//
// Append, per 16 dimensions x of one token and K/V head (a group):
//   s = max(2^-9, e4m3(min(448, max|x| 2^-e / 6))),   c = e2m1(x / (s 2^e)).
// x / (s 2^e) is taken as x times the correctly rounded reciprocal and rounded to
// a grid of 2^-11 (one fused product and sum with a large number, which is taken
// off again) before the rounding to e2m1; that decides as the exact quotient
// would.  The borders between e2m1's numbers, 0.25 the smallest, have 3 bits and
// s 4, so a border times s 2^e has at most 7 and x, a bf16, has 8: where they
// differ the quotient is 2^-10 or more away from the border, which neither
// fp32's 2^-23 nor the grid's half step of 2^-12 moves across; where they are
// equal the product is within 2^-21 of the border, a point of the grid, and it
// goes to the even code.  The quotient
// max|x| / 6 may round: e4m3's own borders have 5 bits and a bf16 max 8, so an
// unequal pair differs by more than 2^-13, far above fp32's rounding.
// A group with an infinity or a NaN stores the scale NaN: all of it reads back
// as NaN, and attention to it gives NaN, as a bf16 cache would.
//
// Both calls move bytes: 2 B in and 9/16 B out per element (append), the
// reverse (read).  One thread per group of K and of V: 64 B of loads in flight
// per thread, 32-byte sectors whole on the bf16 side and 8-byte pieces that
// neighbouring lanes complete to whole rows on the 4-bit side.  A block takes
// some whole rows of one sequence (or part of one when a row has more groups
// than the block threads), so a thread divides once, by small numbers.
#include "internal.h"
#include "kv4.cuh"
#include "paged.h"

namespace dfl {

namespace {

constexpr int KR_THREADS = 256;

struct Kv4Rows {
    Kv4Slab slab;
    const int32_t* table;   // [N][max_pages]
    int max_pages;
    const int32_t* start;   // [N] position of row 0 (negative: the sequence is skipped)
    const int32_t* count;   // [N] rows of each sequence
    const int32_t* pick;    // [N][R] row that goes to place i, nullable: row i (append)
    int N, R;
    int width;              // groups of a row: Hkv * hd / 16
    int rows;               // rows of a block
    uint64_t cells_inv;     // ceil(2^36 / cells of a page)
    int k_exp, v_exp;
};

// A group that exists.
struct Kv4Item {
    int n, i, head, group;  // sequence, row, head, group of the head
    int start;              // position of row 0
    int64_t at;             // the group among all of K
};

// Calls body(item) for every group of the call that exists.
template <int HD, typename Body>
__device__ __forceinline__ void kv4_each(const Kv4Rows& a, const DevErr& err, Body body) {
    constexpr int GROUPS = Kv4Cell<HD>::GROUPS;
    const int down = a.rows == 1 ? 0 : (int)threadIdx.x / a.width, x0 = (int)threadIdx.x - down * a.width;
    #pragma unroll 1
    for (int n = blockIdx.y; n < a.N; n += gridDim.y) {
        const int s = a.start[n], m = a.count[n];
        if (m < 0 || m > a.R || (s >= 0 && s > a.max_pages * a.slab.page - m)) {
            if (blockIdx.x == 0 && threadIdx.x == 0) record_error(err, DFL_ERR_INVALID_ARG);
            continue;
        }
        if (s < 0 || down >= a.rows) continue;
        #pragma unroll 1
        for (int64_t i = (int64_t)blockIdx.x * a.rows + down; i < m; i += (int64_t)gridDim.x * a.rows) {
            #pragma unroll 1
            for (int x = x0; x < a.width; x += KR_THREADS)
                body(Kv4Item{n, (int)i, x / GROUPS, x % GROUPS, s, ((int64_t)n * a.R + i) * a.width + x});
        }
    }
}

// The cell of a row that exists, or nullptr (its page is out of range: recorded).
template <int HD>
__device__ __forceinline__ uint8_t* row_cell(const Kv4Rows& a, const Kv4Item& t, const DevErr& err, int& tok) {
    const int pos = t.start + t.i;
    const uint32_t c = (uint32_t)pos / KV4_CELL_TOKENS;
    const int j = (int)((c * a.cells_inv) >> 36);   // c / cells: c < 2^27, cells <= 64
    const int p = a.table[(int64_t)t.n * a.max_pages + j];
    if (p < 0 || p >= a.slab.num_pages) {
        record_error(err, DFL_ERR_INVALID_ARG);
        return nullptr;
    }
    tok = pos & (KV4_CELL_TOKENS - 1);
    const int cell = (p * a.slab.Hkv + t.head) * a.slab.cells + ((int)c - j * a.slab.cells);   // < 2^31 (checked)
    return a.slab.data + (int64_t)cell * Kv4Cell<HD>::BYTES;
}

// Two floats -> two e2m1 codes (a in the low nibble), nearest, ties to even, larger ones to 6.
__device__ __forceinline__ uint32_t e2m1x2(float a, float b) {
    uint32_t r;
    asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %2, %1;\n\tcvt.u32.u8 %0, t;\n\t}" : "=r"(r) : "f"(a), "f"(b));
    return r;
}

constexpr float SNAP = 1.5f * 4096.f;   // x + SNAP - SNAP is x on the grid of 2^-11

__device__ __forceinline__ void quantise16(const uint4 lo, const uint4 hi, int e, uint2& codes, uint8_t& scale) {
    const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    uint32_t m2 = 0;   // magnitudes of bf16 order as integers
    #pragma unroll
    for (int i = 0; i < 8; ++i) m2 = max_u16x2(m2, w[i] & 0x7FFF7FFFu);
    const uint32_t mx = max(m2 & 0xFFFFu, m2 >> 16);
    codes = make_uint2(0, 0);
    if (mx >= 0x7F80u) { scale = 0x7F; return; }
    const float q = __fdiv_rn(__uint_as_float(mx << 16) * kv4_exp2i(-e), 6.f);
    uint16_t sb;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(sb) : "f"(0.f), "f"(q));
    scale = max((int)(sb & 0xFF), 1);   // code 1 is 2^-9, the smallest scale
    const float r = __frcp_rn(half2_to_float2(e4m3x2_to_half(scale)).x * kv4_exp2i(e));
    uint32_t c[2];
    #pragma unroll
    for (int j = 0; j < 2; ++j) {
        uint32_t b[4];
        #pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 x = make_float2(bf16lo(w[4 * j + i]), bf16hi(w[4 * j + i]));
            const float2 f = add_f32x2(fma_f32x2(x, make_float2(r, r), make_float2(SNAP, SNAP)), make_float2(-SNAP, -SNAP));
            b[i] = e2m1x2(f.x, f.y);
        }
        c[j] = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
    }
    codes = make_uint2(c[0], c[1]);
}

template <int HD>
__global__ void __launch_bounds__(KR_THREADS, 5) kv4_append_kernel(const Kv4Rows a, const uint4* K, const uint4* V, const DevErr err) {
    grid_dep_begin();
    using Cell = Kv4Cell<HD>;
    kv4_each<HD>(a, err, [&](Kv4Item t) {
        if (a.pick) {
            const int from = a.pick[(int64_t)t.n * a.R + t.i];
            if (from < 0 || from >= a.R) {
                record_error(err, DFL_ERR_INVALID_ARG);
                return;
            }
            t.at += (int64_t)(from - t.i) * a.width;
        }
        const uint4 k0 = K[2 * t.at], k1 = K[2 * t.at + 1], v0 = V[2 * t.at], v1 = V[2 * t.at + 1];
        int tok;
        uint8_t* cell = row_cell<HD>(a, t, err, tok);
        if (!cell) return;
        if (!DFL_IN_BOUNDS(err.word, cell - a.slab.data + Cell::BYTES - 1,
                           (int64_t)a.slab.num_pages * a.slab.Hkv * a.slab.cells * Cell::BYTES))
            return;
        uint2 c;
        uint8_t s;
        quantise16(k0, k1, a.k_exp, c, s);
        *reinterpret_cast<uint2*>(cell + Cell::k_code(tok, t.group)) = c;
        cell[Cell::k_scale(tok, t.group)] = s;
        quantise16(v0, v1, a.v_exp, c, s);
        *reinterpret_cast<uint2*>(cell + Cell::v_code(tok, t.group)) = c;
        cell[Cell::v_scale(tok, t.group)] = s;
    });
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
__global__ void __launch_bounds__(KR_THREADS, 5) kv4_read_kernel(const Kv4Rows a, uint4* K, uint4* V, const DevErr err) {
    grid_dep_begin();
    using Cell = Kv4Cell<HD>;
    const float pk = kv4_exp2i(a.k_exp), pv = kv4_exp2i(a.v_exp);
    kv4_each<HD>(a, err, [&](const Kv4Item& t) {
        int tok;
        const uint8_t* cell = row_cell<HD>(a, t, err, tok);
        if (!cell || !DFL_IN_BOUNDS(err.word, t.at, (int64_t)a.N * a.R * a.width)) return;
        const uint2 kc = *reinterpret_cast<const uint2*>(cell + Cell::k_code(tok, t.group));
        const uint2 vc = *reinterpret_cast<const uint2*>(cell + Cell::v_code(tok, t.group));
        uint4 lo, hi;
        expand16(kc, cell[Cell::k_scale(tok, t.group)], pk, lo, hi);
        K[2 * t.at] = lo;
        K[2 * t.at + 1] = hi;
        expand16(vc, cell[Cell::v_scale(tok, t.group)], pv, lo, hi);
        V[2 * t.at] = lo;
        V[2 * t.at + 1] = hi;
    });
}

Kv4Rows rows_args(const dfl_kv4_pool& pool, int layer, const dfl_pages& pg, const int32_t* start, const int32_t* count,
                  const int32_t* pick, int R) {
    Kv4Rows a{kv4_slab(pool, layer), pg.table, pg.max_pages, start, count, pick, pg.N, R};
    a.width = pool.Hkv * (pool.hd / 16);
    a.rows = std::max(1, KR_THREADS / a.width);
    a.cells_inv = (((uint64_t)1 << 36) + a.slab.cells - 1) / a.slab.cells;
    a.k_exp = pool.k_exp;
    a.v_exp = pool.v_exp;
    return a;
}

// Four rounds of the five blocks an SM holds: prompts of 1,025 to 4,097 rows of 8
// sequences (8 heads of 64) are written and read back in 27.1 us so, in 28.7
// with a block for every 8 rows and in 31.2 with one round; 3.5 TB/s.
dim3 rows_grid(const DeviceCtx* ctx, const Kv4Rows& a) {
    const int n = std::min(a.N, 65535);
    const int64_t chunks = ((int64_t)a.R + a.rows - 1) / a.rows;
    return dim3((unsigned)std::min(chunks, std::max<int64_t>(1, (int64_t)ctx->sm_count * 20 / n)), (unsigned)n);
}

}  // namespace

dfl_status kv4_append_run(DeviceCtx* ctx, const dfl_kv4_pool& pool, int layer, const dfl_pages& pg,
                          const int32_t* start, const int32_t* n_new, const int32_t* rows, int R, const void* K,
                          const void* V, cudaStream_t st) {
    ProfScope ps("kv4_append", st);
    const Kv4Rows a = rows_args(pool, layer, pg, start, n_new, rows, R);
    auto kern = pool.hd == 128 ? kv4_append_kernel<128> : kv4_append_kernel<64>;
    return launch_pdl(kern, rows_grid(ctx, a), KR_THREADS, 0, st, a, static_cast<const uint4*>(K),
                      static_cast<const uint4*>(V), dev_err(ctx));
}

dfl_status kv4_read_run(DeviceCtx* ctx, const dfl_kv4_pool& pool, int layer, const dfl_pages& pg, const int32_t* start,
                        const int32_t* count, int R, void* K, void* V, cudaStream_t st) {
    ProfScope ps("kv4_read", st);
    const Kv4Rows a = rows_args(pool, layer, pg, start, count, nullptr, R);
    auto kern = pool.hd == 128 ? kv4_read_kernel<128> : kv4_read_kernel<64>;
    return launch_pdl(kern, rows_grid(ctx, a), KR_THREADS, 0, st, a, static_cast<uint4*>(K), static_cast<uint4*>(V),
                      dev_err(ctx));
}

}  // namespace dfl
