// What the two attention kernels over the 4-bit paged cache share: arguments,
// the line of work units and the sum of partials (kv4_attn.cu says how the
// line is cut).
#pragma once

#include "internal.h"
#include "kv4.cuh"

namespace dfl {

// The triple that starts in a range and ends in range `last` behind it; n < 0: none.
struct alignas(16) KaCross {
    int n, head, tile, last;
};

struct KaArgs {
    Kv4Slab slab;
    const int32_t* table;
    const int32_t* len;
    int max_pages;
    int N, B, Hq, G, R;
    int subs;                 // row tiles per K/V head
    int HS;                   // Hkv * subs
    int unit_log2;            // keys per unit
    int weight, seam;         // see KaLine
    uint64_t g_inv;           // ceil(2^40 / G)
    uint64_t cells_inv;       // ceil(2^36 / cells of a page)
    const __nv_bfloat16* Q;   // [N*B][Hq][hd]
    const __nv_bfloat16* Kb;  // [N*B][Hkv][hd]
    const __nv_bfloat16* Vb;
    __nv_bfloat16* O;         // [N*B][Hq][hd]
    float* Opart;             // [2 * ranges][rows][hd]
    float2* ml;               // [2 * ranges][rows] (maximum in log2 units, sum)
    KaCross* cross;           // [ranges]
    float scale_log2;         // log2(e) / sqrt(hd)
    float k_pow2, k_inv, v_pow2, v_inv;   // 2^k_exp, 2^-k_exp, 2^v_exp, 2^-v_exp
};

// The tensor-memory kernel (kv4_attn_tc.cu): rows of its triples, scratch, launch
// (a complete but for Opart and ml; `units` an upper bound on the line).
inline int kv4_attn_tc_rows(int R) { return R <= 64 ? 64 : 128; }
int kv4_attn_tc_unit_log2(int R, int hd);
int kv4_attn_tc_seam();
int kv4_attn_tc_weight();
size_t kv4_attn_tc_ws_bytes(int R, int hd);
dfl_status kv4_attn_tc_run(DeviceCtx* ctx, KaArgs a, int hd, int64_t units, void* ws, cudaStream_t st);

namespace {

constexpr float KA_LAZY = 8.f;     // rescale when a maximum grows by more (log2)
// P is 2^7 above its nominal value, so at most 2^15: below fp16's largest.
// 7 - m is rounded down: at large m up, it would lift P past that.
constexpr float KA_LIFT = 7.f;
// The running maximum before the first key: no finite score is below it.  A key
// whose score is -inf has the weight 2^(-inf - m) = 0 with it; with -inf in its
// place, keys that are all of that kind had weights of -inf + inf.
constexpr float KA_NONE = -3.402823466e38f;

// One lane of a converged warp.  What it issues (copies, products) has operands
// the compiler knows to be uniform, at half the clocks of a lane in a divergent
// branch.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// Eight of the block's own bf16 elements in units of the pool's power of two
// (inv: its inverse), as fp16.  bf16's 8 bits survive from 2^-14 of the unit
// up; finite values past fp16's range become its largest, as the cache's
// become its own.  Infinities and NaN stay what they are.
__device__ __forceinline__ uint4 block_half8(const uint4 v, float inv) {
    uint32_t w[4] = {v.x, v.y, v.z, v.w}, h[4];
    #pragma unroll
    for (int i = 0; i < 4; ++i)
        asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(h[i]) : "f"(bf16hi(w[i]) * inv), "f"(bf16lo(w[i]) * inv));
    const uint32_t m = max_u16x2(max_u16x2(w[0] & 0x7FFF7FFFu, w[1] & 0x7FFF7FFFu), max_u16x2(w[2] & 0x7FFF7FFFu, w[3] & 0x7FFF7FFFu));
    if (m >= 0x7F800000u || (m & 0xFFFFu) >= 0x7F80u) {
        #pragma unroll
        for (int i = 0; i < 4; ++i)
            #pragma unroll
            for (int s = 0; s < 32; s += 16) {
                const uint32_t x = w[i] >> s & 0xFFFFu;
                const uint32_t y = (x & 0x8000u) | (x & 0x7Fu ? 0x7E00u : 0x7C00u);
                if ((x & 0x7F80u) == 0x7F80u) h[i] = (h[i] & ~(0xFFFFu << s)) | y << s;
            }
    }
    return make_uint4(h[0], h[1], h[2], h[3]);
}

// Biased exponent of the power of two that takes a query row's largest element
// (magnitude mx, a bf16) to [1, 2), or to below 4 at the top of the range, whose
// inverse is to stay normal.  Rows of zeros and subnormals: as they are.
__device__ __forceinline__ int ka_query_exp(uint32_t mx) {
    const int e = (int)(mx >> 7);
    return e == 0 ? 127 : min(e, 253);
}

// Score of fp16 operands -> log2 units, for a row that was divided by `up`.
// Neither 0, which would take a masked score's -inf to NaN, nor infinite, which
// would a 0.
__device__ __forceinline__ float ka_mult(const KaArgs& a, float up) {
    return fminf(fmaxf(up * a.scale_log2 * a.k_pow2, 1.175494351e-38f), 3.402823466e38f);
}

// Block row and head of query row r of a group: element offset of its Q and O.
__device__ __forceinline__ int64_t ka_row(const KaArgs& a, int n, int head, int r, int hd) {
    const int b = (int)(((uint64_t)(uint32_t)r * a.g_inv) >> 40);   // r / G: r G < 2^40
    return ((int64_t)(n * a.B + b) * a.Hq + head * a.G + (r - b * a.G)) * hd;
}

// Pool cell of token k (a multiple of 16) of sequence n for a K/V head; a page
// out of range is recorded and read as page 0.
__device__ __forceinline__ int ka_cell(const KaArgs& a, int n, int head, int k, const DevErr& err) {
    const uint32_t t = (uint32_t)k / KV4_CELL_TOKENS;
    const int j = (int)((t * a.cells_inv) >> 36);                   // t / cells: t cells < 2^36
    int p = a.table[(int64_t)n * a.max_pages + j];
    if (p < 0 || p >= a.slab.num_pages) { record_error(err, DFL_ERR_INVALID_ARG); p = 0; }
    return (p * a.slab.Hkv + head) * a.slab.cells + (int)t - j * a.slab.cells;
}

// Length of sequence n; one out of range is read as the nearest in range.
__device__ __forceinline__ int ka_len(const KaArgs& a, int n) { return min(max(a.len[n], 0), a.max_pages * a.slab.page); }

// Lengths out of range, recorded by the grid's first block.
template <int THREADS>
__device__ __forceinline__ void ka_check_lengths(const KaArgs& a, const DevErr& err) {
    if (blockIdx.x != 0) return;
    #pragma unroll 1
    for (int n = threadIdx.x; n < a.N; n += THREADS)
        if (a.len[n] != ka_len(a, n)) record_error(err, DFL_ERR_INVALID_ARG);
}

// Units of a sequence: its tokens, then the block's own keys.
__device__ __forceinline__ int ka_units(const KaArgs& a, int len) { return ((len + (1 << a.unit_log2) - 1) >> a.unit_log2) + 1; }

// The line of units and how it is cut: into ranges of `per` units, or, when
// there are no more triples than ranges and none is much longer than the rest,
// one whole triple per range.  A triple takes `weight` places on the line ahead
// of its units, for what it costs however short it is (queries, own keys, the
// end): without them a range of many short sequences ended long after the
// others.  Whole triples leave no partials to write, read and add up, and each
// range pays for one start and one end; `seam` is what a cut line costs a range
// beyond that, in units.
struct KaLine {
    int total, per;     // places in all, per range
    bool whole;
};

// Found by ka_locate: the sequence that holds a position, the units of the
// line before it, its length.
struct KaFound {
    int n, before, len, next;
};

template <int THREADS, int P>
struct KaLineSmem {
    int red[THREADS / 32], longest[THREADS / 32];
    KaFound at[P];
};

// The line cut into `ranges`; of the P positions at(i, per, total), those in
// 0 .. total - 1 are located in sm.at[i].  All threads of the block call; one
// read of the lengths when there are no more sequences than threads.
template <int THREADS, int P, typename At>
__device__ __forceinline__ KaLine ka_locate(const KaArgs& a, int ranges, KaLineSmem<THREADS, P>& sm, At at) {
    const int chunk = (a.N + THREADS - 1) / THREADS;
    const int n0 = min(a.N, (int)threadIdx.x * chunk), n1 = min(a.N, n0 + chunk);
    const int len0 = n0 < n1 ? ka_len(a, n0) : 0, len1 = n0 + 1 < a.N ? ka_len(a, n0 + 1) : 0;
    int sum = n0 < n1 ? ka_units(a, len0) + a.weight : 0, longest = sum;
    #pragma unroll 1
    for (int n = n0 + 1; n < n1; ++n) {
        const int nu = ka_units(a, ka_len(a, n)) + a.weight;
        sum += nu;
        longest = max(longest, nu);
    }
    sum *= a.HS;
    longest = __reduce_max_sync(0xFFFFFFFFu, longest);
    if ((threadIdx.x & 31) == 0) sm.longest[threadIdx.x >> 5] = longest;
    KaLine l;
    const int pre = block_exscan<THREADS>(sum, sm.red, &l.total);
    l.per = max(1, (l.total + ranges - 1) / ranges);
    longest = (threadIdx.x & 31) < THREADS / 32 ? sm.longest[threadIdx.x & 31] : 0;
    longest = __reduce_max_sync(0xFFFFFFFFu, longest);
    l.whole = (int64_t)a.N * a.HS <= ranges && longest <= l.per + a.seam;
    if (l.whole) return l;
    #pragma unroll 1
    for (int i = 0; i < P; ++i) {
        const int x = at(i, l.per, l.total);
        if (x < pre || x >= pre + sum) continue;
        int p = pre, len = len0, next = len1;
        #pragma unroll 1
        for (int n = n0; ; ++n) {
            const int w = (ka_units(a, len) + a.weight) * a.HS;
            if (x < p + w) { sm.at[i] = KaFound{n, p, len, next}; break; }
            p += w;
            len = next;
            next = n + 2 < a.N ? ka_len(a, n + 2) : 0;
        }
    }
    __syncthreads();
    return l;
}

// A position on the line as (sequence, head and row tile, unit); u < 0 in the
// places ahead of a triple's units.  The next sequence's length is read ahead.
struct KaPos {
    int n, hs, head, tile, u, nu, len, next;
    // Position x of the line, which ka_locate found.
    __device__ __forceinline__ void set(const KaArgs& a, const KaFound& f, int x) {
        n = f.n;
        len = f.len;
        next = f.next;
        nu = ka_units(a, len);
        hs = (x - f.before) / (nu + a.weight);
        u = x - f.before - hs * (nu + a.weight) - a.weight;
        head = hs / a.subs;
        tile = hs - head * a.subs;
    }
    // The start of triple t of all.
    __device__ __forceinline__ void set_triple(const KaArgs& a, int t) {
        n = t / a.HS;
        hs = t - n * a.HS;
        len = ka_len(a, n);
        next = 0;
        nu = ka_units(a, len);
        u = 0;
        head = hs / a.subs;
        tile = hs - head * a.subs;
    }
    // From place x to the unit that follows; false at the range's end x1.
    __device__ __forceinline__ bool enter(int& x, int x1) {
        x -= min(u, 0);
        u = max(u, 0);
        return x < x1;
    }
    __device__ __forceinline__ void next_triple(const KaArgs& a) {
        u = -a.weight;
        ++hs;
        if (++tile == a.subs) { tile = 0; ++head; }
        if (hs == a.HS) {
            hs = head = 0;
            ++n;
            len = next;
            nu = ka_units(a, len);
            next = n + 1 < a.N ? ka_len(a, n + 1) : 0;
        }
    }
};

// Adds up the triple that starts in range blockIdx.x and ends past it, if there
// is one: partials of that range (its second) and of the following ones (their
// first), in the order of the keys.  gridDim.x ranges; blockIdx.y takes some of
// the rows.  The attention kernel says which triple that is: found again from
// the lengths, it cost this kernel 2 us of its 4.
template <int HD, int ROWS>
struct KjCfg {
    static constexpr int AT_ONCE = ROWS < 64 ? 8 : 16;   // rows of a block
    static constexpr int THREADS = HD / 4 * AT_ONCE;
};
template <int HD, int ROWS>
__global__ void __launch_bounds__(KjCfg<HD, ROWS>::THREADS) kv4_attn_join_kernel(const KaArgs a, const DevErr err) {
    constexpr int TPR = HD / 4;
    grid_dep_begin();
    const KaCross t = a.cross[blockIdx.x];
    if (t.n < 0) return;
    const int first = blockIdx.x, last = t.last, row0 = t.tile * ROWS;
    const int row = blockIdx.y * KjCfg<HD, ROWS>::AT_ONCE + threadIdx.x / TPR, c = (threadIdx.x % TPR) * 4, r = row0 + row;
    if (row >= ROWS || r >= a.R) return;
    // eight partials are read at once: a long triple waits for memory once per eight
    constexpr int BATCH = 8;
    float M = KA_NONE, L = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    #pragma unroll 1
    for (int j0 = first; j0 <= last; j0 += BATCH) {
        float2 ml[BATCH];
        float4 v[BATCH];
        float mn = M;
        #pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            const int j = min(j0 + i, last);
            const int64_t at = (int64_t)(2 * j + (j == first)) * ROWS + row;
            ml[i] = a.ml[at];
            v[i] = *reinterpret_cast<const float4*>(a.Opart + at * HD + c);
        }
        #pragma unroll
        for (int i = 0; i < BATCH; ++i) mn = fmaxf(mn, ml[i].x);
        const float old = ex2_ftz(M - mn);
        M = mn;
        L *= old; o.x *= old; o.y *= old; o.z *= old; o.w *= old;
        #pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            const float f = j0 + i > last ? 0.f : ex2_ftz(ml[i].x - M);
            L += f * ml[i].y;
            o.x += f * v[i].x; o.y += f * v[i].y; o.z += f * v[i].z; o.w += f * v[i].w;
        }
    }
    const float inv = __fdividef(a.v_pow2, L);
    const int64_t at = ka_row(a, t.n, t.head, r, HD) + c;
    if (DFL_IN_BOUNDS(err.word, at + 3, (int64_t)a.N * a.B * a.Hq * HD))
        *reinterpret_cast<uint2*>(a.O + at) =
            make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
}

}  // namespace

}  // namespace dfl
