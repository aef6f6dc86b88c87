// Block attention over the 4-bit paged cache for many query rows per K/V head,
// on the 5th-generation tensor cores.  The same sum and the same line of work
// units as kv4_attn.cu, with up to 128 rows to a triple, where products and
// exponentials, not bytes, are most of the work.
//
// One CTA per SM, two pipelines of ten warps, each with a range of the line of
// its own, so that one pipeline's products run under the other's exponentials:
//   producer (1 warp)   bulk copies of a unit's cells (4-bit) into a ring;
//   expanders (4 warps) one cell each: codes * scales in fp16 into a K tile
//                       and a V tile [64 keys][hd] with 128-byte swizzle; the
//                       block's own keys come as bf16 straight from memory;
//   issuer (1 thread)   S = Q K^T (M = 64 or 128 rows, N = 64), then
//                       O += P V (N = hd); Q and P are A operands in tensor
//                       memory, so the products read only K and V tiles from
//                       shared memory;
//   softmax (4 warps)   Q into tensor memory (fp16, and bf16 for the block's
//                       own unit), running maximum and sum, P over S's
//                       columns, the triple's output.
// What bounds it: a unit's tiles (hd = 128) are 32 KB written by the expanders
// and read by the products, with 18 KB of codes in and out: 650 clocks of
// shared memory at 128 B per clock, against 390 of HBM at its measured rate.
// 256 tensor-memory columns per pipeline: S (64), Q (hd / 2), O (hd); at
// hd = 128 a second S buffer has no room, so S of a unit follows P V of the
// one before, and the other pipeline fills the gap.
#include "internal.h"
#include "kv4_attn.cuh"
#include "paged.h"

namespace dfl {

namespace {

constexpr int KT_PIPES = 2;
constexpr int KT_WARPS = KT_PIPES * 8 + 4;     // softmax, expanders; producers and issuers
constexpr int KT_THREADS = KT_WARPS * 32;

template <int HD, int MM>
struct KtCfg {
    static constexpr int KB = HD / 64;                  // 128-byte blocks of a tile row
    static constexpr int TKB = 64 * 128;                // bytes of one such block of a tile
    static constexpr int TILE = KB * TKB;
    static constexpr int CELL = Kv4Cell<HD>::BYTES;
    static constexpr int RAW = 4 * CELL;                // a unit's cells
    static constexpr int RST = 4, KST = 2, VST = 2;     // slots per pipeline
    static constexpr int PIPE = (KST + VST) * TILE + RST * RAW;
    static constexpr int S_COL = 0, Q_COL = 64, O_COL = 128, COLS = 256;
    static constexpr int SMEM = 1024 + KT_PIPES * PIPE;
    static_assert(O_COL + HD <= COLS && Q_COL + HD / 2 <= O_COL, "tensor memory columns");
    static_assert(SMEM <= 226 * 1024, "shared memory");
    static_assert(PIPE % 1024 == 0, "tiles start on 1024-byte boundaries");
};

template <int RST, int KST, int VST>
struct KtBars {
    uint64_t raw_full[RST], raw_empty[RST];
    uint64_t k_full[KST], k_empty[KST];
    uint64_t v_full[VST], v_empty[VST];
    uint64_t q_full, s_full, p_full, pv_done, o_empty, drain;
};

__host__ __device__ constexpr uint32_t kt_idesc_f16(int M, int N) {   // fp16 A and B, fp32 sums
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// Wait as mbar_wait, and give up when another role of the CTA has.
__device__ __forceinline__ bool kt_wait(uint64_t* bar, uint32_t parity, const DevErr& e, volatile int* abort) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    while (true) {
        #pragma unroll 1
        for (int i = 0; i < 32; ++i)
            if (mbar_try_wait(bar, parity)) return true;
        if (*abort) return false;
        if (globaltimer_ns() - t0 > e.limit_ns) {
            record_error(e, DFL_ERR_TIMEOUT);
            *abort = 1;
            return false;
        }
    }
}

// Position in a ring of N slots and its parity.
template <int N>
struct KtRing {
    uint32_t i = 0, ph = 0;
    __device__ __forceinline__ void step() {
        if (++i == N) { i = 0; ph ^= 1u; }
    }
};

// 8 codes times an fp16 pair (s, s) -> 16 bytes of a tile.
__device__ __forceinline__ uint4 kt_expand(uint32_t codes, uint32_t s) {
    uint32_t h[4];
    e2m1x8_to_half(codes, h);
    return make_uint4(hmul2u(h[0], s), hmul2u(h[1], s), hmul2u(h[2], s), hmul2u(h[3], s));
}

// One cell's K codes into rows 16 w .. of a K tile.  A quarter warp writes the
// eight 16-byte pieces of one tile row: no bank conflicts on either side.
template <int HD>
__device__ __forceinline__ void kt_expand_k(const uint8_t* cell, uint8_t* tile, int lane) {
    using Cell = Kv4Cell<HD>;
    constexpr int WPR = HD / 8;             // words (8 codes) of a row
    constexpr int RPL = 32 / WPR;           // rows per warp-wide load
    const int c = lane % WPR, h = lane / WPR;
    uint8_t* kb = tile + (c >> 3) * 64 * 128;
    #pragma unroll
    for (int i = 0; i < 8 / RPL; ++i) {     // slots s and s + 8
        const int s = RPL * i + h, tok = Cell::token(s);
        const uint32_t w0 = *reinterpret_cast<const uint32_t*>(cell + Cell::K_CODES + s * Cell::ROW + 4 * c);
        const uint32_t w1 = *reinterpret_cast<const uint32_t*>(cell + Cell::K_CODES + (s + 8) * Cell::ROW + 4 * c);
        uint32_t s0, s1;
        if constexpr (HD == 128) {
            const uint32_t sw = *reinterpret_cast<const uint32_t*>(cell + Cell::K_SCALES + (s * 4 + (c >> 2)) * 4);
            const uint32_t sel = c & 2 ? 0x3232u : 0x1010u;
            const uint32_t h0 = e4m3x2_to_half(sw & 0xFFFFu), h1 = e4m3x2_to_half(sw >> 16);
            s0 = __byte_perm(h0, h0, sel);
            s1 = __byte_perm(h1, h1, sel);
        } else {
            const uint32_t hp = e4m3x2_to_half(*reinterpret_cast<const uint16_t*>(cell + Cell::K_SCALES + (s * 4 + (c >> 1)) * 2));
            s0 = __byte_perm(hp, hp, 0x1010);
            s1 = __byte_perm(hp, hp, 0x3232);
        }
        uint8_t* d = kb + tok * 128 + (((c & 7) ^ (tok & 7)) << 4);
        *reinterpret_cast<uint4*>(d) = kt_expand(w0, s0);
        *reinterpret_cast<uint4*>(d + 8 * 128) = kt_expand(w1, s1);
    }
}

// The same for V; tokens from `left` on become zeros (a weight of 0 times
// whatever is stored there must add nothing).
template <int HD>
__device__ __forceinline__ void kt_expand_v(const uint8_t* cell, uint8_t* tile, int lane, int left) {
    using Cell = Kv4Cell<HD>;
    constexpr int WPR = HD / 8, RPL = 32 / WPR;
    const int pos = lane % WPR, h = lane / WPR;
    #pragma unroll
    for (int b = 0; b < 4 / RPL; ++b) {     // tokens t, 4 + t, 8 + t, 12 + t
        const int t = RPL * b + h;
        const int c = HD == 128 ? pos ^ (t & 2 ? 8 : 0) : pos;
        const uint32_t sw = *reinterpret_cast<const uint32_t*>(cell + Cell::V_SCALES + (c >> 1) * 16 + t * 4);
        const uint32_t sp[2] = {e4m3x2_to_half(sw & 0xFFFFu), e4m3x2_to_half(sw >> 16)};
        uint8_t* kb = tile + (c >> 3) * 64 * 128;
        #pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int tok = 4 * i + t;
            const uint32_t w = *reinterpret_cast<const uint32_t*>(cell + Cell::V_CODES + tok * Cell::ROW + 4 * pos);
            uint32_t s = __byte_perm(sp[i >> 1], sp[i >> 1], i & 1 ? 0x3232 : 0x1010);
            if (tok >= left) s = 0;
            *reinterpret_cast<uint4*>(kb + tok * 128 + (((c & 7) ^ (tok & 7)) << 4)) = kt_expand(w, s);
        }
    }
}

// Rows 16 w .. 16 w + 15 of a tile from bf16 rows of the block (zeros past B).
template <int HD>
__device__ __forceinline__ void kt_block_rows(const __nv_bfloat16* src, int64_t row_stride, uint8_t* tile, int lane, int left) {
    constexpr int WPR = HD / 8, RPL = 32 / WPR;
    const int c = lane % WPR, h = lane / WPR;
    uint8_t* kb = tile + (c >> 3) * 64 * 128;
    #pragma unroll
    for (int i = 0; i < 16 / RPL; ++i) {
        const int tok = RPL * i + h;
        const uint4 v = tok < left ? *reinterpret_cast<const uint4*>(src + tok * row_stride + c * 8) : make_uint4(0, 0, 0, 0);
        *reinterpret_cast<uint4*>(kb + tok * 128 + (((c & 7) ^ (tok & 7)) << 4)) = v;
    }
}

// Softmax side: M = 128 gives a thread one row (its tensor-memory lane); at
// M = 64 the 16 rows of a warp's quadrant are shared by its two half-warps,
// each with half of a row's columns.
template <int HD, int MM>
struct KtRow {
    static constexpr bool HALF = MM == 64;
    static constexpr int KPT = HALF ? 32 : 64;          // keys per thread and unit
    static constexpr int OPT = HALF ? HD / 2 : HD;      // O columns per thread
    static constexpr int QPT = HALF ? HD / 4 : HD / 2;  // Q columns (pairs) per thread

    // Q of one row (nullptr: no such row) -> tensor memory, as fp16 after a
    // power of two or as it is; returns the power that was taken out.  16 words
    // at a time, read twice: a row in registers would set the kernel's count.
    static __device__ __forceinline__ float load_q(const __nv_bfloat16* src, int hh, bool half_form, uint32_t q_addr) {
        const uint4* p = reinterpret_cast<const uint4*>(src + hh * (HD / 2));
        float up = 1.f, down = 1.f;
        if (half_form) {
            uint32_t mx = 0;
            #pragma unroll 4
            for (int i = 0; i < QPT / 4; ++i) {
                const uint4 w = src ? p[i] : make_uint4(0, 0, 0, 0);
                mx = max(mx, max(max(w.x & 0x7FFFu, (w.x >> 16) & 0x7FFFu), max(w.y & 0x7FFFu, (w.y >> 16) & 0x7FFFu)));
                mx = max(mx, max(max(w.z & 0x7FFFu, (w.z >> 16) & 0x7FFFu), max(w.w & 0x7FFFu, (w.w >> 16) & 0x7FFFu)));
            }
            if constexpr (HALF) mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 16));
            int e = (int)(mx >> 7);
            e = (e == 0 || e >= 254) ? 127 : e;   // zero, subnormal, huge or not finite: as it is
            down = __int_as_float((254 - e) << 23);
            up = __int_as_float(e << 23);
        }
        #pragma unroll 1
        for (int c = 0; c < QPT; c += 16) {
            uint32_t q[16];
            #pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint4 w = src ? p[c / 4 + i] : make_uint4(0, 0, 0, 0);
                q[4 * i] = w.x; q[4 * i + 1] = w.y; q[4 * i + 2] = w.z; q[4 * i + 3] = w.w;
            }
            if (half_form) {
                #pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const __half2 h = __floats2half2_rn(bf16lo(q[i]) * down, bf16hi(q[i]) * down);
                    q[i] = *reinterpret_cast<const uint32_t*>(&h);
                }
            }
            if constexpr (HALF) tmem_st16u_hx2<QPT>(q_addr + c, q);
            else tmem_st16(q_addr + c, q);
        }
        tmem_st_wait();
        tc_fence_before();
        return up;
    }
};

template <int HD, int MM>
__global__ void __launch_bounds__(KT_THREADS, 1) kv4_attn_tc_kernel(const KaArgs a, const DevErr err) {
    using Cfg = KtCfg<HD, MM>;
    using Bars = KtBars<Cfg::RST, Cfg::KST, Cfg::VST>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ Bars bars[KT_PIPES];
    __shared__ KaLineSmem<KT_THREADS> line_sm;
    __shared__ uint32_t tmem_holder;
    __shared__ int abort_flag;
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // warps 0-7 softmax, 8-15 expanders (four of each pipeline), 16, 17 producers, 18, 19 issuers
    const int pipe = warp < 16 ? (warp >> 2) & 1 : warp & 1;
    Bars& bb = bars[pipe];
    uint8_t* sK = sm + pipe * Cfg::PIPE;
    uint8_t* sV = sK + Cfg::KST * Cfg::TILE;
    uint8_t* sR = sV + Cfg::VST * Cfg::TILE;
    volatile int* abort = &abort_flag;

    if (threadIdx.x < KT_PIPES) {
        Bars& b = bars[threadIdx.x];
        for (int i = 0; i < Cfg::RST; ++i) { mbar_init(&b.raw_full[i], 1); mbar_init(&b.raw_empty[i], 4); }
        for (int i = 0; i < Cfg::KST; ++i) { mbar_init(&b.k_full[i], 4); mbar_init(&b.k_empty[i], 1); }
        for (int i = 0; i < Cfg::VST; ++i) { mbar_init(&b.v_full[i], 4); mbar_init(&b.v_empty[i], 1); }
        mbar_init(&b.q_full, 128); mbar_init(&b.s_full, 1); mbar_init(&b.p_full, 128); mbar_init(&b.pv_done, 1);
        mbar_init(&b.o_empty, 128); mbar_init(&b.drain, 1);
        if (threadIdx.x == 0) abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 16) { tmem_alloc(&tmem_holder, KT_PIPES * Cfg::COLS); tmem_relinquish(); }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_holder + pipe * Cfg::COLS;
    grid_dep_begin();

    // both pipelines' ranges: the line is cut into 2 * gridDim.x
    const int ranges = KT_PIPES * gridDim.x;
    KaLine line;
    for (int p = 0; p < KT_PIPES; ++p) {
        const KaLine l = ka_locate<KT_THREADS>(a, ranges, line_sm, err, [&](int per, int total) {
            const int64_t x = (int64_t)(KT_PIPES * blockIdx.x + p) * per;
            return x < total ? (int)x : -1;
        });
        if (p == pipe) line = l;
        __syncthreads();
    }
    const int range = KT_PIPES * blockIdx.x + pipe;
    const int64_t x0l = (int64_t)range * line.per;
    const bool work = x0l < line.total;
    const int x0 = work ? (int)x0l : 0, x1 = work ? x0 + min(line.total - x0, line.per) : 0;
    KaPos pos{};
    if (work) {
        pos.n = line.n;
        pos.len = ka_len(a, pos.n, err);
        pos.nu = ka_units(pos.len);
        pos.hs = (x0 - line.before) / pos.nu;
        pos.u = (x0 - line.before) - pos.hs * pos.nu;
    }
    // one unit further along the line (with the segment's bounds x < x1)
    auto advance = [&](KaPos& p) { if (++p.u == p.nu) p.next_triple(a, err); };

    if (warp >= 16 && warp < 18) {
        // ------------------------------------------------------------ producer
        KtRing<Cfg::RST> r;
        unsigned issued = 0;
        int base = -1, cells = 0;   // lane 4 i + w: pool cell w of unit base + i
        for (int x = x0; x < x1; ++x) {
            const int left = pos.len - pos.u * KA_UNIT;
            if (pos.u == pos.nu - 1) { base = -1; advance(pos); continue; }   // the block's own unit
            if (base < 0 || pos.u >= base + 8) {
                base = pos.u;
                const int k = base * KA_UNIT + lane * KV4_CELL_TOKENS;
                if (k < pos.len) {
                    const int j = k / a.slab.page, in = k - j * a.slab.page;
                    int p = a.table[(int64_t)pos.n * a.max_pages + j];
                    if (p < 0 || p >= a.slab.num_pages) { record_error(err, DFL_ERR_INVALID_ARG); p = 0; }
                    cells = (p * a.slab.Hkv + pos.hs / a.subs) * a.slab.cells + in / KV4_CELL_TOKENS;
                }
            }
            const int cell = __shfl_sync(0xFFFFFFFFu, cells, 4 * (pos.u - base) + (lane & 3));
            const int count = min(4, (left + KV4_CELL_TOKENS - 1) / KV4_CELL_TOKENS);
            const bool ok = kt_wait(&bb.raw_empty[r.i], r.ph ^ 1, err, abort);
            if (!__all_sync(0xFFFFFFFFu, ok)) break;
            if (lane == 0) mbar_arrive_expect_tx(&bb.raw_full[r.i], count * Cfg::CELL);
            __syncwarp();
            if (lane < count)
                bulk_g2s(sR + r.i * Cfg::RAW + lane * Cfg::CELL, a.slab.data + (int64_t)cell * Cfg::CELL, Cfg::CELL,
                         &bb.raw_full[r.i]);
            ++issued;
            r.step();
            advance(pos);
        }
        // copies in flight land before the CTA's shared memory goes (they have, unless a wait ran out)
        for (unsigned i = issued > Cfg::RST ? issued - Cfg::RST : 0; i < issued; ++i)
            mbar_wait(&bb.raw_full[i % Cfg::RST], (i / Cfg::RST) & 1, err);
    } else if (warp >= 18) {
        // -------------------------------------------------------------- issuer
        if (lane == 0) {
            KtRing<Cfg::KST> ks;
            KtRing<Cfg::VST> vs;
            uint32_t unit = 0, triple = 0, q_ph = 0;
            const uint32_t k32 = smem_u32(sK), v32 = smem_u32(sV);
            bool fresh = true, issued = false, ok = true;
            for (int x = x0; x < x1; ++x) {
                const bool own = pos.u == pos.nu - 1, last = own || x == x1 - 1;
                const uint32_t id_s = own ? idesc_bf16(MM, 64) : kt_idesc_f16(MM, 64);
                const uint32_t id_o = (own ? idesc_bf16(MM, HD) : kt_idesc_f16(MM, HD)) | (1u << 16);   // V is MN-major
                // Q in the form this unit needs; the previous unit's P V has read S's columns
                if (fresh || own) {
                    if (!(ok = kt_wait(&bb.q_full, q_ph, err, abort))) break;
                    q_ph ^= 1;
                }
                if (!(ok = kt_wait(&bb.k_full[ks.i], ks.ph, err, abort))) break;
                if (unit > 0 && !(ok = kt_wait(&bb.pv_done, (unit - 1) & 1, err, abort))) break;
                tc_fence_after();
                issued = true;
                #pragma unroll
                for (int j = 0; j < HD / 16; ++j)
                    mma_bf16_ts(tmem + Cfg::S_COL, tmem + Cfg::Q_COL + 8 * j,
                                sw128_desc(k32 + ks.i * Cfg::TILE + (j >> 2) * Cfg::TKB + (j & 3) * 32), id_s, j > 0);
                mma_commit(&bb.s_full);
                mma_commit(&bb.k_empty[ks.i]);
                if (!(ok = kt_wait(&bb.v_full[vs.i], vs.ph, err, abort))) break;
                // O is free once the previous triple's output has been read
                if (fresh && !(ok = kt_wait(&bb.o_empty, (triple & 1) ^ 1, err, abort))) break;
                if (!(ok = kt_wait(&bb.p_full, unit & 1, err, abort))) break;
                tc_fence_after();
                #pragma unroll
                for (int j = 0; j < 4; ++j)
                    mma_bf16_ts(tmem + Cfg::O_COL, tmem + Cfg::S_COL + 8 * j,
                                sw128_desc_mn(v32 + vs.i * Cfg::TILE + j * 16 * 128, Cfg::TKB, 1024), id_o,
                                (fresh && j == 0) ? 0 : 1);
                mma_commit(&bb.pv_done);
                mma_commit(&bb.v_empty[vs.i]);
                ks.step();
                vs.step();
                ++unit;
                fresh = last;
                if (last) ++triple;
                advance(pos);
            }
            if (!ok && issued) {   // products in flight end before tensor memory is released
                mma_commit(&bb.drain);
                mbar_wait(&bb.drain, 0, err);
            }
        }
    } else if (warp >= 8) {
        // ----------------------------------------------------------- expanders
        const int w = warp & 3;
        KtRing<Cfg::RST> r;
        KtRing<Cfg::KST> ks;
        KtRing<Cfg::VST> vs;
        for (int x = x0; x < x1; ++x) {
            const bool own = pos.u == pos.nu - 1;
            const int left = (own ? a.B : pos.len - pos.u * KA_UNIT) - w * KV4_CELL_TOKENS;
            uint8_t* kt = sK + ks.i * Cfg::TILE + w * 16 * 128;
            uint8_t* vt = sV + vs.i * Cfg::TILE + w * 16 * 128;
            const uint8_t* cell = sR + r.i * Cfg::RAW + w * Cfg::CELL;
            const int head = pos.hs / a.subs;
            const int64_t own_row = (int64_t)(pos.n * a.B + w * KV4_CELL_TOKENS) * a.slab.Hkv + head;
            bool ok = own || kt_wait(&bb.raw_full[r.i], r.ph, err, abort);
            ok = ok && kt_wait(&bb.k_empty[ks.i], ks.ph ^ 1, err, abort);
            if (!__all_sync(0xFFFFFFFFu, ok)) break;
            if (own) kt_block_rows<HD>(a.Kb + own_row * HD, (int64_t)a.slab.Hkv * HD, kt, lane, left);
            else if (left > 0) kt_expand_k<HD>(cell, kt, lane);   // rows without a key: masked scores
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bb.k_full[ks.i]);
            ok = kt_wait(&bb.v_empty[vs.i], vs.ph ^ 1, err, abort);
            if (!__all_sync(0xFFFFFFFFu, ok)) break;
            if (own || left <= 0) kt_block_rows<HD>(a.Vb + own_row * HD, (int64_t)a.slab.Hkv * HD, vt, lane, left);
            else kt_expand_v<HD>(cell, vt, lane, left);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&bb.v_full[vs.i]);
                if (!own) mbar_arrive(&bb.raw_empty[r.i]);
            }
            if (!own) r.step();
            ks.step();
            vs.step();
            advance(pos);
        }
    } else {
        // ------------------------------------------------------------- softmax
        using Row = KtRow<HD, MM>;
        constexpr bool HALF = Row::HALF;
        constexpr int KPT = Row::KPT, OPT = Row::OPT;
        const int q4 = warp & 3, hh = HALF ? lane >> 4 : 0;
        const int row = HALF ? 16 * q4 + (lane & 15) : 32 * q4 + lane;   // row of the triple held by this thread
        const uint32_t my = tmem + ((uint32_t)(q4 * 32) << 16);
        uint32_t unit = 0;
        bool ok = true;
        int x = x0;
        while (x < x1) {
            const int head = pos.hs / a.subs, row0 = (pos.hs - head * a.subs) * MM;
            const int u0 = pos.u, u1 = min(pos.nu, u0 + (x1 - x));
            const bool pad = row0 + (HALF ? 16 : 32) * q4 >= a.R;   // the warp holds no row of the block
            const int rr = row0 + row;
            const bool real = rr < a.R;
            const int64_t qrow = real ? (int64_t)(pos.n * a.B + rr / a.G) * a.Hq + head * a.G + rr % a.G : 0;
            const __nv_bfloat16* qsrc = real ? a.Q + qrow * HD : nullptr;
            float mult = 0.f, m = -INFINITY, l = 0.f;
            for (int u = u0; u < u1; ++u) {
                const bool own = u == pos.nu - 1;
                if (u == u0 || own) {   // the products that read Q before have ended: their S has been read
                    if (!pad) mult = Row::load_q(qsrc, hh, !own, my + Cfg::Q_COL) * a.scale_log2 * (own ? 1.f : a.k_pow2);
                    mbar_arrive(&bb.q_full);
                }
                ok = kt_wait(&bb.s_full, unit & 1, err, abort);
                if (!__all_sync(0xFFFFFFFFu, ok)) { ok = false; break; }
                tc_fence_after();
                if (!pad) {
                    // scores 32 at a time (at M = 128 read twice, once for the maximum: 64 in
                    // registers beside their weights spill)
                    float s[32], mt = -INFINITY;
                    auto load = [&](int k0) {
                        if constexpr (HALF) tmem_ld32_hx2<32>(my + Cfg::S_COL, s);
                        else tmem_ld32(my + Cfg::S_COL + k0, s);
                        const int valid = (own ? a.B : pos.len - u * KA_UNIT) - (HALF ? hh * 32 : k0);
                        if (valid < 32) {
                            #pragma unroll
                            for (int j = 0; j < 32; ++j)
                                if (j >= valid) s[j] = -INFINITY;
                        }
                    };
                    #pragma unroll 1
                    for (int k0 = 0; k0 < KPT; k0 += 32) {
                        load(k0);
                        float m4[4] = {s[0], s[1], s[2], s[3]};
                        #pragma unroll
                        for (int j = 4; j < 32; j += 4) {
                            m4[0] = fmaxf(m4[0], s[j]); m4[1] = fmaxf(m4[1], s[j + 1]);
                            m4[2] = fmaxf(m4[2], s[j + 2]); m4[3] = fmaxf(m4[3], s[j + 3]);
                        }
                        mt = fmaxf(mt, fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])));
                    }
                    if constexpr (HALF) mt = fmaxf(mt, __shfl_xor_sync(0xFFFFFFFFu, mt, 16));
                    mt *= mult;   // mult > 0: the maximum commutes
                    const bool need = mt > m + KA_LAZY;
                    if (u == u0) {
                        m = mt;
                    } else if (__any_sync(0xFFFFFFFFu, need)) {
                        // O holds the units before (S of this one was issued after their P V had ended)
                        const float mn = need ? mt : m, al = mn == m ? 1.f : ex2_ftz(m - mn);
                        #pragma unroll 1
                        for (int c = 0; c < OPT; c += 32) {
                            float o[32];
                            if constexpr (HALF) tmem_ld32_hx2<HD / 2>(my + Cfg::O_COL + c, o);
                            else tmem_ld32(my + Cfg::O_COL + c, o);
                            #pragma unroll
                            for (int j = 0; j < 32; ++j) o[j] *= al;
                            if constexpr (HALF) tmem_st32_hx2<HD / 2>(my + Cfg::O_COL + c, o);
                            else tmem_st32(my + Cfg::O_COL + c, o);
                        }
                        tmem_st_wait();
                        l *= al;
                        m = mn;
                    }
                    const float off = KA_LIFT - m;
                    #pragma unroll 1
                    for (int k0 = 0; k0 < KPT; k0 += 32) {
                        if (!HALF) load(k0);
                        float l4[4] = {0.f, 0.f, 0.f, 0.f};
                        #pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            s[j] = ex2_ftz(fmaf(s[j], mult, off));
                            l4[j & 3] += s[j];
                        }
                        l += (l4[0] + l4[1]) + (l4[2] + l4[3]);
                        uint32_t pk[16];
                        if (own) {   // O is kept in units of 2^v_exp
                            #pragma unroll
                            for (int j = 0; j < 32; j += 2) pk[j / 2] = pack_bf16(s[j] * a.v_inv, s[j + 1] * a.v_inv);
                        } else {
                            #pragma unroll
                            for (int j = 0; j < 32; j += 2) {
                                const __half2 h = __floats2half2_rn(s[j], s[j + 1]);
                                pk[j / 2] = *reinterpret_cast<const uint32_t*>(&h);
                            }
                        }
                        // P of 32 keys over 16 of S's columns that have been read
                        if constexpr (HALF) tmem_st16u_hx2<16>(my + Cfg::S_COL, pk);
                        else tmem_st16(my + Cfg::S_COL + k0 / 2, pk);
                    }
                    tmem_st_wait();
                }
                tc_fence_before();
                mbar_arrive(&bb.p_full);
                ++unit;
            }
            if (!ok) break;
            ok = kt_wait(&bb.pv_done, (unit - 1) & 1, err, abort);
            if (!__all_sync(0xFFFFFFFFu, ok)) { ok = false; break; }
            tc_fence_after();
            const bool whole = u0 == 0 && u1 == pos.nu;
            const int64_t part = ((int64_t)2 * range + (u0 == 0 ? 1 : 0)) * MM + row;
            if constexpr (HALF) l += __shfl_xor_sync(0xFFFFFFFFu, l, 16);
            const float inv = whole ? a.v_pow2 / l : 1.f;
            #pragma unroll 1
            for (int c0 = 0; c0 < OPT && !pad; c0 += 32) {
                float o[32];
                __syncwarp();
                if constexpr (HALF) tmem_ld32_hx2<HD / 2>(my + Cfg::O_COL + c0, o);
                else tmem_ld32(my + Cfg::O_COL + c0, o);
                if (!real) continue;
                const int c = hh * OPT + c0;
                if (whole) {
                    if (!DFL_IN_BOUNDS(err.word, qrow * HD + c + 31, (int64_t)a.N * a.B * a.Hq * HD)) continue;
                    uint4* dst = reinterpret_cast<uint4*>(a.O + qrow * HD + c);
                    #pragma unroll
                    for (int j = 0; j < 4; ++j)
                        dst[j] = make_uint4(pack_bf16(o[8 * j] * inv, o[8 * j + 1] * inv),
                                            pack_bf16(o[8 * j + 2] * inv, o[8 * j + 3] * inv),
                                            pack_bf16(o[8 * j + 4] * inv, o[8 * j + 5] * inv),
                                            pack_bf16(o[8 * j + 6] * inv, o[8 * j + 7] * inv));
                } else {
                    if (!DFL_IN_BOUNDS(err.word, part * HD + c + 31, (int64_t)2 * ranges * MM * HD)) continue;
                    float4* dst = reinterpret_cast<float4*>(a.Opart + part * HD + c);
                    #pragma unroll
                    for (int j = 0; j < 8; ++j) dst[j] = make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
                }
            }
            if (real && !whole && hh == 0 && DFL_IN_BOUNDS(err.word, part, (int64_t)2 * ranges * MM))
                a.ml[part] = make_float2(m, l);
            __syncwarp();
            tc_fence_before();
            mbar_arrive(&bb.o_empty);
            x += u1 - u0;
            pos.u = u1;
            if (u1 == pos.nu) pos.next_triple(a, err);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 16) {
        tc_fence_after();
        tmem_dealloc(tmem_holder, KT_PIPES * Cfg::COLS);
    }
}

constexpr int KT_SMS = 152;   // SMs of a GB300

int kt_grid(int64_t units) { return (int)std::min<int64_t>((units + KT_PIPES - 1) / KT_PIPES, KT_SMS); }

inline size_t al256(size_t b) { return (b + 255) & ~size_t(255); }

}  // namespace

size_t kv4_attn_tc_ws_bytes(int R, int hd) {
    const size_t rows = (size_t)2 * KT_PIPES * KT_SMS * kv4_attn_tc_rows(R);
    return al256(rows * hd * 4) + al256(rows * 8);
}

dfl_status kv4_attn_tc_run(DeviceCtx* ctx, KaArgs a, int hd, int64_t units, void* ws, cudaStream_t st) {
    const int mm = kv4_attn_tc_rows(a.R);
    const size_t rows = (size_t)2 * KT_PIPES * KT_SMS * mm;
    a.Opart = static_cast<float*>(ws);
    a.ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(ws) + al256(rows * hd * 4));
    const int grid = kt_grid(units);
    const DevErr err = dev_err(ctx);
    auto run = [&](auto kern, auto join, int smem, int slot) -> dfl_status {
        if (!ctx->kv4_attr_set[slot]) {
            if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
                return DFL_ERR_CUDA;
            ctx->kv4_attr_set[slot] = true;
        }
        {
            ProfScope ps("kv4_attn_tc", st);
            const dfl_status rc = launch_pdl(kern, grid, KT_THREADS, smem, st, a, err);
            if (rc != DFL_OK) return rc;
        }
        ProfScope ps("kv4_attn_join", st);
        return launch_pdl(join, dim3(KT_PIPES * grid, mm / KJ_ROWS), hd / 4 * KJ_ROWS, 0, st, a, err);
    };
    if (hd == 128)
        return mm == 64 ? run(kv4_attn_tc_kernel<128, 64>, kv4_attn_join_kernel<128, 64>, KtCfg<128, 64>::SMEM, 4)
                        : run(kv4_attn_tc_kernel<128, 128>, kv4_attn_join_kernel<128, 128>, KtCfg<128, 128>::SMEM, 5);
    return mm == 64 ? run(kv4_attn_tc_kernel<64, 64>, kv4_attn_join_kernel<64, 64>, KtCfg<64, 64>::SMEM, 6)
                    : run(kv4_attn_tc_kernel<64, 128>, kv4_attn_join_kernel<64, 128>, KtCfg<64, 128>::SMEM, 7);
}

}  // namespace dfl
