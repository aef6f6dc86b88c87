// Block attention over the 4-bit paged cache for many query rows per K/V head,
// on the 5th-generation tensor cores.  The same sum and the same line of work
// units as kv4_attn.cu, with up to 128 rows to a triple, where products and
// exponentials, not bytes, are most of the work.  A block of 16 at 4 query heads
// a K/V head (32 sequences of 2,048 tokens, 8 heads of 128): 51 us, 338 TFLOP/s
// of products and 1.7 TB/s of cache; 64 rows of a head of 64 over 33,333 to
// 100,001 tokens: 71.7 us; 128 rows: 74 and 106 us.
//
// One CTA per SM, two pipelines of eight warps, each with a range of the line of
// its own, so that one pipeline's products run under the other's exponentials:
//   expanders (4 warps) a quarter of a unit's keys each, K, then V: bulk copies
//                       of half cells into a ring of the warp's own, then codes
//                       * scales in fp16 into a tile [keys][hd] with 128-byte
//                       swizzle; the block's own rows come straight from memory;
//   softmax (4 warps)   Q as fp16 into shared memory, running maximum and sum,
//                       P over S's columns, the triple's output.  The first of
//                       them issues the products: S = Q K^T (M = 64 or 128
//                       rows, N = keys) and O += P V (N = hd, P from tensor
//                       memory).
// The issuing warp has nothing else to do between its P and the next S, which
// needs that P V to have read S's columns; a warp of its own would take the
// fifth place on its scheduler and with it 32 registers from every thread.
//
// What bounds it: how fast one warp issues, about one instruction in 4.7 clocks
// with four warps to a scheduler (dependent instructions, branches, fetches), so
// control code counts: the expanders' full units have a path of their own (the
// block of 16 above 57 us without).  Clocks of a pipeline per unit of 128 keys and
// 64 rows:
//   hd = 128  expanders 2 x 1,000 of expansion, 950 of copies ahead, 1,100 of
//             waits and arrivals: 4,100, the longest turn; S 900 to its commit,
//             450 until it is seen, softmax 1,500, P V 900, its end 260;
//   hd = 64   the products' chain, 2,900: S, 500, softmax 1,100, P V 640, 190;
//             the expanders wait for it.
// Hence units of 128 keys where shared and tensor memory allow (64 at hd = 128
// with 128 rows), and four expanders on K, then on V: two on each waited for
// their one tile's product in turn (64-row heads of 64 98 against 92 us then).
#include "internal.h"
#include "kv4_attn.cuh"
#include "paged.h"

namespace dfl {

namespace {

constexpr int KT_PIPES = 2;
constexpr int KT_WARPS = KT_PIPES * 8;         // softmax, expanders
constexpr int KT_THREADS = KT_WARPS * 32;
// |maximum| from which scores are multiplied before they are weighed: below it
// fp32 steps by at most 2^-2, and two roundings leave P under 2^15.6.
constexpr float KT_BIG = 4194304.f;   // 2^22

// Keys per unit.
constexpr int kt_unit(int hd, int mm) { return hd == 128 && mm == 128 ? 64 : 128; }

template <int HD, int MM>
struct KtCfg {
    static constexpr int KU = kt_unit(HD, MM);
    static constexpr int KB = HD / 64;                  // 128-byte blocks of a tile row
    static constexpr int TKB = KU * 128;                // bytes of one such block of a K or V tile
    static constexpr int QKB = MM * 128;                // of Q
    static constexpr int TILE = KB * TKB;
    static constexpr int Q = KB * QKB;
    static constexpr int CELL = Kv4Cell<HD>::BYTES;
    // slots per pipeline: codes of an expander's share of a unit (K and V as one copy where a few of them fit, else one
    // after the other), K and V tiles
    static constexpr int PARTS = HD == 64 || KU == 64 ? 1 : 2;
    static constexpr int RST = 3, ST = HD == 64 ? 2 : 1;
    static constexpr int SLOT = KU / 4 / KV4_CELL_TOKENS * CELL / PARTS;
    static constexpr int PIPE = Q + 2 * ST * TILE + RST * 4 * SLOT;
    static constexpr int S_COL = 0, O_COL = 128, COLS = 256;
    static constexpr int SMEM = 1024 + KT_PIPES * PIPE;
    static_assert(KU <= O_COL && O_COL + HD <= COLS, "tensor memory columns");
    static_assert(SMEM <= 225 * 1024, "shared memory");
    static_assert(PIPE % 1024 == 0, "tiles start on 1024-byte boundaries");
};

template <int RST, int ST>
struct KtBars {
    uint64_t raw_full[4][RST];   // of each expander
    uint64_t t_full[2][ST], t_empty[2][ST];   // of the K and the V tiles
    uint64_t q_full, s_full, p_full, pv_done, o_empty, drain;
};

__host__ __device__ constexpr uint32_t kt_idesc_f16(int M, int N) {   // fp16 A and B, fp32 sums
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// Wait as mbar_wait, and give up when another role of the CTA has.  Few
// instructions: the roles' waits are a good part of the kernel's code, and its
// loops barely fit the instruction cache.
__device__ __forceinline__ bool kt_wait(uint64_t* bar, uint32_t parity, const DevErr& e, volatile int* abort) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    #pragma unroll 1
    do {
        if (mbar_try_wait_for(bar, parity, 20000)) return true;
    } while (*abort == 0 && globaltimer_ns() - t0 <= e.limit_ns);
    if (*abort == 0) record_error(e, DFL_ERR_TIMEOUT);
    *abort = 1;
    return false;
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

// The expanders' shared-memory accesses by 32-bit address.  Volatile: they keep
// the order they are written in.
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ void sts128(uint32_t a, uint4 v) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" :: "r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// Where lane's piece c (16 bytes, 8 dims) of tile row `row` lies: KU rows of 128
// bytes, 128-byte swizzle, blocks of 64 dims one after the other.  Rows that
// differ in bits the start row has clear: (at ^ bits << 4) + rows * 128.
template <int KU>
__device__ __forceinline__ uint32_t kt_piece(uint32_t tile, int row, int c) {
    return tile + (c >> 3) * KU * 128 + row * 128 + (((c & 7) ^ (row & 7)) << 4);
}

// Expansion of the K or V half of a cell into 16 rows of a tile.  A quarter
// warp writes the eight 16-byte pieces of one tile row: no bank conflicts on
// either side.  All of a lane's words are read before the first is expanded:
// read one by one, each row waited for its own (the block of 16 above 67 us).
template <int HD, int KU>
struct KtExpandK {   // scores of tokens past the length are masked
    static __device__ __forceinline__ void run(uint32_t half, uint32_t tile, int lane) {
        using Cell = Kv4Cell<HD>;
        constexpr int WPR = HD / 8, RPL = 32 / WPR;   // words (8 codes) of a row, rows per warp-wide load
        constexpr int D = HD == 128 ? 1 : 2;          // slot s + RPL i is token + D i
        const int c = lane % WPR, h = lane / WPR;
        const uint32_t codes = half + h * Cell::ROW + 4 * c;
        const uint32_t scales = half + Cell::K_SCALES + (HD == 128 ? h * 16 + (c >> 2) * 4 : h * 8 + (c >> 1) * 2);
        const uint32_t at = kt_piece<KU>(tile, Cell::token(h), c);
        constexpr int NI = 8 / RPL;
        uint32_t w[2 * NI], sw[NI];                   // all of the lane's codes and scales are on their way before the first is used
        #pragma unroll
        for (int i = 0; i < NI; ++i) {                // slots s and s + 8, s = RPL i + h
            if constexpr (HD == 128) sw[i] = lds32(scales + RPL * i * 16);
            else sw[i] = lds16(scales + RPL * i * 8);
            w[2 * i] = lds32(codes + RPL * i * Cell::ROW);
            w[2 * i + 1] = lds32(codes + (RPL * i + 8) * Cell::ROW);
        }
        #pragma unroll
        for (int i = 0; i < NI; ++i) {
            uint32_t s0, s1;
            if constexpr (HD == 128) {
                const uint32_t sel = c & 2 ? 0x3232u : 0x1010u;
                const uint32_t h0 = e4m3x2_to_half(sw[i] & 0xFFFFu), h1 = e4m3x2_to_half(sw[i] >> 16);
                s0 = __byte_perm(h0, h0, sel);
                s1 = __byte_perm(h1, h1, sel);
            } else {
                const uint32_t hp = e4m3x2_to_half(sw[i]);
                s0 = __byte_perm(hp, hp, 0x1010);
                s1 = __byte_perm(hp, hp, 0x3232);
            }
            const uint32_t d = (at ^ (D * i << 4)) + D * i * 128;
            sts128(d, kt_expand(w[2 * i], s0));
            sts128(d + 8 * 128, kt_expand(w[2 * i + 1], s1));
        }
    }
};

template <int HD, int KU>
struct KtExpandV {   // tokens from `left` on become zeros: a weight of 0 times whatever is stored there must add nothing
    static __device__ __forceinline__ void run(uint32_t half, uint32_t tile, int lane, int left) {
        using Cell = Kv4Cell<HD>;
        constexpr int WPR = HD / 8, RPL = 32 / WPR;
        const int pos = lane % WPR, h = lane / WPR;
        const uint32_t codes = half + h * Cell::ROW + 4 * pos;
        const uint32_t scales = half + (Cell::V_SCALES - Cell::V_CODES) + h * 4;
        constexpr int NB = 4 / RPL;
        uint32_t w[4 * NB], sw[NB];
        #pragma unroll
        for (int b = 0; b < NB; ++b) {                // tokens t, 4 + t, 8 + t, 12 + t, t = RPL b + h
            const int c = HD == 128 && b ? pos ^ 8 : pos;   // tokens 2 and 3 of four: the row's halves trade places
            sw[b] = lds32(scales + (c >> 1) * 16 + RPL * b * 4);
            #pragma unroll
            for (int i = 0; i < 4; ++i) w[4 * b + i] = lds32(codes + (4 * i + RPL * b) * Cell::ROW);
        }
        if (left < KV4_CELL_TOKENS) {   // scale bytes of absent tokens
            #pragma unroll
            for (int b = 0; b < NB; ++b) {
                const int held = min(max((left - RPL * b - h + 3) >> 2, 0), 4);
                sw[b] &= held == 4 ? 0xFFFFFFFFu : (1u << 8 * held) - 1;
            }
        }
        #pragma unroll
        for (int b = 0; b < NB; ++b) {
            const int c = HD == 128 && b ? pos ^ 8 : pos;
            const uint32_t at = kt_piece<KU>(tile, h, c);
            const uint32_t sp[2] = {e4m3x2_to_half(sw[b] & 0xFFFFu), e4m3x2_to_half(sw[b] >> 16)};
            #pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = 4 * i + RPL * b;
                const uint32_t s = __byte_perm(sp[i >> 1], sp[i >> 1], i & 1 ? 0x3232 : 0x1010);
                sts128((at ^ ((r & 7) << 4)) + r * 128, kt_expand(w[4 * b + i], s));
            }
        }
    }
};

// 16 rows of a tile from bf16 rows of the block (zeros from `left` on), as fp16
// in units of the pool's power of two, like the cached values.
template <int HD, int KU>
__device__ __forceinline__ void kt_block_rows(const __nv_bfloat16* src, int64_t row_stride, uint32_t tile, int lane, int left,
                                              float inv) {
    constexpr int WPR = HD / 8, RPL = 32 / WPR, NR = 16 / RPL;
    const int c = lane % WPR, h = lane / WPR;
    const uint32_t at = kt_piece<KU>(tile, h, c);
    if (left <= 0) {
        #pragma unroll
        for (int i = 0; i < NR; ++i) sts128((at ^ (((RPL * i) & 7) << 4)) + RPL * i * 128, make_uint4(0, 0, 0, 0));
        return;
    }
    uint4 v[NR];   // all on their way before the first is used
    #pragma unroll
    for (int i = 0; i < NR; ++i) {
        const int tok = RPL * i + h;
        v[i] = tok < left ? *reinterpret_cast<const uint4*>(src + tok * row_stride + c * 8) : make_uint4(0, 0, 0, 0);
    }
    #pragma unroll
    for (int i = 0; i < NR; ++i) {
        const int r = RPL * i;
        sts128((at ^ ((r & 7) << 4)) + r * 128, block_half8(v[i], inv));
    }
}

// Bulk copies of the half cells that one expander warp needs, ahead of their use.
// A warp's share of a unit is KU / 4 keys; its cells are one ring slot and one
// step (PARTS = 1), or its K half cells are and its V half cells the next (2).
// Steps are numbered along a sequence.
template <int HD, int KU, int RST, int PARTS>
struct KtFeed {
    static constexpr int PART = Kv4Cell<HD>::BYTES / PARTS, SHARE = KU / 4, NC = SHARE / KV4_CELL_TOKENS;
    static constexpr int WIN = 32 / NC;   // units whose cells the lanes hold
    const KaArgs& a;
    const DevErr& err;
    uint8_t* ring;
    uint64_t* full;
    int w, lane;
    KaPos pos;                 // the segment after the one being copied
    int x, x1;                 // units of the range up to it, and in all
    int st = 0, end = 0, win = 0, len = 0, n = 0, head = 0;   // step copied next, end of the segment's, first unit of the window
    int cells = 0;             // lane NC i + j: pool cell j of the warp's in unit win + i
    uint32_t slot = 0, issued = 0;

    __device__ __forceinline__ KtFeed(const KaArgs& a_, const DevErr& err_, uint8_t* ring_, uint64_t* full_, int w_, int lane_,
                                      const KaPos& pos_, int x0, int x1_)
        : a(a_), err(err_), ring(ring_), full(full_), w(w_), lane(lane_), pos(pos_), x(x0), x1(x1_) {}

    __device__ __forceinline__ void window(int u) {
        win = u;
        const int k = (u + lane / NC) * KU + w * SHARE + lane % NC * KV4_CELL_TOKENS;
        if (k < len) cells = ka_cell(a, n, head, k, err);
    }
    // Whether a step with a token is left; moves to it.
    __device__ __forceinline__ bool more() {
        #pragma unroll 1
        while (st == end) {
            if (!pos.enter(x, x1)) return false;
            const int u1 = min(pos.nu, pos.u + (x1 - x));
            st = PARTS * pos.u;
            len = pos.len; n = pos.n; head = pos.head;
            end = max(st, PARTS * min(u1, (len - w * SHARE + KU - 1) / KU));   // units with a token of this warp's
            x += u1 - pos.u;
            if (u1 == pos.nu) pos.next_triple(a);
            win = st / PARTS - WIN;
        }
        return true;
    }
    // That step; one slot is free.
    __device__ __forceinline__ void produce() {
        const int u = st / PARTS;
        if (u == win + WIN) window(u);
        const int c0 = __shfl_sync(0xFFFFFFFFu, cells, NC * (u - win));
        const int c1 = NC == 2 ? __shfl_sync(0xFFFFFFFFu, cells, NC * (u - win) + 1) : 0;
        const bool more_than_one = NC == 2 && u * KU + w * SHARE + KV4_CELL_TOKENS < len;
        if (elect_one()) {
            uint8_t* d = ring + slot * NC * PART;
            const uint8_t* base = a.slab.data + st % PARTS * PART;
            mbar_arrive_expect_tx(&full[slot], more_than_one ? 2 * PART : PART);
            bulk_g2s(d, base + (int64_t)c0 * (PARTS * PART), PART, &full[slot]);
            if (more_than_one) bulk_g2s(d + PART, base + (int64_t)c1 * (PARTS * PART), PART, &full[slot]);
        }
        __syncwarp();
        slot = slot + 1 == RST ? 0 : slot + 1;
        ++issued;
        ++st;
    }
};

// One expander warp: a quarter of the keys of the K tile, then of the V tile, of
// all units of a range.
template <int HD, int KU, int RST, int PARTS, int ST>
__device__ __forceinline__ void kt_expander(const KaArgs& a, const DevErr& err, volatile int* abort, int w, int lane,
                                            uint8_t* ring, uint64_t* raw_full, uint32_t tiles, int tile_bytes,
                                            uint64_t (*t_full)[ST], uint64_t (*t_empty)[ST], KaPos pos, int x0, int x1) {
    constexpr int HALF = Kv4Cell<HD>::BYTES / 2;
    using Feed = KtFeed<HD, KU, RST, PARTS>;
    constexpr int PART = Feed::PART;
    constexpr int SHARE = Feed::SHARE, NC = Feed::NC;
    Feed feed(a, err, ring, raw_full, w, lane, pos, x0, x1);
    KtRing<RST> r;
    KtRing<ST> ts;
    uint32_t taken = 0;
    bool ok = true;
    int x = x0;
    pos.enter(x, x1);
    int u = pos.u, u1 = min(pos.nu, u + (x1 - x));
    auto own_ahead = [&] {   // the own rows of this triple on their way to L2
        const int row = w * SHARE + lane;
        if (lane >= SHARE || row >= a.B) return;
        const int64_t at = ((int64_t)(pos.n * a.B + row) * a.slab.Hkv + pos.head) * HD;
        #pragma unroll
        for (int i = 0; i < HD; i += 64) { prefetch_l2(a.Kb + at + i); prefetch_l2(a.Vb + at + i); }
    };
    if (x < x1) own_ahead();
    #pragma unroll 1
    while (x < x1) {
        const bool own = u == pos.nu - 1;
        const int share = w * SHARE;
        const int left = (own ? a.B : pos.len - u * KU) - share;   // keys of the unit from this warp's first on
        auto turn = [&](int half, auto&& expand) {
            if (PARTS == 2 || half == 0)
                if (feed.issued < taken + RST && feed.more()) feed.produce();
            ok = kt_wait(&t_empty[half][ts.i], ts.ph ^ 1, err, abort) && ((PARTS == 1 && half) || kt_wait(&raw_full[r.i], r.ph, err, abort));
            if (!__all_sync(0xFFFFFFFFu, ok)) { ok = false; return; }
            const uint32_t t = tiles + (half * ST + ts.i) * tile_bytes + share * 128;
            const uint32_t src = smem_u32(ring) + r.i * NC * PART + (PARTS == 1 ? half * HALF : 0);
            #pragma unroll
            for (int j = 0; j < NC; ++j) expand(src + j * PART, t + j * 16 * 128);
            fence_proxy_async_smem();
            __syncwarp();
            if (elect_one()) mbar_arrive(&t_full[half][ts.i]);
            if (PARTS == 2 || half) { ++taken; r.step(); }
        };
        if (!own && left >= SHARE && feed.issued > taken + 1) {
            turn(0, [&](uint32_t src, uint32_t t) { KtExpandK<HD, KU>::run(src, t, lane); });
            if (ok) turn(1, [&](uint32_t src, uint32_t t) { KtExpandV<HD, KU>::run(src, t, lane, KV4_CELL_TOKENS); });
        } else
        #pragma unroll 1
        for (int half = 0; half < 2; ++half) {   // K, V
            if (PARTS == 2 || half == 0)
                #pragma unroll 1
                while (feed.issued < taken + RST && feed.more()) feed.produce();
            const bool cell = !own && left > 0;
            ok = kt_wait(&t_empty[half][ts.i], ts.ph ^ 1, err, abort) && (!cell || (PARTS == 1 && half) || kt_wait(&raw_full[r.i], r.ph, err, abort));
            if (!__all_sync(0xFFFFFFFFu, ok)) { ok = false; break; }
            const uint32_t t = tiles + (half * ST + ts.i) * tile_bytes + share * 128;
            const uint32_t src = smem_u32(ring) + r.i * NC * PART + (PARTS == 1 ? half * HALF : 0);
            #pragma unroll 1
            for (int j = 0; j < NC; ++j) {   // 16 tokens at a time
                const int lj = left - j * KV4_CELL_TOKENS;
                if (!own && lj > 0) {
                    if (half) KtExpandV<HD, KU>::run(src + j * PART, t + j * 16 * 128, lane, lj);
                    else KtExpandK<HD, KU>::run(src + j * PART, t + j * 16 * 128, lane);
                } else if (own || half) {   // the block's own rows, zeros past B; zero values past the length
                    const int64_t at = ((int64_t)(pos.n * a.B + share + j * 16) * a.slab.Hkv + pos.head) * HD;
                    kt_block_rows<HD, KU>((half ? a.Vb : a.Kb) + at, (int64_t)a.slab.Hkv * HD, t + j * 16 * 128, lane, lj,
                                          half ? a.v_inv : a.k_inv);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();   // the slot has been read, the rows are written by every lane
            if (elect_one()) mbar_arrive(&t_full[half][ts.i]);
            if (cell && (PARTS == 2 || half)) { ++taken; r.step(); }
        }
        if (!ok) break;
        ts.step();
        ++x;
        if (++u == u1) {
            if (u1 == pos.nu) pos.next_triple(a);
            pos.enter(x, x1);
            u = pos.u;
            u1 = min(pos.nu, u + (x1 - x));
            if (x < x1) own_ahead();
        }
    }
    // copies in flight land before the CTA's shared memory goes (they have, unless a wait ran out)
    #pragma unroll 1
    for (; taken < feed.issued; ++taken) mbar_wait(&raw_full[taken % RST], (taken / RST) & 1, err);
}

// ROWS rows of Q (rows first .. first + ROWS - 1 of the triple; past R zeros)
// into the Q tile as fp16, each after the power of two that takes its largest
// element to [1, 2); the powers taken out go to up[].  One warp.
template <int HD, int MM, int ROWS>
__device__ __forceinline__ void kt_load_q(const KaArgs& a, int n, int head, int row0, int first, uint32_t tile, float* up, int lane) {
    constexpr int WPR = HD / 8, RPL = 32 / WPR;   // 16-byte pieces of a row, rows per warp-wide load
    const int c = lane % WPR, h = lane / WPR;
    constexpr int NB = 4;   // loads in flight
    #pragma unroll 1
    for (int i0 = 0; i0 < ROWS; i0 += NB * RPL) {
        uint4 v[NB];
        #pragma unroll
        for (int i = 0; i < NB; ++i) {
            const int r = row0 + first + i0 + i * RPL + h;
            v[i] = r < a.R ? *reinterpret_cast<const uint4*>(a.Q + ka_row(a, n, head, r, HD) + c * 8) : make_uint4(0, 0, 0, 0);
        }
        #pragma unroll
        for (int i = 0; i < NB; ++i) {
            const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
            uint32_t m2 = max_u16x2(max_u16x2(w[0] & 0x7FFF7FFFu, w[1] & 0x7FFF7FFFu),
                                    max_u16x2(w[2] & 0x7FFF7FFFu, w[3] & 0x7FFF7FFFu));
            uint32_t mx = max(m2 & 0xFFFFu, m2 >> 16), q[4];
            #pragma unroll
            for (int o = 1; o < WPR; o <<= 1) mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
            const int e = ka_query_exp(mx);
            const float down = __int_as_float((254 - e) << 23);
            #pragma unroll
            for (int j = 0; j < 4; ++j) {
                const __half2 hw = __floats2half2_rn(bf16lo(w[j]) * down, bf16hi(w[j]) * down);
                q[j] = *reinterpret_cast<const uint32_t*>(&hw);
            }
            const int row = first + i0 + i * RPL + h;
            sts128(tile + (c >> 3) * (MM * 128) + row * 128 + (((c & 7) ^ (row & 7)) << 4), make_uint4(q[0], q[1], q[2], q[3]));
            if (c == 0) up[row] = __int_as_float(e << 23);
        }
    }
}

// Softmax side: M = 128 gives a thread one row (its tensor-memory lane); at
// M = 64 the 16 rows of a warp's quadrant are shared by its two half-warps,
// each with half of a row's columns.
template <int HD, int MM>
__global__ void __launch_bounds__(KT_THREADS, 1) kv4_attn_tc_kernel(const KaArgs a, const DevErr err) {
    using Cfg = KtCfg<HD, MM>;
    using Bars = KtBars<Cfg::RST, Cfg::ST>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ Bars bars[KT_PIPES];
    __shared__ KaLineSmem<KT_THREADS, KT_PIPES> line_sm;
    __shared__ float q_up[KT_PIPES][MM];
    __shared__ uint32_t tmem_holder;
    __shared__ int abort_flag;
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // warps 0-7 softmax, 8-15 expanders, four of each pipeline
    const int pipe = (warp >> 2) & 1;
    Bars& bb = bars[pipe];
    uint8_t* sQ = sm + pipe * Cfg::PIPE;
    uint8_t* sK = sQ + Cfg::Q;
    uint8_t* sV = sK + Cfg::ST * Cfg::TILE;
    uint8_t* sR = sV + Cfg::ST * Cfg::TILE;
    volatile int* abort = &abort_flag;

    if (threadIdx.x < KT_PIPES) {
        Bars& b = bars[threadIdx.x];
        for (int i = 0; i < 4 * Cfg::RST; ++i) mbar_init(&b.raw_full[0][0] + i, 1);
        for (int i = 0; i < 2 * Cfg::ST; ++i) { mbar_init(&b.t_full[0][0] + i, 4); mbar_init(&b.t_empty[0][0] + i, 1); }
        mbar_init(&b.q_full, 4); mbar_init(&b.s_full, 1); mbar_init(&b.p_full, 4); mbar_init(&b.pv_done, 1);
        mbar_init(&b.o_empty, 4); mbar_init(&b.drain, 1);
        if (threadIdx.x == 0) abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 8) { tmem_alloc(&tmem_holder, KT_PIPES * Cfg::COLS); tmem_relinquish(); }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_holder + pipe * Cfg::COLS;
    grid_dep_begin();

    // ranges go round the CTAs, so that a few of them spread over the SMs
    const int ranges = KT_PIPES * gridDim.x;
    ka_check_lengths<KT_THREADS>(a, err);
    const KaLine line = ka_locate<KT_THREADS, KT_PIPES>(a, ranges, line_sm, [&](int p, int per, int total) {
        const int64_t x = (int64_t)(p * gridDim.x + blockIdx.x) * per;
        return x < total ? (int)x : -1;
    });
    const int range = pipe * gridDim.x + blockIdx.x;
    const int64_t x0l = (int64_t)range * line.per;
    KaPos pos{};
    int x0 = 0, x1 = 0;   // the range's units (none: x0 = x1)
    if (line.whole) {
        if (range < a.N * a.HS) {
            pos.set_triple(a, range);
            x1 = pos.nu;
        }
    } else if (x0l < line.total) {
        x0 = (int)x0l;
        x1 = x0 + min(line.total - x0, line.per);
        pos.set(a, line_sm.at[pipe], x0);
    }

    if (warp >= 8) {
        const int w = warp & 3;
        kt_expander<HD, Cfg::KU, Cfg::RST, Cfg::PARTS, Cfg::ST>(a, err, abort, w, lane, sR + w * Cfg::RST * Cfg::SLOT, bb.raw_full[w], smem_u32(sK),
                                                   Cfg::TILE, bb.t_full, bb.t_empty, pos, x0, x1);
    } else {
        // ------------------------------------------------------------- softmax
        constexpr bool HALF = MM == 64;
        constexpr int KU = Cfg::KU;
        constexpr int KPT = HALF ? KU / 2 : KU;      // keys per thread and unit
        constexpr int OPT = HALF ? HD / 2 : HD;      // O columns per thread
        constexpr int RPW = HALF ? 16 : 32;          // rows per warp
        const int q4 = warp & 3, hh = HALF ? lane >> 4 : 0;
        const int row = RPW * q4 + (HALF ? lane & 15 : lane);   // row of the triple held by this thread
        const uint32_t my = tmem + ((uint32_t)(q4 * 32) << 16), s_at = my + Cfg::S_COL;
        uint32_t unit = 0, triple = 0;
        bool ok = true, issued = false;
        // ---- products, by the first warp: one elected lane issues them (operands
        // the compiler knows to be uniform cost half the clocks per product of
        // those of a lone lane in a divergent branch, 8 products 214 against 510)
        const bool issuer = q4 == 0;
        KtRing<Cfg::ST> ks, vs;
        // descriptors of slot 0; slots and K blocks are added to the address field (16-byte units)
        const uint64_t qd = sw128_desc(smem_u32(sQ)), kd = sw128_desc(smem_u32(sK));
        const uint64_t vd = sw128_desc_mn(smem_u32(sV), Cfg::TKB, 1024);
        auto issue_s = [&](bool first) {   // S of the next unit; S's columns are free
            const bool ready = kt_wait(&bb.t_full[0][ks.i], ks.ph, err, abort) &&
                               (!first || kt_wait(&bb.q_full, triple & 1, err, abort));
            if (!__all_sync(0xFFFFFFFFu, ready)) return false;
            tc_fence_after();
            const uint64_t kdi = kd + ks.i * (Cfg::TILE >> 4);
            if (elect_one()) {
                #pragma unroll
                for (int j = 0; j < HD / 16; ++j)
                    mma_bf16(tmem + Cfg::S_COL, qd + (j >> 2) * (Cfg::QKB >> 4) + (j & 3) * 2,
                             kdi + (j >> 2) * (Cfg::TKB >> 4) + (j & 3) * 2, kt_idesc_f16(MM, KU), j > 0);
                mma_commit(&bb.s_full);
                mma_commit(&bb.t_empty[0][ks.i]);
            }
            __syncwarp();
            issued = true;
            ks.step();
            return true;
        };
        auto issue_pv = [&](bool first) {   // P of the unit written by all four warps
            const bool ready = kt_wait(&bb.t_full[1][vs.i], vs.ph, err, abort) &&
                               // O is free once the previous triple's output has been read
                               (!first || kt_wait(&bb.o_empty, (triple & 1) ^ 1, err, abort)) &&
                               kt_wait(&bb.p_full, unit & 1, err, abort);
            if (!__all_sync(0xFFFFFFFFu, ready)) return false;
            tc_fence_after();
            const uint64_t vdi = vd + vs.i * (Cfg::TILE >> 4);
            if (elect_one()) {
                #pragma unroll
                for (int j = 0; j < KU / 16; ++j)   // V is MN-major
                    mma_bf16_ts(tmem + Cfg::O_COL, tmem + Cfg::S_COL + 8 * j, vdi + j * (16 * 128 >> 4),
                                kt_idesc_f16(MM, HD) | (1u << 16), j > 0 || !first);
                mma_commit(&bb.pv_done);
                mma_commit(&bb.t_empty[1][vs.i]);
            }
            __syncwarp();
            vs.step();
            return true;
        };
        if (issuer && lane == 0) a.cross[range] = KaCross{-1, 0, 0, 0};
        int x = x0;
        while (pos.enter(x, x1)) {
            const int head = pos.head, row0 = pos.tile * MM;
            const int u0 = pos.u, u1 = min(pos.nu, u0 + (x1 - x));
            const bool pad = row0 + RPW * q4 >= a.R;   // the warp holds no row of the block
            // the products that read the previous Q have ended: their S has been read
            kt_load_q<HD, MM, RPW>(a, pos.n, head, row0, RPW * q4, smem_u32(sQ), q_up[pipe], lane);
            fence_proxy_async_smem();
            __syncwarp();
            if (elect_one()) mbar_arrive(&bb.q_full);
            if (issuer && !issue_s(true)) { ok = false; break; }
            const float mult = ka_mult(a, q_up[pipe][row]);
            if (x + u1 - u0 < x1) {   // the next triple's Q on its way to L2
                const bool wrap = pos.hs + 1 == a.HS;
                const int hs = wrap ? 0 : pos.hs + 1, nn = pos.n + wrap;
                const int nrow = (hs % a.subs) * MM + row;
                if (nrow < a.R) {
                    const __nv_bfloat16* p = a.Q + ka_row(a, nn, hs / a.subs, nrow, HD);
                    prefetch_l2(p + hh * (HD / 2));
                    if (!HALF && HD == 128) prefetch_l2(p + HD / 2);
                }
            }
            float m = KA_NONE, l = 0.f;
            bool big = false;   // some row of the warp has a maximum past KT_BIG
            for (int u = u0; u < u1; ++u) {
                ok = kt_wait(&bb.s_full, unit & 1, err, abort);
                if (!__all_sync(0xFFFFFFFFu, ok)) { ok = false; break; }
                tc_fence_after();
                if (!pad) {
                    // The maximum first: O is rescaled only where it grows by more than 2^8
                    // (S of this unit was issued after the P V of the units before had ended).
                    const int keys = (u == pos.nu - 1 ? a.B : pos.len - u * KU) - hh * KPT;   // from this thread's first on
                    if (__any_sync(0xFFFFFFFFu, keys < KPT)) {   // a unit's keys past the last: their scores become -inf
                        #pragma unroll 1
                        for (int k0 = 0; k0 < KPT; k0 += 16) {
                            float s[16];
                            if constexpr (HALF) tmem_ld16_hx2<KPT>(s_at + k0, s);
                            else tmem_ld16(s_at + k0, s);
                            uint32_t v[16];
                            #pragma unroll
                            for (int j = 0; j < 16; ++j) v[j] = k0 + j < keys ? __float_as_uint(s[j]) : 0xFF800000u;
                            if constexpr (HALF) tmem_st16u_hx2<KPT>(s_at + k0, v);
                            else tmem_st16(s_at + k0, v);
                        }
                        tmem_st_wait();
                    }
                    auto grow = [&] {   // the maximum; O is rescaled only where it grows by more than 2^8
                        float mt = -INFINITY;
                        #pragma unroll 1
                        for (int k0 = 0; k0 < KPT; k0 += 32) {
                            float s[32];
                            if constexpr (HALF) tmem_ld32_hx2<KPT>(s_at + k0, s);
                            else tmem_ld32(s_at + k0, s);
                            float m4[4] = {mt, -INFINITY, -INFINITY, -INFINITY};
                            #pragma unroll
                            for (int j = 0; j < 32; j += 2) m4[(j >> 1) & 3] = max3(m4[(j >> 1) & 3], s[j], s[j + 1]);
                            mt = max3(fmaxf(m4[0], m4[1]), m4[2], m4[3]);
                        }
                        if constexpr (HALF) mt = fmaxf(mt, __shfl_xor_sync(0xFFFFFFFFu, mt, 16));
                        mt *= mult;   // mult > 0: the maximum commutes
                        const bool need = mt > m + KA_LAZY;
                        if (__any_sync(0xFFFFFFFFu, need)) {
                            const float mn = need ? mt : m, al = mn == m ? 1.f : ex2_ftz(m - mn);
                            if (u > u0) {
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
                            }
                            l *= al;
                            m = mn;
                            big = __any_sync(0xFFFFFFFFu, fabsf(m) >= KT_BIG);
                        }
                    };
                    // The weights' exponent is s mult + (7 - m), one fused product and sum: the product is exact there and
                    // m rounded, which from KT_BIG on would lift P past fp16's range or drop it to 0.  Such scores are
                    // multiplied in place first.  (The block of 16 above takes 51.2 us with this look at `big`, 50.6
                    // without; products rounded for every score 51.9.  The compiler fuses a packed product and sum again.)
                    auto round_big = [&] {
                        if (__builtin_expect(!big, 1)) return;
                        #pragma unroll 1
                        for (int k0 = 0; k0 < KPT; k0 += 16) {
                            float s[16];
                            if constexpr (HALF) tmem_ld16_hx2<KPT>(s_at + k0, s);
                            else tmem_ld16(s_at + k0, s);
                            uint32_t v[16];
                            #pragma unroll
                            for (int j = 0; j < 16; ++j) v[j] = __float_as_uint(s[j] * mult);
                            if constexpr (HALF) tmem_st16u_hx2<KPT>(s_at + k0, v);
                            else tmem_st16(s_at + k0, v);
                        }
                        tmem_st_wait();
                    };
                    float2 off2, mult2, l2[2];
                    auto begin = [&] {
                        const float off = __fsub_rd(KA_LIFT, m);
                        off2 = make_float2(off, off);
                        mult2 = big ? make_float2(1.f, 1.f) : make_float2(mult, mult);
                        l2[0] = l2[1] = make_float2(0.f, 0.f);
                    };
                    auto weigh16 = [&](int k0, uint32_t* pk) {   // weights of 16 of this thread's keys, two per word
                        float s[16];
                        if constexpr (HALF) tmem_ld16_hx2<KPT>(s_at + k0, s);
                        else tmem_ld16(s_at + k0, s);
                        #pragma unroll
                        for (int j = 0; j < 16; j += 2) {
                            const float2 e = fma_f32x2(make_float2(s[j], s[j + 1]), mult2, off2);
                            const float2 p = make_float2(ex2_ftz(e.x), ex2_ftz(e.y));
                            l2[(j >> 1) & 1] = add_f32x2(l2[(j >> 1) & 1], p);
                            const __half2 h = __floats2half2_rn(p.x, p.y);
                            pk[j / 2] = *reinterpret_cast<const uint32_t*>(&h);
                        }
                    };
                    auto sum = [&] { return (l2[0].x + l2[0].y) + (l2[1].x + l2[1].y); };
                    // P, two keys per column, over the first half of S's columns
                    if constexpr (HALF) {   // both halves of a row share its columns: all of S is read first
                        // The weights by the maximum that is known: they stand when no thread's sum shows one past
                        // 2^15 (2^8 above the maximum); else, and at first, by the unit's own maximum.  With heads of
                        // 128 the look at the maximum hides under the expansion (with it the block of 16 takes 51.7 us,
                        // without 52.7); with heads of 64 it does not (64 rows over long contexts 81 and 74.5 us).
                        uint32_t pk[KPT / 16][8];
                        bool known = HD == 64 && u > u0 && !big;
                        #pragma unroll 1
                        while (true) {
                            if (!known) { grow(); round_big(); }
                            begin();
                            #pragma unroll
                            for (int g = 0; g < KPT / 16; ++g) weigh16(16 * g, pk[g]);
                            if (!known || !__any_sync(0xFFFFFFFFu, !(sum() <= 32768.f))) break;
                            known = false;
                        }
                        #pragma unroll
                        for (int g = 0; g < KPT / 16; g += 2) {
                            uint32_t v[16];
                            #pragma unroll
                            for (int j = 0; j < 16; ++j) v[j] = pk[g + j / 8][j % 8];
                            tmem_st16u_hx2<KPT / 2>(s_at + 8 * g, v);
                        }
                    } else {
                        grow();
                        round_big();
                        begin();
                        #pragma unroll 1
                        for (int k0 = 0; k0 < KPT; k0 += 16) {   // over columns already read
                            uint32_t pk[8];
                            weigh16(k0, pk);
                            tmem_st8u(s_at + k0 / 2, pk);
                        }
                    }
                    l += sum();
                    tmem_st_wait();
                }
                tc_fence_before();
                __syncwarp();
                if (elect_one()) mbar_arrive(&bb.p_full);
                if (issuer) {
                    ok = issue_pv(u == u0);
                    if (ok && u + 1 < u1) {
                        ok = kt_wait(&bb.pv_done, unit & 1, err, abort);
                        ok = __all_sync(0xFFFFFFFFu, ok) && issue_s(false);
                    }
                    if (!ok) break;
                }
                ++unit;
            }
            if (!ok) break;
            ok = kt_wait(&bb.pv_done, (unit - 1) & 1, err, abort);
            if (!__all_sync(0xFFFFFFFFu, ok)) { ok = false; break; }
            tc_fence_after();
            const bool whole = u0 == 0 && u1 == pos.nu;
            const int rr = row0 + row;
            const bool real = rr < a.R;
            const int64_t qrow = real ? ka_row(a, pos.n, head, rr, 1) : 0;
            const int64_t part = ((int64_t)2 * range + (u0 == 0 ? 1 : 0)) * MM + row;
            if constexpr (HALF) l += __shfl_xor_sync(0xFFFFFFFFu, l, 16);
            const float inv = whole ? __fdividef(a.v_pow2, l) : 1.f;
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
            tc_fence_before();
            __syncwarp();
            if (elect_one()) mbar_arrive(&bb.o_empty);
            if (u0 == 0 && u1 < pos.nu && issuer && lane == 0)
                a.cross[range] = KaCross{pos.n, head, pos.tile, (x + pos.nu - 1) / line.per};
            x += u1 - u0;
            pos.u = u1;
            if (u1 == pos.nu) pos.next_triple(a);
            ++triple;
        }
        if (!ok && issued) {   // products in flight end before tensor memory is released
            if (elect_one()) mma_commit(&bb.drain);
            __syncwarp();
            mbar_wait(&bb.drain, 0, err);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        tmem_dealloc(tmem_holder, KT_PIPES * Cfg::COLS);
    }
}

// See KaLine.  The seam, 0, 4, 8 and 16: the block of 16 above 59.8 us with 0 and
// 49.2 with the others, 32 sequences of 900 52.9 and 32.8, 16 of 900 29.4, 29.5,
// 26.7 and 26.7.  Weights of 1 and 3 give the same times.
constexpr int KT_SEAM = 8;
constexpr int KT_WEIGHT = 1;
constexpr int KT_SMS = 152;   // SMs of a GB300

int kt_grid(int64_t units) { return (int)std::min<int64_t>(units, KT_SMS); }

inline size_t al256(size_t b) { return (b + 255) & ~size_t(255); }

}  // namespace

int kv4_attn_tc_unit_log2(int R, int hd) { return kt_unit(hd, kv4_attn_tc_rows(R)) == 128 ? 7 : 6; }

int kv4_attn_tc_seam() { return KT_SEAM; }

int kv4_attn_tc_weight() { return KT_WEIGHT; }

size_t kv4_attn_tc_ws_bytes(int R, int hd) {
    const size_t rows = (size_t)2 * KT_PIPES * KT_SMS * kv4_attn_tc_rows(R);
    return al256(rows * hd * 4) + al256(rows * 8) + al256(sizeof(KaCross) * KT_PIPES * KT_SMS);
}

dfl_status kv4_attn_tc_run(DeviceCtx* ctx, KaArgs a, int hd, int64_t units, void* ws, cudaStream_t st) {
    const int mm = kv4_attn_tc_rows(a.R);
    const size_t rows = (size_t)2 * KT_PIPES * KT_SMS * mm;
    a.Opart = static_cast<float*>(ws);
    a.ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(ws) + al256(rows * hd * 4));
    a.cross = reinterpret_cast<KaCross*>(reinterpret_cast<uint8_t*>(a.ml) + al256(rows * 8));
    const int grid = kt_grid(units);
    const DevErr err = dev_err(ctx);
    auto run = [&](auto kern, auto join, int smem, int slot, int at_once) -> dfl_status {
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
        return launch_pdl(join, dim3(KT_PIPES * grid, mm / at_once), hd / 4 * at_once, 0, st, a, err);
    };
    if (hd == 128)
        return mm == 64 ? run(kv4_attn_tc_kernel<128, 64>, kv4_attn_join_kernel<128, 64>, KtCfg<128, 64>::SMEM, 4,
                              KjCfg<128, 64>::AT_ONCE)
                        : run(kv4_attn_tc_kernel<128, 128>, kv4_attn_join_kernel<128, 128>, KtCfg<128, 128>::SMEM, 5,
                              KjCfg<128, 128>::AT_ONCE);
    return mm == 64 ? run(kv4_attn_tc_kernel<64, 64>, kv4_attn_join_kernel<64, 64>, KtCfg<64, 64>::SMEM, 6,
                              KjCfg<64, 64>::AT_ONCE)
                    : run(kv4_attn_tc_kernel<64, 128>, kv4_attn_join_kernel<64, 128>, KtCfg<64, 128>::SMEM, 7,
                              KjCfg<64, 128>::AT_ONCE);
}

}  // namespace dfl
