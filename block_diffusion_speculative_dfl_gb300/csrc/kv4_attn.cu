// Block attention over the 4-bit paged context cache.
//
//   O = softmax(Q [Kc; Kb]^T / sqrt(hd)) [Vc; Vb]
// for the R = B * (Hq / Hkv) query rows that share K/V head h of sequence n:
// Kc, Vc the len[n] cached tokens of the sequence's pages (4-bit cells, see
// kv4.cuh), Kb, Vb the block's own B keys in bf16.  No mask.
//
// Work.  The keys of a sequence are cut into units of 64: ceil(len / 64)
// context units and one unit of the block's own keys.  All units of all
// (sequence, K/V head, row tile) triples in order form one line, cut into
// equal ranges, whatever the lengths: no range waits for a longer
// sequence, and the scratch depends on the grid alone.  A triple that lies
// within one range is written directly; one that crosses borders leaves
// one partial (sum, maximum, unnormalised O) per range, and a second kernel adds
// a triple's partials in the order of the keys, so results repeat bit for bit.
//
// A range belongs to a group of four warps; warp w takes tokens 16w .. 16w + 15
// (one cell) of every unit with its own running maximum, sum and O, so the
// warps meet only at the end of a triple.  One CTA per SM holds four such groups
// (three with 16 rows of 128): as CTAs of their own the hardware put five on one SM
// and three on another, and all waited for the five.  Each warp keeps a ring of
// cells in flight (one bulk copy of 18 hd bytes each, K, V and scales together)
// and expands codes in registers straight into operand fragments:
//   S^T (16 tokens x 8 rows)  = K Q^T,  A = K codes * scale in fp16
//   O^T (hd x 8 rows)        += V^T P^T, A = V codes * scale in fp16
// with m16n8k16 warp products.  At these row counts the kernel is bound by
// bytes and by the expansion, not by products: expanding into shared memory
// for tcgen05 operands would write and read 4 hd bytes per key more than the
// 9/8 hd that arrive, and that traffic alone takes longer than the reads from
// HBM (18 B per token and dimension pair through 128 B per clock and SM).
// Single tokens of 48 sequences of 65 to 16,000 (8 heads of 128, 4 query heads
// each): 93.4 us, 4.8 TB/s, 70 % of a copy's rate.  A cell of 16 tokens is about
// 370 warp instructions, 192 of them the conversions, scales and products; the
// schedulers issue in 66 % of the clocks, waiting for dependent results and for
// the conversion pipe.  More warps do not fit (five groups spill: 130 us).
//
// Numbers.  Expanded codes are exact in fp16.  Q is brought to fp16 after a
// power of two per row takes its largest element to [1, 2): bf16's 8 bits
// survive, elements below 2^-14 of the largest lose bits that are under 2^-24
// of it.  P = 2^(s - m + 7) is rounded to fp16 (11 bits; the 7 keeps weights
// down to 2^-31 of the largest, m trails the true maximum by at most 8); sums
// of P are fp32 of the unrounded values.  The block's own keys and values are
// taken to fp16 in units of the pool's powers of two (block_half8).  Maxima are
// per row; O is rescaled only when a maximum grows by more than 2^8.
#include "internal.h"
#include "kv4_attn.cuh"
#include "paged.h"

namespace dfl {

namespace {

constexpr int KA_UNIT = 64;        // keys per unit
constexpr int KA_WARPS = 4;        // of a group: one cell of 16 keys per warp and unit
constexpr int KA_THREADS = KA_WARPS * 32;
constexpr int KA_SLOTS = 3;        // cells in flight per warp

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

template <int HD, int NT>
struct KaCfg {
    static constexpr int ROWS = 8 * NT;               // query rows of a tile
    static constexpr int KSTEPS = HD / 16;            // products over the head dim
    static constexpr int MT = HD / 16;                // 16-dim tiles of O^T
    static constexpr int CELL = Kv4Cell<HD>::BYTES;
    static constexpr int PITCH = HD + 4;              // floats per row of the warps' O in shared memory
    static constexpr int GROUPS = HD == 128 && NT == 2 ? 3 : 4;   // per CTA (registers)
    static constexpr int THREADS = GROUPS * KA_THREADS;
    static constexpr int RING = KA_WARPS * KA_SLOTS * CELL;
    static constexpr int MERGE = KA_WARPS * 8 * PITCH * 4;   // of one 8-row tile
    static constexpr int QS = NT == 1 ? 0 : ROWS * HD * 2;   // Q of two tiles is read from here: registers (see below)
    static constexpr int ML = KA_WARPS * ROWS * 8;
    static constexpr int GROUP = (RING + MERGE + QS + ML + KA_WARPS * KA_SLOTS * 8 + 127) / 128 * 128;
    static constexpr int SMEM = GROUPS * GROUP;
    static_assert(SMEM <= 226 * 1024, "shared memory");
};

// The cells of one warp, copied ahead of their use.  Lane i holds the pool cell
// of the warp's tokens in unit win + i.
template <int HD, int ROWS>
struct KaFeed {
    static constexpr int CELL = Kv4Cell<HD>::BYTES;
    const KaArgs& a;
    const DevErr& err;
    uint8_t* ring;
    uint64_t* full;
    int w, lane;
    KaPos pos;                 // the segment after the one being copied
    int x, x1;                 // units of the range up to it, and in all
    int u = 0, end = 0, win = 0, cells = 0, len = 0, n = 0, head = 0;
    uint32_t issued = 0;

    __device__ __forceinline__ KaFeed(const KaArgs& a_, const DevErr& err_, uint8_t* ring_, uint64_t* full_, int w_, int lane_,
                                      const KaPos& pos_, int x0, int x1_)
        : a(a_), err(err_), ring(ring_), full(full_), w(w_), lane(lane_), pos(pos_), x(x0), x1(x1_) {}

    // The next cell into a free slot, if any is left.
    __device__ __forceinline__ void produce() {
        #pragma unroll 1
        while (u == end) {
            if (!pos.enter(x, x1)) return;
            u = pos.u;
            len = pos.len; n = pos.n; head = pos.head;
            const int u1 = min(pos.nu, u + (x1 - x));
            end = max(u, min(u1, (len - w * KV4_CELL_TOKENS + KA_UNIT - 1) / KA_UNIT));   // units with a token of this warp's
            x += u1 - u;
            // this triple's queries and own rows on their way to L2
            const int r = pos.tile * ROWS + 8 * w + lane / 4, b = w * KV4_CELL_TOKENS + lane / 2;
            if (8 * w < ROWS && r < a.R) prefetch_l2(a.Q + ka_row(a, n, head, r, HD) + lane % 4 * (HD / 4));
            if (u1 == pos.nu && b < a.B) {
                const int64_t at = ((int64_t)(n * a.B + b) * a.slab.Hkv + head) * HD + lane % 2 * (HD / 2);
                prefetch_l2(a.Kb + at);
                prefetch_l2(a.Vb + at);
            }
            if (u1 == pos.nu) pos.next_triple(a);
            win = u - 32;
        }
        if (u == win + 32) {
            win = u;
            const int k = (u + lane) * KA_UNIT + w * KV4_CELL_TOKENS;
            if (k < len) cells = ka_cell(a, n, head, k, err);
        }
        const int cell = __shfl_sync(0xFFFFFFFFu, cells, u - win);
        if (elect_one()) {
            const uint32_t s = issued % KA_SLOTS;
            mbar_arrive_expect_tx(&full[s], CELL);
            bulk_g2s(ring + s * CELL, a.slab.data + (int64_t)cell * CELL, CELL, &full[s]);
        }
        __syncwarp();
        ++issued;
        ++u;
    }
};

// All threads of one group.
__device__ __forceinline__ void group_sync(int group) { asm volatile("bar.sync %0, 128;" :: "r"(group + 1) : "memory"); }

// State of one warp over one triple: per lane, for query rows 2t and 2t + 1 of
// each 8-row tile (t = lane % 4).
template <int HD, int NT>
struct KaAcc {
    float o[NT][HD / 16][4];   // O^T: dims of this lane's eighth (lane / 4) x the two rows
    float m[NT][2], l[NT][2];
};

// Softmax of one cell: s[nt] = (slot g, rows 2t, 2t+1), (slot g + 8, same), in
// log2 units, masked slots -inf.  Updates m, l, rescales O; s becomes P.
template <int HD, int NT>
__device__ __forceinline__ void ka_softmax(KaAcc<HD, NT>& acc, float (&s)[NT][4]) {
    bool need = false;
    #pragma unroll
    for (int nt = 0; nt < NT; ++nt)
        need |= fmaxf(s[nt][0], s[nt][2]) > acc.m[nt][0] + KA_LAZY || fmaxf(s[nt][1], s[nt][3]) > acc.m[nt][1] + KA_LAZY;
    if (__any_sync(0xFFFFFFFFu, need)) {
        #pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            #pragma unroll
            for (int r = 0; r < 2; ++r) {
                float mx = fmaxf(s[nt][r], s[nt][r + 2]);
                #pragma unroll
                for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
                const float mo = acc.m[nt][r], mn = fmaxf(mo, mx);
                const float al = mn == mo ? 1.f : ex2_ftz(mo - mn);   // 0 for the first cell
                acc.m[nt][r] = mn;
                acc.l[nt][r] *= al;
                #pragma unroll
                for (int i = 0; i < HD / 16; ++i) { acc.o[nt][i][r] *= al; acc.o[nt][i][r + 2] *= al; }
            }
        }
    }
    #pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        #pragma unroll
        for (int r = 0; r < 2; ++r) {
            const float off = __fsub_rd(KA_LIFT, acc.m[nt][r]);
            s[nt][r] = ex2_ftz(s[nt][r] + off);
            s[nt][r + 2] = ex2_ftz(s[nt][r + 2] + off);
            acc.l[nt][r] += s[nt][r] + s[nt][r + 2];
        }
    }
}

template <int HD, int NT>
__global__ void __launch_bounds__(KaCfg<HD, NT>::THREADS, 1) kv4_attn_kernel(const KaArgs a, const DevErr err) {
    using Cfg = KaCfg<HD, NT>;
    using Cell = Kv4Cell<HD>;
    constexpr int KW = HD / 32;          // words of a lane's quarter of a K row (codes)
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ KaLineSmem<Cfg::THREADS, Cfg::GROUPS> line_sm;
    const int group = threadIdx.x / KA_THREADS, tid = threadIdx.x % KA_THREADS;
    const int warp = tid >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    uint8_t* sm = smem + group * Cfg::GROUP;
    uint8_t* ring = sm + warp * KA_SLOTS * Cfg::CELL;
    float* merge = reinterpret_cast<float*>(sm + Cfg::RING);
    uint4* qs = reinterpret_cast<uint4*>(sm + Cfg::RING + Cfg::MERGE);
    float2* mlsm = reinterpret_cast<float2*>(sm + Cfg::RING + Cfg::MERGE + Cfg::QS);
    uint64_t* full = reinterpret_cast<uint64_t*>(sm + Cfg::RING + Cfg::MERGE + Cfg::QS + Cfg::ML) + warp * KA_SLOTS;
    if (lane == 0) {
        for (int i = 0; i < KA_SLOTS; ++i) mbar_init(&full[i], 1);
        fence_barrier_init();
    }
    __syncwarp();
    grid_dep_begin();

    ka_check_lengths<Cfg::THREADS>(a, err);
    // ranges go round the CTAs, so that a few of them spread over the SMs
    const int ranges = Cfg::GROUPS * gridDim.x, range = group * gridDim.x + blockIdx.x;
    const KaLine line = ka_locate<Cfg::THREADS, Cfg::GROUPS>(a, ranges, line_sm, [&](int i, int per, int total) {
        const int64_t x = (int64_t)(i * gridDim.x + blockIdx.x) * per;
        return x < total ? (int)x : -1;
    });
    const int64_t x0l = (int64_t)range * line.per;
    if (tid == 0) a.cross[range] = KaCross{-1, 0, 0, 0};
    if (line.whole ? range >= a.N * a.HS : x0l >= line.total) return;   // no block-wide barrier follows
    const int x0 = line.whole ? 0 : (int)x0l;

    KaPos pos;   // the triple being computed
    if (line.whole) pos.set_triple(a, range);
    else pos.set(a, line_sm.at[group], x0);
    const int x1 = line.whole ? pos.nu : min(line.total - x0, line.per) + x0;

    KaFeed<HD, Cfg::ROWS> feed(a, err, ring, full, warp, lane, pos, x0, x1);
    uint32_t taken = 0;
    bool dead = false;         // a wait ran out: no more copies, no more computation
    #pragma unroll 1
    for (int i = 0; i < KA_SLOTS; ++i) feed.produce();

    int x = x0;
    #pragma unroll 1
    while (pos.enter(x, x1)) {
        const int head = pos.head, row0 = pos.tile * Cfg::ROWS;
        const int u0 = pos.u, u1 = min(pos.nu, u0 + (x1 - x));
        // ---- Q of this triple: lane (g, t) holds row g's quarter t of each 8-row tile
        uint32_t q1[2 * Cfg::KSTEPS];   // (NT = 1)
        float mult[NT][2];   // rows 2t, 2t + 1: score of fp16 operands -> log2 units
        #pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int r = row0 + nt * 8 + g;
            uint32_t q[2 * Cfg::KSTEPS];
            uint32_t mx = 0;
            const uint4* src = reinterpret_cast<const uint4*>(
                a.Q + ka_row(a, pos.n, head, r, HD) + t * (HD / 4));
            #pragma unroll
            for (int i = 0; i < HD / 32; ++i) {
                const uint4 w = r < a.R ? src[i] : make_uint4(0, 0, 0, 0);
                q[4 * i] = w.x; q[4 * i + 1] = w.y; q[4 * i + 2] = w.z; q[4 * i + 3] = w.w;
            }
            #pragma unroll
            for (int i = 0; i < 2 * Cfg::KSTEPS; ++i) mx = max(mx, max(q[i] & 0x7FFFu, (q[i] >> 16) & 0x7FFFu));
            mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
            mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
            const int e = ka_query_exp(mx);
            const float down = __int_as_float((254 - e) << 23);
            #pragma unroll
            for (int i = 0; i < 2 * Cfg::KSTEPS; ++i) q[i] = pack_half(bf16lo(q[i]) * down, bf16hi(q[i]) * down);
            if constexpr (NT == 1) {
                #pragma unroll
                for (int i = 0; i < 2 * Cfg::KSTEPS; ++i) q1[i] = q[i];
            } else if (warp == nt) {   // a warp per tile writes it for all
                #pragma unroll
                for (int i = 0; i < HD / 32; ++i) qs[(nt * (HD / 32) + i) * 32 + lane] = make_uint4(q[4 * i], q[4 * i + 1], q[4 * i + 2], q[4 * i + 3]);
            }
            const float up = ka_mult(a, __int_as_float(e << 23));
            mult[nt][0] = __shfl_sync(0xFFFFFFFFu, up, 8 * t);       // lane of row 2t
            mult[nt][1] = __shfl_sync(0xFFFFFFFFu, up, 8 * t + 4);   // lane of row 2t + 1
        }
        // Two tiles' Q would take 32 registers beside 64 of O (hd = 128): spilled, 16 rows over the single-token
        // batch's lengths take 150 us, read from shared memory 136.
        if constexpr (NT > 1) group_sync(group);
        // words 4i .. 4i + 3 of this lane's quarter of its row of tile nt
        auto q_words = [&](int nt, int i) {
            if constexpr (NT == 1) return make_uint4(q1[4 * i], q1[4 * i + 1], q1[4 * i + 2], q1[4 * i + 3]);
            else return qs[(nt * (HD / 32) + i) * 32 + lane];
        };
        KaAcc<HD, NT> acc;
        #pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            #pragma unroll
            for (int i = 0; i < Cfg::MT; ++i)
                #pragma unroll
                for (int c = 0; c < 4; ++c) acc.o[nt][i][c] = 0.f;
            acc.m[nt][0] = acc.m[nt][1] = KA_NONE;
            acc.l[nt][0] = acc.l[nt][1] = 0.f;
        }
        // ---- context cells
        const int ctx_end = min(u1, pos.nu - 1);
        #pragma unroll 1
        for (int u = u0; u < ctx_end; ++u) {
            const int left = pos.len - u * KA_UNIT - warp * KV4_CELL_TOKENS;   // tokens from this cell on
            if (left <= 0 || dead) continue;
            const int sl = taken % KA_SLOTS;
            const bool ok = mbar_wait(&full[sl], (taken / KA_SLOTS) & 1, err);
            if (!__all_sync(0xFFFFFFFFu, ok)) { dead = true; continue; }
            const uint8_t* cell = ring + sl * Cfg::CELL;
            ++taken;
            float s[NT][4];
            #pragma unroll
            for (int nt = 0; nt < NT; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
            {   // S^T: slots g and g + 8
                uint32_t kc[2][KW];   // codes of this lane's quarter
                #pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint8_t* p = cell + Cell::K_CODES + (g + 8 * h) * Cell::ROW + t * (Cell::ROW / 4);
                    if constexpr (HD == 128) {
                        const uint4 w = *reinterpret_cast<const uint4*>(p);
                        kc[h][0] = w.x; kc[h][1] = w.y; kc[h][2] = w.z; kc[h][3] = w.w;
                    } else {
                        const uint2 w = *reinterpret_cast<const uint2*>(p);
                        kc[h][0] = w.x; kc[h][1] = w.y;
                    }
                }
                uint32_t sc[2][HD / 64];   // fp16 pairs (s, s) of the lane's groups
                if constexpr (HD == 128) {
                    const uint32_t w = *reinterpret_cast<const uint32_t*>(cell + Cell::K_SCALES + lane * 4);
                    const uint32_t h0 = e4m3x2_to_half(w & 0xFFFFu), h1 = e4m3x2_to_half(w >> 16);
                    sc[0][0] = __byte_perm(h0, h0, 0x1010); sc[0][1] = __byte_perm(h0, h0, 0x3232);
                    sc[1][0] = __byte_perm(h1, h1, 0x1010); sc[1][1] = __byte_perm(h1, h1, 0x3232);
                } else {
                    const uint32_t w = *reinterpret_cast<const uint16_t*>(cell + Cell::K_SCALES + lane * 2);
                    const uint32_t h0 = e4m3x2_to_half(w);
                    sc[0][0] = __byte_perm(h0, h0, 0x1010);
                    sc[1][0] = __byte_perm(h0, h0, 0x3232);
                }
                #pragma unroll
                for (int w = 0; w < KW; ++w) {   // 8 dims: two products over the head dim
                    uint32_t h0[4], h1[4];
                    e2m1x8_to_half(kc[0][w], h0);
                    e2m1x8_to_half(kc[1][w], h1);
                    #pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        h0[i] = hmul2u(h0[i], sc[0][w / 2]);
                        h1[i] = hmul2u(h1[i], sc[1][w / 2]);
                    }
                    #pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const uint32_t af[4] = {h0[2 * j], h1[2 * j], h0[2 * j + 1], h1[2 * j + 1]};
                        #pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            const uint4 qw = q_words(nt, w);
                            mma_f16(s[nt], af, j ? qw.z : qw.x, j ? qw.w : qw.y);
                        }
                    }
                }
            }
            #pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                #pragma unroll
                for (int c = 0; c < 4; ++c) s[nt][c] = __fmul_rn(s[nt][c], mult[nt][c & 1]);   // rounded before 7 - m is added
            if (left < KV4_CELL_TOKENS) {   // the cell's last tokens do not exist
                const bool v0 = Cell::token(g) < left, v1 = Cell::token(g + 8) < left;
                #pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    if (!v0) s[nt][0] = s[nt][1] = -INFINITY;
                    if (!v1) s[nt][2] = s[nt][3] = -INFINITY;
                }
            }
            ka_softmax<HD, NT>(acc, s);
            uint32_t pb[NT][2];
            #pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                pb[nt][0] = transpose8x8(pack_half(s[nt][0], s[nt][1]));
                pb[nt][1] = transpose8x8(pack_half(s[nt][2], s[nt][3]));
            }
            {   // O^T: tokens t, 4 + t (slots 2t, 2t + 1) and 8 + t, 12 + t
                const int vg = HD == 128 ? g : g >> 1;
                uint32_t sw = *reinterpret_cast<const uint32_t*>(cell + Cell::V_SCALES + vg * 16 + t * 4);
                uint32_t sp[2] = {e4m3x2_to_half(sw & 0xFFFFu), e4m3x2_to_half(sw >> 16)};
                if (left < KV4_CELL_TOKENS) {   // weight 0 times a stored NaN would be NaN
                    #pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        if (8 * i + t >= left) sp[i] &= 0xFFFF0000u;
                        if (8 * i + 4 + t >= left) sp[i] &= 0x0000FFFFu;
                    }
                }
                uint32_t ev[2][HD / 64], od[2][HD / 64];   // (token pair) x even / odd dims of the lane's eighth
                #pragma unroll
                for (int i = 0; i < 2; ++i) {
                    uint32_t A[HD / 64], Bw[HD / 64];
                    const uint8_t* pa = cell + Cell::V_CODES + (8 * i + t) * Cell::ROW;
                    const uint8_t* pbp = pa + 4 * Cell::ROW;
                    if constexpr (HD == 128) {
                        const int off = (g * 8) ^ Cell::v_swap(t);   // tokens t and t + 4 k swap alike
                        const uint2 wa = *reinterpret_cast<const uint2*>(pa + off);
                        const uint2 wb = *reinterpret_cast<const uint2*>(pbp + off);
                        A[0] = wa.x; A[1] = wa.y; Bw[0] = wb.x; Bw[1] = wb.y;
                    } else {
                        A[0] = *reinterpret_cast<const uint32_t*>(pa + g * 4);
                        Bw[0] = *reinterpret_cast<const uint32_t*>(pbp + g * 4);
                    }
                    #pragma unroll
                    for (int w = 0; w < HD / 64; ++w) {
                        ev[i][w] = (A[w] & 0x0F0F0F0Fu) | ((Bw[w] << 4) & 0xF0F0F0F0u);
                        od[i][w] = ((A[w] >> 4) & 0x0F0F0F0Fu) | (Bw[w] & 0xF0F0F0F0u);
                    }
                }
                #pragma unroll
                for (int w = 0; w < HD / 64; ++w) {
                    uint32_t e0[4], e1[4], o0[4], o1[4];
                    e2m1x8_to_half(ev[0][w], e0);
                    e2m1x8_to_half(ev[1][w], e1);
                    e2m1x8_to_half(od[0][w], o0);
                    e2m1x8_to_half(od[1][w], o1);
                    #pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t af[4] = {hmul2u(e0[i], sp[0]), hmul2u(o0[i], sp[0]), hmul2u(e1[i], sp[1]),
                                                hmul2u(o1[i], sp[1])};
                        #pragma unroll
                        for (int nt = 0; nt < NT; ++nt) mma_f16(acc.o[nt][4 * w + i], af, pb[nt][0], pb[nt][1]);
                    }
                }
            }
            __syncwarp();   // the slot has been read by every lane
            feed.produce();
        }
        // ---- the block's own keys, 16 per warp
        if (u1 == pos.nu && warp * KV4_CELL_TOKENS < a.B && !dead) {
            const int Hkv = a.slab.Hkv;
            float s[NT][4];
            #pragma unroll
            for (int nt = 0; nt < NT; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
            const int b0 = warp * KV4_CELL_TOKENS + Cell::token(g), b1 = warp * KV4_CELL_TOKENS + Cell::token(g + 8);
            const uint4* k0 = reinterpret_cast<const uint4*>(a.Kb + ((int64_t)(pos.n * a.B + b0) * Hkv + head) * HD + t * (HD / 4));
            const uint4* k1 = reinterpret_cast<const uint4*>(a.Kb + ((int64_t)(pos.n * a.B + b1) * Hkv + head) * HD + t * (HD / 4));
            #pragma unroll
            for (int i = 0; i < HD / 32; ++i) {
                const uint4 z = make_uint4(0, 0, 0, 0);
                const uint4 w0 = block_half8(b0 < a.B ? k0[i] : z, a.k_inv), w1 = block_half8(b1 < a.B ? k1[i] : z, a.k_inv);
                const uint32_t f0[4] = {w0.x, w1.x, w0.y, w1.y}, f1[4] = {w0.z, w1.z, w0.w, w1.w};
                #pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const uint4 qw = q_words(nt, i);
                    mma_f16(s[nt], f0, qw.x, qw.y);
                    mma_f16(s[nt], f1, qw.z, qw.w);
                }
            }
            #pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                #pragma unroll
                for (int c = 0; c < 4; ++c) s[nt][c] = (c < 2 ? b0 : b1) < a.B ? __fmul_rn(s[nt][c], mult[nt][c & 1]) : -INFINITY;
            ka_softmax<HD, NT>(acc, s);
            uint32_t pb[NT][2];
            #pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                pb[nt][0] = transpose8x8(pack_half(s[nt][0], s[nt][1]));
                pb[nt][1] = transpose8x8(pack_half(s[nt][2], s[nt][3]));
            }
            #pragma unroll
            for (int w = 0; w < HD / 64; ++w) {   // 8 dims of the lane's eighth at a time
                uint32_t v[4][4];
                #pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int b = warp * KV4_CELL_TOKENS + 4 * i + t;
                    const uint4 x4 = block_half8(b < a.B ? *reinterpret_cast<const uint4*>(
                        a.Vb + ((int64_t)(pos.n * a.B + b) * Hkv + head) * HD + g * (HD / 8) + 8 * w) : make_uint4(0, 0, 0, 0), a.v_inv);
                    v[i][0] = x4.x; v[i][1] = x4.y; v[i][2] = x4.z; v[i][3] = x4.w;
                }
                #pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t af[4] = {__byte_perm(v[0][i], v[1][i], 0x5410), __byte_perm(v[0][i], v[1][i], 0x7632),
                                            __byte_perm(v[2][i], v[3][i], 0x5410), __byte_perm(v[2][i], v[3][i], 0x7632)};
                    #pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma_f16(acc.o[nt][4 * w + i], af, pb[nt][0], pb[nt][1]);
                }
            }
        }
        // ---- the warps' parts of this triple
        #pragma unroll
        for (int nt = 0; nt < NT; ++nt) {   // a tile at a time: shared memory
            if (nt > 0) group_sync(group);
            #pragma unroll
            for (int r = 0; r < 2; ++r) {
                float l = acc.l[nt][r];
                #pragma unroll
                for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
                const int row = nt * 8 + 2 * t + r;
                if (g == 0) mlsm[warp * Cfg::ROWS + row] = make_float2(acc.m[nt][r], l);
                float* dst = merge + (warp * 8 + 2 * t + r) * Cfg::PITCH + g * (HD / 8);
                #pragma unroll
                for (int i = 0; i < Cfg::MT; i += 2)
                    *reinterpret_cast<float4*>(dst + 2 * i) = make_float4(acc.o[nt][i][r], acc.o[nt][i][r + 2],
                                                                          acc.o[nt][i + 1][r], acc.o[nt][i + 1][r + 2]);
            }
            group_sync(group);
            const bool whole = u0 == 0 && u1 == pos.nu;
            const int part = 2 * range + (u0 == 0 ? 1 : 0);
            constexpr int TPR = HD / 4;   // threads per row
            #pragma unroll 1
            for (int row = nt * 8 + tid / TPR; row < nt * 8 + 8; row += KA_THREADS / TPR) {
                const int r = row0 + row, c = (tid % TPR) * 4;
                if (r >= a.R) break;
                float2 ml[KA_WARPS];
                float M = KA_NONE, L = 0.f;
                #pragma unroll
                for (int w = 0; w < KA_WARPS; ++w) { ml[w] = mlsm[w * Cfg::ROWS + row]; M = fmaxf(M, ml[w].x); }
                float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
                #pragma unroll
                for (int w = 0; w < KA_WARPS; ++w) {
                    const float f = ex2_ftz(ml[w].x - M);
                    const float4 v = *reinterpret_cast<const float4*>(merge + (w * 8 + row - nt * 8) * Cfg::PITCH + c);
                    L += f * ml[w].y;
                    o.x += f * v.x; o.y += f * v.y; o.z += f * v.z; o.w += f * v.w;
                }
                if (whole) {
                    const float inv = __fdividef(a.v_pow2, L);
                    const int64_t at = ka_row(a, pos.n, head, r, HD) + c;
                    if (DFL_IN_BOUNDS(err.word, at + 3, (int64_t)a.N * a.B * a.Hq * HD))
                        *reinterpret_cast<uint2*>(a.O + at) =
                            make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
                } else {
                    const int64_t at = ((int64_t)part * Cfg::ROWS + row) * HD + c;
                    if (DFL_IN_BOUNDS(err.word, at + 3, (int64_t)2 * ranges * Cfg::ROWS * HD)) {
                        *reinterpret_cast<float4*>(a.Opart + at) = o;
                        if (c == 0) a.ml[part * Cfg::ROWS + row] = make_float2(M, L);
                    }
                }
            }
        }
        if (u0 == 0 && u1 < pos.nu && tid == 0) a.cross[range] = KaCross{pos.n, head, pos.tile, (x + pos.nu - 1) / line.per};
        group_sync(group);
        x += u1 - u0;
        pos.u = u1;
        if (u1 == pos.nu) pos.next_triple(a);
    }
    // After a wait that ran out: let the copies in flight land before the CTA's shared memory goes.
    #pragma unroll 1
    for (; taken < feed.issued; ++taken) mbar_wait(&full[taken % KA_SLOTS], (taken / KA_SLOTS) & 1, err);
}

constexpr int KA_SMS = 152;   // SMs of a GB300

// Row tiles of 8 query rows when a group has at most 8, of 16 up to 16: a wider
// tile expands each key for more rows at once.  More rows go to the
// tensor-memory kernel: 32 sequences of 2,048 tokens with 16 rows to a head take
// 35.5 us here and 52 there, with 32 rows, as two tiles of 16, 64 and 52; there
// 17 to 64 rows cost the same (17 53, 24 51, 64 52 us).
// See KaLine.  The seam, 0, 8 and 16 (one token, 32/8 heads of 128): 64 sequences
// of 300 18.5, 16.4 and 16.4 us, 70 of 2,000 47.1, 45.1 and 45.1, 4 of 300 10.3,
// 10.4 and 12.3.  The weight: a triple costs some 4.5 us beside 1.1 us per unit
// (the batch above 107, 102 and 103 us with weights 2, 4 and 6).
constexpr int KA_SEAM = 8;
constexpr int KA_WEIGHT = 4;
constexpr int KJ_ROWS = KjCfg<128, 8>::AT_ONCE;
constexpr int KA_MAX_ROWS = 16;
int ka_nt(int R) { return R <= 8 ? 1 : 2; }

int ka_groups(int hd, int nt) { return hd == 128 && nt == 2 ? KaCfg<128, 2>::GROUPS : KaCfg<128, 1>::GROUPS; }

// CTAs of the launch: one per SM, fewer when there are fewer units.
int ka_grid(int64_t units) { return (int)std::min<int64_t>(units, KA_SMS); }

// Rows of a triple, row tiles of a K/V head, keys of a unit, places of a triple.
int ka_rows(int R) { return R > KA_MAX_ROWS ? kv4_attn_tc_rows(R) : 8 * ka_nt(R); }
int ka_subs(int R) { return (R + ka_rows(R) - 1) / ka_rows(R); }
int ka_unit_log2(int R, int hd) { return R > KA_MAX_ROWS ? kv4_attn_tc_unit_log2(R, hd) : 6; }   // KA_UNIT
int ka_weight(int R) { return R > KA_MAX_ROWS ? kv4_attn_tc_weight() : KA_WEIGHT; }
int64_t ka_most_units(const dfl_kv4_pool& pool, const dfl_pages& pg, int R) {
    return ((int64_t)pg.max_pages * pool.page >> ka_unit_log2(R, pool.hd)) + 2 + ka_weight(R);
}

inline size_t al256(size_t b) { return (b + 255) & ~size_t(255); }

}  // namespace

dfl_status kv4_attn_check(const dfl_kv4_pool& pool, const dfl_pages& pg, int B, int Hq) {
    const int G = Hq / pool.Hkv;
    if (B > 64 || (int64_t)B * G > KV4_MAX_HEAD_ROWS || !rows_fit((int64_t)pg.N * B)) return DFL_ERR_UNSUPPORTED_SHAPE;
    if ((int64_t)pg.max_pages * pool.page > KV4_ATTN_TOKENS) return DFL_ERR_UNSUPPORTED_SHAPE;
    const int R = B * G;
    const int64_t triples = (int64_t)pool.Hkv * ka_subs(R) * pg.N;
    if (triples >= (int64_t)1 << 31 || triples * ka_most_units(pool, pg, R) >= (int64_t)1 << 31) return DFL_ERR_UNSUPPORTED_SHAPE;
    return DFL_OK;
}

size_t kv4_attn_ws_bytes(int N, int B, int Hq, int Hkv, int hd) {
    if (N <= 0 || B <= 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0) return 0;
    if ((int64_t)B * (Hq / Hkv) > KV4_MAX_HEAD_ROWS) return 0;
    const int R = B * (Hq / Hkv), nt = ka_nt(R);
    if (R > KA_MAX_ROWS) return kv4_attn_tc_ws_bytes(R, hd);
    const size_t parts = 2 * (size_t)KA_SMS * ka_groups(hd, nt) * 8 * nt;
    return al256(parts * hd * 4) + al256(parts * 8) + al256(sizeof(KaCross) * KA_SMS * ka_groups(hd, nt));
}

dfl_status kv4_attn_run(DeviceCtx* ctx, const dfl_kv4_pool& pool, int layer, const dfl_pages& pg, const void* Q,
                        const void* Kb, const void* Vb, int B, int Hq, void* O, void* ws, cudaStream_t st) {
    const int G = Hq / pool.Hkv, R = B * G, nt = ka_nt(R);
    const bool tc = R > KA_MAX_ROWS;
    const int rows = ka_rows(R);
    KaArgs a{};
    a.slab = kv4_slab(pool, layer);
    a.table = pg.table; a.len = pg.len; a.max_pages = pg.max_pages;
    a.N = pg.N; a.B = B; a.Hq = Hq; a.G = G; a.R = R;
    a.subs = ka_subs(R);
    a.HS = pool.Hkv * a.subs;
    a.g_inv = (((uint64_t)1 << 40) + G - 1) / G;
    a.cells_inv = (((uint64_t)1 << 36) + a.slab.cells - 1) / a.slab.cells;
    a.Q = static_cast<const __nv_bfloat16*>(Q);
    a.Kb = static_cast<const __nv_bfloat16*>(Kb);
    a.Vb = static_cast<const __nv_bfloat16*>(Vb);
    a.O = static_cast<__nv_bfloat16*>(O);
    a.scale_log2 = 1.4426950408889634f / sqrtf((float)pool.hd);
    a.k_pow2 = kv4_exp2i(pool.k_exp); a.k_inv = kv4_exp2i(-pool.k_exp);
    a.v_pow2 = kv4_exp2i(pool.v_exp); a.v_inv = kv4_exp2i(-pool.v_exp);
    a.unit_log2 = ka_unit_log2(R, pool.hd);
    a.weight = ka_weight(R);
    a.seam = tc ? kv4_attn_tc_seam() : KA_SEAM;
    static_assert(KA_UNIT == 64, "unit_log2");
    const int64_t units = ka_most_units(pool, pg, R) * pg.N * a.HS;   // < 2^31: kv4_attn_check
    if (tc) return kv4_attn_tc_run(ctx, a, pool.hd, units, ws, st);
    const size_t parts = 2 * (size_t)KA_SMS * ka_groups(pool.hd, nt) * rows;
    a.Opart = static_cast<float*>(ws);
    a.ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(ws) + al256(parts * pool.hd * 4));
    a.cross = reinterpret_cast<KaCross*>(reinterpret_cast<uint8_t*>(a.ml) + al256(parts * 8));
    const int grid = ka_grid(units), groups = ka_groups(pool.hd, nt);
    const DevErr err = dev_err(ctx);
    auto run = [&](auto kern, auto join, int smem, int slot) -> dfl_status {
        if (!ctx->kv4_attr_set[slot]) {
            if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
                return DFL_ERR_CUDA;
            ctx->kv4_attr_set[slot] = true;
        }
        {
            ProfScope ps("kv4_attn", st);
            const dfl_status rc = launch_pdl(kern, grid, groups * KA_THREADS, smem, st, a, err);
            if (rc != DFL_OK) return rc;
        }
        ProfScope ps("kv4_attn_join", st);
        return launch_pdl(join, dim3(grid * groups, rows / KJ_ROWS), pool.hd / 4 * KJ_ROWS, 0, st, a, err);
    };
    if (pool.hd == 128)
        return nt == 1 ? run(kv4_attn_kernel<128, 1>, kv4_attn_join_kernel<128, 8>, KaCfg<128, 1>::SMEM, 0)
                       : run(kv4_attn_kernel<128, 2>, kv4_attn_join_kernel<128, 16>, KaCfg<128, 2>::SMEM, 1);
    return nt == 1 ? run(kv4_attn_kernel<64, 1>, kv4_attn_join_kernel<64, 8>, KaCfg<64, 1>::SMEM, 2)
                   : run(kv4_attn_kernel<64, 2>, kv4_attn_join_kernel<64, 16>, KaCfg<64, 2>::SMEM, 3);
}

}  // namespace dfl
