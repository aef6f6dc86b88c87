// Page operations of the paged context cache: reserve (with copies of shared
// pages on their first write), remap (fork, reorder, roll back, free) and
// compact.
//
// Bookkeeping is small (a few bytes per page and sequence) and every decision
// depends on counts over all of it, so one block of 1024 threads makes the
// plan of a reservation or a compaction: 32 pages per thread and pass, a block
// scan per pass.  Everything it decides is a function of ranks (the k-th free
// page goes to the k-th request), so results do not depend on timing.  The
// bytes (pages copied or moved in every layer, table entries) are the second
// kernel's, spread over all SMs in 16-KB pieces; it finds its list on the
// device, so neither call reads anything back to the host.
//
// Measured (replayed): 256 forked sequences that copy their last page in 7 layers
// (256 MB read and written) 37 us, 8 of them the plan; moving the scattered half
// of a pool of 7 layers (525 MB) 95 us, 9 of them the plan, the moves at 90 % of
// a plain copy's rate; reordering 512 rows of 1,024 pages 11-12 us.  Copies go
// through registers: rings of bulk copies through shared memory moved the pool in
// 98 to 101 us.
#include "internal.h"
#include "paged.h"

namespace dfl {

namespace {

constexpr int PG_PLAN = 1024;        // threads of a planning block
constexpr int PG_PASS = PG_PLAN * 32;  // pages per pass
constexpr int PG_FEW = 4096;         // free pages that are handed out from shared memory
// At most this many bytes to copy (every sequence's last page in every layer) are
// copied by the planning block, PG_WORDS 16-byte words a thread, all read before
// the first is written; more go to a kernel of its own.  Here and there, us
// replayed, and issued one after another (which the host bounds):
//   nothing shared, any size          2.9  6.5 |  3.8  8.6
//   all copied, 16 pages of 1,152 B   5.5  6.3 |  6.2  8.8
//               28 pages of 2,304 B   6.4  7.0 |  5.6  8.2
//               56 pages of 2,304 B   9.1  9.3 |  6.3  8.6
//              224 pages of 1,152 B  16.3 15.8 |  9.5  9.5
// Copied page by page here, the last two took 19.8 and 62.9: a round trip each.
constexpr int PG_WORDS = 4;
constexpr int64_t PG_HERE = PG_PLAN * PG_WORDS * 16;
constexpr int PG_PIECE = 16384;      // bytes a block copies at a time
constexpr int PG_THREADS = 256;

inline size_t al256(size_t b) { return (b + 255) & ~size_t(255); }

struct PgArgs {
    int32_t* table;
    int32_t* len;
    int32_t* ref;
    int N, max_pages, num_pages, page;
};

PgArgs pg_args(const dfl_kv4_pool& pool, const dfl_pages& pg) {
    return PgArgs{pg.table, pg.len, pg.ref, pg.N, pg.max_pages, pool.num_pages, pool.page};
}

// Where the second kernel finds the pages to copy.  (The bounds-checked build
// checks what goes through these lists and through the free list: the page
// numbers, and the entries' own places.)
struct PgMoves {
    int32_t* count;   // [1]
    int32_t* src;     // [<= capacity]
    int32_t* dst;
};

// Pages base + 32 * thread .. + 31 as a mask of the used ones.  A warp reads
// its 1024 counts in 32 coalesced loads; lane i keeps the i-th ballot.  Pages
// past the pool read as unused.  Whole warps.
__device__ __forceinline__ uint32_t used_mask(const int32_t* ref, int num_pages, int base) {
    const int lane = threadIdx.x & 31, first = base + (int)(threadIdx.x & ~31u) * 32;
    uint32_t mine = 0;
    if (first < num_pages) {
        #pragma unroll
        for (int i = 0; i < 32; ++i) {
            const int p = first + 32 * i + lane;
            const uint32_t b = __ballot_sync(0xFFFFFFFFu, p < num_pages && ref[p] > 0);
            if (lane == i) mine = b;
        }
    }
    return mine;
}

// The low n bits (0 <= n <= 32).
__device__ __forceinline__ uint32_t low_bits(int n) { return n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1; }
__device__ __forceinline__ int valid_count(int num_pages, int first) { return min(max(num_pages - first, 0), 32); }

// ---------------------------------------------------------------- reserve --

struct ReservePlan {
    int32_t* off;     // [N] pages asked for by the sequences before n
    int32_t* need;    // [N] pages sequence n asks for; -1: arguments out of range
    int32_t* tail;    // [N] its shared last page, or -1
    int32_t* free_;   // [num_pages] free pages in order, as many as asked for
    PgMoves cow;
};

// Pages of every layer that a block copies by itself (`data` null: another launch does).
struct PgHere {
    uint8_t* data;
    int64_t layer_stride, page_bytes;
    int layers;
};

__global__ void __launch_bounds__(PG_PLAN) pages_reserve_plan_kernel(const PgArgs a, const int32_t* n_new, int max_new,
                                                                    int32_t* start, const ReservePlan p,
                                                                    const PgHere here, const DevErr err) {
    __shared__ int red[PG_PLAN / 32];
    __shared__ int cows;
    __shared__ int32_t few[PG_FEW];
    grid_dep_begin();
    if (threadIdx.x == 0) cows = 0;
    const bool one = a.N <= PG_PLAN;   // a sequence per thread: what it asks for stays in registers
    // the first counts are read while the requests are looked up
    const uint32_t used0 = used_mask(a.ref, a.num_pages, 0);
    // what each sequence asks for, on the counts as they were before the call
    int asked = 0, need = 0, off = 0, tail = -1, l = 0, m = 0;
    for (int base = 0; base < a.N; base += PG_PLAN) {
        const int n = base + threadIdx.x;
        need = 0;
        tail = -1;
        if (n < a.N) {
            l = a.len[n];
            m = n_new[n];
            if (l < 0 || m < 0 || m > max_new || l > a.max_pages * a.page - m) {
                record_error(err, DFL_ERR_INVALID_ARG);
                need = -1;
            } else {
                const int have = (l + a.page - 1) / a.page;
                need = (l + m + a.page - 1) / a.page - have;
                if (m > 0 && l % a.page != 0) {
                    const int t = a.table[(int64_t)n * a.max_pages + have - 1];
                    if (t < 0 || t >= a.num_pages) {   // new tokens would share a page that is none
                        record_error(err, DFL_ERR_INVALID_ARG);
                        need = -1;
                    } else if (a.ref[t] > 1) { tail = t; ++need; }
                }
            }
        }
        int sum;
        off = asked + block_exscan<PG_PLAN>(max(need, 0), red, &sum);
        asked += sum;
        if (!one && n < a.N) { p.off[n] = off; p.need[n] = need; p.tail[n] = tail; }
    }
    // the first `asked` free pages
    int32_t* free_ = asked <= PG_FEW ? few : p.free_;
    int found = 0;
    for (int base = 0; base < a.num_pages && found < asked; base += PG_PASS) {
        const int first = base + (int)threadIdx.x * 32;
        const uint32_t u = base == 0 ? used0 : used_mask(a.ref, a.num_pages, base);
        uint32_t f = ~u & low_bits(valid_count(a.num_pages, first));
        int sum;
        int k = found + block_exscan<PG_PLAN>(__popc(f), red, &sum);
        for (; f && k < asked; f &= f - 1, ++k)
            if (DFL_IN_BOUNDS(err.word, k, asked <= PG_FEW ? PG_FEW : a.num_pages)) free_[k] = first + __ffs(f) - 1;
        found += sum;
    }
    __syncthreads();   // the lists are read by other threads (and the counts are written) from here on
    const int lane = threadIdx.x & 31;
    for (int base = 0; base < a.N; base += PG_PLAN) {
        const int n = base + threadIdx.x;
        if (!one && n < a.N) {
            off = p.off[n]; need = p.need[n]; tail = p.tail[n];
            l = a.len[n];
            m = need < 0 ? 0 : n_new[n];
        }
        const bool served = n < a.N && (need == 0 || (need > 0 && off + need <= found));
        if (served && tail >= 0) {
            const int c = atomicAdd(&cows, 1);   // the order of copies does not matter
            if (DFL_IN_BOUNDS(err.word, c, a.N)) {
                p.cow.src[c] = tail;
                p.cow.dst[c] = free_[off];
            }
            atomicSub(&a.ref[tail], 1);
        }
        if (n < a.N) {
            start[n] = served ? l : -1;
            if (served) a.len[n] = l + m;
        }
        // the pages of a warp's sequences, one sequence after another, a page per lane
        const int first = (l + a.page - 1) / a.page - (tail >= 0 ? 1 : 0);
        for (uint32_t who = __ballot_sync(0xFFFFFFFFu, served && need > 0); who; who &= who - 1) {
            const int j = __ffs(who) - 1;
            const int nj = __shfl_sync(0xFFFFFFFFu, need, j), oj = __shfl_sync(0xFFFFFFFFu, off, j);
            const int fj = __shfl_sync(0xFFFFFFFFu, first, j);
            int32_t* row = a.table + (int64_t)(n - lane + j) * a.max_pages + fj;
            for (int k = lane; k < nj; k += 32) {
                const int f = free_[oj + k];
                if (!DFL_IN_BOUNDS(err.word, fj + k, a.max_pages) || !DFL_IN_BOUNDS(err.word, f, a.num_pages)) continue;
                row[k] = f;
                a.ref[f] = 1;
            }
        }
    }
    __syncthreads();
    if (!here.data) {
        if (threadIdx.x == 0) *p.cow.count = cows;
        return;
    }
    // one index over (copied page, layer, 16 bytes)
    const uint32_t n16 = (uint32_t)(here.page_bytes / 16), all = (uint32_t)cows * here.layers * n16;   // <= PG_HERE / 16
    uint4 v[PG_WORDS];
    uint4* to[PG_WORDS];
    #pragma unroll
    for (int j = 0; j < PG_WORDS; ++j) {
        const uint32_t i = threadIdx.x + j * PG_PLAN;
        if (i >= all) continue;
        const uint32_t pl = i / n16, c = pl / here.layers;
        uint8_t* layer = here.data + (int64_t)(pl - c * here.layers) * here.layer_stride + (i - pl * n16) * 16;
        const int src = p.cow.src[c], dst = p.cow.dst[c];
        to[j] = nullptr;
        if (!DFL_IN_BOUNDS(err.word, src, a.num_pages) || !DFL_IN_BOUNDS(err.word, dst, a.num_pages)) continue;
        v[j] = *reinterpret_cast<const uint4*>(layer + src * here.page_bytes);
        to[j] = reinterpret_cast<uint4*>(layer + dst * here.page_bytes);
    }
    #pragma unroll
    for (int j = 0; j < PG_WORDS; ++j)
        if (threadIdx.x + j * PG_PLAN < all && to[j]) *to[j] = v[j];
}

// Copies whole pages src[k] -> dst[k] of every layer, in pieces.
__device__ __forceinline__ void copy_pages(const PgMoves& mv, uint8_t* data, int64_t layer_stride, int layers,
                                           int64_t page_bytes, int num_pages, const DevErr& err) {
    const int64_t pieces = (page_bytes + PG_PIECE - 1) / PG_PIECE;
    const int64_t items = (int64_t)*mv.count * layers * pieces;
    for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
        const int64_t pl = it / pieces;
        const int64_t at = (it - pl * pieces) * PG_PIECE;
        const int k = (int)(pl / layers), layer = (int)(pl - (int64_t)k * layers);
        const int src = mv.src[k], dst = mv.dst[k];
        if (!DFL_IN_BOUNDS(err.word, src, num_pages) || !DFL_IN_BOUNDS(err.word, dst, num_pages)) continue;
        const uint8_t* s = data + layer * layer_stride + src * page_bytes + at;
        uint8_t* d = data + layer * layer_stride + dst * page_bytes + at;
        const int n16 = (int)(min((int64_t)PG_PIECE, page_bytes - at) / 16);
        uint4 v[PG_PIECE / 16 / PG_THREADS];
        #pragma unroll
        for (int i = 0; i < PG_PIECE / 16 / PG_THREADS; ++i) {
            const int j = threadIdx.x + i * PG_THREADS;
            if (j < n16) v[i] = reinterpret_cast<const uint4*>(s)[j];
        }
        #pragma unroll
        for (int i = 0; i < PG_PIECE / 16 / PG_THREADS; ++i) {
            const int j = threadIdx.x + i * PG_THREADS;
            if (j < n16) reinterpret_cast<uint4*>(d)[j] = v[i];
        }
    }
}

__global__ void __launch_bounds__(PG_THREADS) pages_copy_kernel(const PgMoves mv, uint8_t* data, int64_t layer_stride,
                                                               int layers, int64_t page_bytes, int num_pages,
                                                               const DevErr err) {
    grid_dep_begin();
    copy_pages(mv, data, layer_stride, layers, page_bytes, num_pages, err);
}

// ------------------------------------------------------------------ remap --

// A row takes from its parent's row, which another row's owner overwrites: all
// old rows are read before the first new one is written.  A small table is held
// by one block, with its barrier between; a larger one is saved to the workspace
// by a launch of its own and rewritten by a block per sequence.  One launch
// costs the host 1.4 us less; past some thousand entries one block is the slower
// on the GPU (16 x 125 entries 6.3 us either way, 64 x 375 8.3 us with two).
constexpr int PG_HELD = 4096;        // entries and sequences that one block takes

// What sequence n becomes: its parent's row (its own where the arguments are
// out of range), pages kept, length.
struct RemapRow {
    int parent, keep, len;
};
__device__ __forceinline__ RemapRow remap_row(const PgArgs& a, int n, const int32_t* len0, const int32_t* parent,
                                              const int32_t* keep_len, bool report, const DevErr& err) {
    int p = parent[n];
    bool ok = p < a.N;
    int l = 0;
    if (!ok) p = n;   // out of range: the row stays as it was
    if (p >= 0) {
        l = len0[p];
        if (ok && keep_len && keep_len[n] >= 0) l = min(l, keep_len[n]);
        if (l < 0 || l > a.max_pages * a.page) {   // a length that no table row can hold: the row stays
            ok = false;
            p = n;
            l = len0[n];
        }
    }
    if (!ok && report) record_error(err, DFL_ERR_INVALID_ARG);
    return RemapRow{p, ok ? (l + a.page - 1) / a.page : a.max_pages, l};
}

__device__ __forceinline__ void remap_entry(const PgArgs& a, int64_t at, int was, int now, const DevErr& err) {
    if (was == now || !DFL_IN_BOUNDS(err.word, at, (int64_t)a.N * a.max_pages)) return;
    a.table[at] = now;
    if (was >= 0 && was < a.num_pages) atomicSub(&a.ref[was], 1);
    if (now >= 0 && now < a.num_pages) atomicAdd(&a.ref[now], 1);
}

// One block; a warp per row.
__global__ void __launch_bounds__(PG_PLAN) pages_remap_small_kernel(const PgArgs a, const int32_t* parent,
                                                                    const int32_t* keep_len, const DevErr err) {
    __shared__ int32_t held[PG_HELD], lens[PG_HELD];   // the new rows and lengths
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    grid_dep_begin();
    for (int n = warp; n < a.N; n += PG_PLAN / 32) {
        const RemapRow w = remap_row(a, n, a.len, parent, keep_len, lane == 0, err);
        for (int j = lane; j < a.max_pages; j += 32)
            if (DFL_IN_BOUNDS(err.word, n * a.max_pages + j, PG_HELD))
                held[n * a.max_pages + j] = j < w.keep ? a.table[w.parent * a.max_pages + j] : -1;
        if (lane == 0) lens[n] = w.len;
    }
    __syncthreads();
    for (int at = threadIdx.x; at < a.N * a.max_pages; at += PG_PLAN) remap_entry(a, at, a.table[at], held[at], err);
    for (int n = threadIdx.x; n < a.N; n += PG_PLAN) a.len[n] = lens[n];
}

__global__ void __launch_bounds__(PG_THREADS) pages_save_kernel(const PgArgs a, int32_t* table0, int32_t* len0) {
    grid_dep_begin();
    const int64_t total = (int64_t)a.N * a.max_pages, step = (int64_t)gridDim.x * PG_THREADS;
    const int64_t i0 = blockIdx.x * (int64_t)PG_THREADS + threadIdx.x;
    for (int64_t i = i0; i < total; i += step) table0[i] = a.table[i];
    for (int64_t i = i0; i < a.N; i += step) len0[i] = a.len[i];
}

__global__ void __launch_bounds__(PG_THREADS) pages_remap_kernel(const PgArgs a, const int32_t* table0, const int32_t* len0,
                                                                const int32_t* parent, const int32_t* keep_len,
                                                                const DevErr err) {
    grid_dep_begin();
    const int n = blockIdx.x;
    const RemapRow w = remap_row(a, n, len0, parent, keep_len, threadIdx.x == 0, err);
    for (int j = threadIdx.x; j < a.max_pages; j += PG_THREADS)
        remap_entry(a, (int64_t)n * a.max_pages + j, table0[(int64_t)n * a.max_pages + j],
                    j < w.keep ? table0[(int64_t)w.parent * a.max_pages + j] : -1, err);
    if (threadIdx.x == 0) a.len[n] = w.len;
}

// ---------------------------------------------------------------- compact --

__global__ void __launch_bounds__(PG_PLAN) pages_compact_plan_kernel(const PgArgs a, int32_t* map, int32_t* live,
                                                                    const PgMoves mv, const DevErr err) {
    __shared__ int red[PG_PLAN / 32];
    grid_dep_begin();
    const uint32_t used0 = used_mask(a.ref, a.num_pages, 0);
    int cnt = __popc(used0);
    for (int base = PG_PASS; base < a.num_pages; base += PG_PASS) cnt += __popc(used_mask(a.ref, a.num_pages, base));
    int m;
    block_exscan<PG_PLAN>(cnt, red, &m);   // m: live pages, the new size of the pool's used part
    // holes below m take the live pages from m on, both in order
    const int lane = threadIdx.x & 31;
    int holes = 0, movers = 0;
    for (int base = 0; base < a.num_pages; base += PG_PASS) {
        const int first = base + (int)threadIdx.x * 32;
        const uint32_t u = base == 0 ? used0 : used_mask(a.ref, a.num_pages, base);
        const uint32_t low = low_bits(valid_count(m, first));   // the pages below m (m <= num_pages)
        const uint32_t h = ~u & low, v = u & ~low;
        int sh, sv;
        int kh = holes + block_exscan<PG_PLAN>(__popc(h), red, &sh);
        int kv = movers + block_exscan<PG_PLAN>(__popc(v), red, &sv);
        for (uint32_t f = h; f; f &= f - 1, ++kh)
            if (DFL_IN_BOUNDS(err.word, kh, a.num_pages)) mv.dst[kh] = first + __ffs(f) - 1;
        for (uint32_t f = v; f; f &= f - 1, ++kv)
            if (DFL_IN_BOUNDS(err.word, kv, a.num_pages)) mv.src[kv] = first + __ffs(f) - 1;
        const int first0 = first - 32 * lane;   // of the warp's 1024 pages
        for (int i = 0; i < 32 && first0 + 32 * i < a.num_pages; ++i) {
            const int pg = first0 + 32 * i + lane;
            const bool used = __shfl_sync(0xFFFFFFFFu, u, i) >> lane & 1;
            if (pg < a.num_pages) map[pg] = used ? pg : -1;   // pages that move: below
        }
        holes += sh;
        movers += sv;
    }
    __syncthreads();
    #pragma unroll 4
    for (int k = threadIdx.x; k < movers; k += PG_PLAN) {
        const int s = mv.src[k], d = mv.dst[k];
        if (!DFL_IN_BOUNDS(err.word, s, a.num_pages) || !DFL_IN_BOUNDS(err.word, d, a.num_pages)) continue;
        map[s] = d;
        a.ref[d] = a.ref[s];
        a.ref[s] = 0;
    }
    if (threadIdx.x == 0) { *mv.count = movers; *live = m; }
}

__global__ void __launch_bounds__(PG_THREADS) pages_compact_move_kernel(const PgArgs a, const int32_t* map, const PgMoves mv,
                                                                       uint8_t* data, int64_t layer_stride, int layers,
                                                                       int64_t page_bytes, const DevErr err) {
    grid_dep_begin();
    const int64_t total = (int64_t)a.N * a.max_pages;
    for (int64_t i = blockIdx.x * (int64_t)PG_THREADS + threadIdx.x; i < total; i += (int64_t)gridDim.x * PG_THREADS) {
        const int p = a.table[i];
        if (p < 0) continue;
        if (p >= a.num_pages) { record_error(err, DFL_ERR_INVALID_ARG); continue; }
        const int q = map[p];
        if (q != p) a.table[i] = q;
    }
    copy_pages(mv, data, layer_stride, layers, page_bytes, a.num_pages, err);
}

}  // namespace

size_t pages_reserve_ws(int64_t N, int64_t num_pages) { return al256(4) + 5 * al256(N * 4) + al256(num_pages * 4); }
size_t pages_remap_ws(int64_t N, int64_t max_pages) { return al256(N * max_pages * 4) + al256(N * 4); }
size_t pages_compact_ws(int64_t num_pages) { return al256(4) + 2 * al256(num_pages * 4); }

dfl_status pages_reserve_run(DeviceCtx* ctx, const dfl_kv4_pool& pool, const dfl_pages& pg, const int32_t* n_new,
                             int max_new, int32_t* start, void* ws, cudaStream_t st) {
    const PgArgs a = pg_args(pool, pg);
    uint8_t* w = static_cast<uint8_t*>(ws);
    auto take = [&](int64_t ints) {
        int32_t* r = reinterpret_cast<int32_t*>(w);
        w += al256(ints * 4);
        return r;
    };
    ReservePlan p;
    p.cow.count = take(1);
    p.cow.src = take(pg.N);
    p.cow.dst = take(pg.N);
    p.off = take(pg.N);
    p.need = take(pg.N);
    p.tail = take(pg.N);
    p.free_ = take(pool.num_pages);
    const int64_t bytes = kv4_page_bytes(pool.page, pool.Hkv, pool.hd);
    const bool here = bytes <= PG_HERE && bytes * pg.N <= PG_HERE / pool.layers;
    const PgHere h{here ? static_cast<uint8_t*>(pool.data) : nullptr, pool.layer_stride, bytes, pool.layers};
    {
        ProfScope ps("pages_reserve_plan", st);
        const dfl_status rc = launch_pdl(pages_reserve_plan_kernel, 1, PG_PLAN, 0, st, a, n_new, max_new, start, p, h, dev_err(ctx));
        if (rc != DFL_OK || here) return rc;
    }
    ProfScope ps("pages_copy", st);
    const int64_t most = (int64_t)pg.N * pool.layers * ((bytes + PG_PIECE - 1) / PG_PIECE);
    const unsigned grid = (unsigned)std::min<int64_t>(most, (int64_t)ctx->sm_count * 8);
    return launch_pdl(pages_copy_kernel, grid, PG_THREADS, 0, st, p.cow, static_cast<uint8_t*>(pool.data),
                      pool.layer_stride, pool.layers, bytes, pool.num_pages, dev_err(ctx));
}

dfl_status pages_remap_run(DeviceCtx* ctx, const dfl_kv4_pool& pool, const dfl_pages& pg, const int32_t* parent,
                           const int32_t* keep_len, void* ws, cudaStream_t st) {
    const PgArgs a = pg_args(pool, pg);
    if ((int64_t)pg.N * pg.max_pages <= PG_HELD) {
        ProfScope ps("pages_remap", st);
        return launch_pdl(pages_remap_small_kernel, 1, PG_PLAN, 0, st, a, parent, keep_len, dev_err(ctx));
    }
    int32_t* table0 = static_cast<int32_t*>(ws);
    int32_t* len0 = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(ws) + al256((size_t)pg.N * pg.max_pages * 4));
    dfl_status rc;
    {
        ProfScope ps("pages_save", st);
        const int64_t blocks = ((int64_t)pg.N * pg.max_pages + PG_THREADS - 1) / PG_THREADS;
        const unsigned grid = (unsigned)std::min<int64_t>(blocks, (int64_t)ctx->sm_count * 8);
        if ((rc = launch_pdl(pages_save_kernel, grid, PG_THREADS, 0, st, a, table0, len0)) != DFL_OK) return rc;
    }
    ProfScope ps("pages_remap", st);
    return launch_pdl(pages_remap_kernel, (unsigned)pg.N, PG_THREADS, 0, st, a, table0, len0, parent, keep_len,
                      dev_err(ctx));
}

dfl_status pages_compact_run(DeviceCtx* ctx, const dfl_kv4_pool& pool, const dfl_pages& pg, int32_t* map,
                             int32_t* live, void* ws, cudaStream_t st) {
    const PgArgs a = pg_args(pool, pg);
    uint8_t* w = static_cast<uint8_t*>(ws);
    PgMoves mv;
    mv.count = reinterpret_cast<int32_t*>(w);
    mv.src = reinterpret_cast<int32_t*>(w + al256(4));
    mv.dst = reinterpret_cast<int32_t*>(w + al256(4) + al256((size_t)pool.num_pages * 4));
    const int64_t bytes = kv4_page_bytes(pool.page, pool.Hkv, pool.hd);
    dfl_status rc;
    {
        ProfScope ps("pages_compact_plan", st);
        if ((rc = launch_pdl(pages_compact_plan_kernel, 1, PG_PLAN, 0, st, a, map, live, mv, dev_err(ctx))) != DFL_OK) return rc;
    }
    ProfScope ps("pages_compact_move", st);
    const int64_t most = std::max((int64_t)pool.num_pages * pool.layers * ((bytes + PG_PIECE - 1) / PG_PIECE),
                                  ((int64_t)pg.N * pg.max_pages + PG_THREADS - 1) / PG_THREADS);
    const unsigned grid = (unsigned)std::min<int64_t>(most, (int64_t)ctx->sm_count * 8);
    return launch_pdl(pages_compact_move_kernel, grid, PG_THREADS, 0, st, a, map, mv, static_cast<uint8_t*>(pool.data),
                      pool.layer_stride, pool.layers, bytes, dev_err(ctx));
}

}  // namespace dfl
