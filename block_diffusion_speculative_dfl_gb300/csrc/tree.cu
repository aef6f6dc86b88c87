// Trees of drafted tokens: building one from the alternatives of every drafted
// position, and accepting along it.
//
// A block-diffusion drafter gives one marginal per position, so the probability
// of a path is the product of its tokens' and the B - 1 most probable prefixes
// are closed under parents: they are a tree.  It is grown best first: a row's
// next child is the best alternative of its position that is not a row yet, with
// the score (the row's score + logp); the best of all rows' next children is the
// next row.  Ties go to the lowest parent.  Scores are fp64 sums of the fp32 log
// probabilities: exact for the ranges that occur, so the order does not depend on
// how the sum is taken.
//
// Both are chains of short steps (a tree of 64 rows is 63 of them) over some KB:
// latency bounds them.  One warp per sequence holds two rows per lane, finds the
// best candidate by a warp-wide maximum and keeps the log probabilities in
// shared memory.
#include "internal.h"
#include "tree.h"

namespace dfl {

namespace {

// Order-preserving 64-bit integer of a double that is no NaN.
__device__ __forceinline__ uint64_t ordered(double x) {
    const uint64_t b = (uint64_t)__double_as_longlong(x);
    return b >> 63 ? ~b : b | 1ull << 63;
}

constexpr uint64_t NO_CHILD = 0;   // below every score

// G positions, K alternatives of each (row pitch K0 in memory); B rows.
__global__ void __launch_bounds__(32) draft_tree_kernel(const int32_t* anchor, const int32_t* top_ids, const float* top_logp, int N,
                                                        int G0, int K0, int G, int K, int B, int32_t* token, int32_t* parent,
                                                        int32_t* depth, uint64_t* mask, int32_t* count, const DevErr err) {
    extern __shared__ float lp[];   // [G][K]
    grid_dep_begin();
    const int n = blockIdx.x, lane = threadIdx.x;
    const int64_t base = (int64_t)n * G0 * K0;
    for (int i = lane; i < G * K; i += 32) lp[i] = top_logp[base + (int64_t)(i / K) * K0 + i % K];
    __syncwarp();
    // this lane's rows: lane and lane + 32
    double score[2] = {0.0, 0.0};
    int level[2] = {0, 0}, rank[2] = {0, 0}, from[2] = {lane == 0 ? -1 : -2, -2}, alt[2] = {0, 0};
    uint64_t seen[2] = {lane == 0 ? 1ull : 0ull, 0ull}, cand[2] = {NO_CHILD, NO_CHILD};
    // the next child of this lane's row s
    auto child = [&](int s) {
        cand[s] = NO_CHILD;
        if (level[s] >= G || rank[s] >= K) return;
        const float x = lp[level[s] * K + rank[s]];
        if (x > -INFINITY) cand[s] = ordered(score[s] + (double)x);   // a NaN is no candidate
    };
    if (lane == 0) child(0);
    int rows = 1;
    #pragma unroll 1
    for (; rows < B; ++rows) {
        const uint64_t mine = max(cand[0], cand[1]);
        const uint32_t hi = (uint32_t)(mine >> 32), best_hi = __reduce_max_sync(0xFFFFFFFFu, hi);
        const uint32_t best_lo = __reduce_max_sync(0xFFFFFFFFu, hi == best_hi ? (uint32_t)mine : 0u);
        const uint64_t best = (uint64_t)best_hi << 32 | best_lo;
        if (best == NO_CHILD) break;
        const uint32_t low = __ballot_sync(0xFFFFFFFFu, cand[0] == best), high = __ballot_sync(0xFFFFFFFFu, cand[1] == best);
        const int p = low ? __ffs(low) - 1 : 32 + __ffs(high) - 1;
        const uint64_t best_bits = best >> 63 ? best ^ 1ull << 63 : ~best;
        const int l = __shfl_sync(0xFFFFFFFFu, low ? level[0] : level[1], p & 31);
        const int k = __shfl_sync(0xFFFFFFFFu, low ? rank[0] : rank[1], p & 31);
        const uint64_t up = __shfl_sync(0xFFFFFFFFu, low ? seen[0] : seen[1], p & 31);
        #pragma unroll
        for (int s = 0; s < 2; ++s) {
            if (lane + 32 * s == p) {
                ++rank[s];
                child(s);
            }
            if (lane + 32 * s == rows) {
                score[s] = __longlong_as_double((long long)best_bits);
                level[s] = l + 1;
                from[s] = p;
                alt[s] = l * K0 + k;
                seen[s] = up | 1ull << rows;
                child(s);
            }
        }
    }
    if (lane == 0 && DFL_IN_BOUNDS(err.word, n, N)) count[n] = rows;
    #pragma unroll
    for (int s = 0; s < 2; ++s) {
        const int row = lane + 32 * s;
        if (row >= B || !DFL_IN_BOUNDS(err.word, (int64_t)n * B + row, (int64_t)N * B)) continue;
        const int64_t at = (int64_t)n * B + row;
        token[at] = row >= rows ? -1 : row == 0 ? anchor[n] : top_ids[base + alt[s]];
        parent[at] = from[s];
        depth[at] = level[s];
        mask[at] = seen[s];
    }
}

constexpr int TA_WARPS = 4;

// From the anchor along children whose token is the target's behind the current row.
__global__ void __launch_bounds__(TA_WARPS * 32) tree_accept_kernel(const int32_t* token, const int32_t* parent, const int32_t* target,
                                                                     int N, int B, int32_t* path, int32_t* accept_len, int32_t* n_rows,
                                                                     int32_t* bonus, const DevErr err) {
    grid_dep_begin();
    const int n = blockIdx.x * TA_WARPS + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (n >= N) return;
    int tok[2], par[2], tgt[2], out[2] = {lane == 0 ? 0 : -1, -1};
    #pragma unroll
    for (int s = 0; s < 2; ++s) {
        const int row = lane + 32 * s;
        const int64_t at = (int64_t)n * B + row;
        const bool there = row < B;
        tok[s] = there ? token[at] : -1;
        par[s] = there ? parent[at] : -2;
        tgt[s] = there ? target[at] : -1;
    }
    int cur = 0, done = 1, want;
    #pragma unroll 1
    while (true) {
        const int w0 = __shfl_sync(0xFFFFFFFFu, tgt[0], cur & 31), w1 = __shfl_sync(0xFFFFFFFFu, tgt[1], cur & 31);
        want = cur < 32 ? w0 : w1;
        const uint32_t low = __ballot_sync(0xFFFFFFFFu, par[0] == cur && tok[0] == want && lane > cur);
        const uint32_t high = __ballot_sync(0xFFFFFFFFu, par[1] == cur && tok[1] == want && lane + 32 > cur);
        if (!(low | high)) break;
        cur = low ? __ffs(low) - 1 : 32 + __ffs(high) - 1;   // above the row before: at most B - 1 turns
        if (lane == (done & 31)) out[done >> 5] = cur;
        ++done;
    }
    if (lane == 0 && DFL_IN_BOUNDS(err.word, n, N)) {
        accept_len[n] = done - 1;
        if (n_rows) n_rows[n] = done;
        bonus[n] = want;
    }
    #pragma unroll
    for (int s = 0; s < 2; ++s) {
        const int row = lane + 32 * s;
        if (row < B && DFL_IN_BOUNDS(err.word, (int64_t)n * B + row, (int64_t)N * B)) path[(int64_t)n * B + row] = out[s];
    }
}

}  // namespace

dfl_status draft_tree_run(const int32_t* anchor, const int32_t* top_ids, const float* top_logp, int N, int G, int K, int B,
                          int32_t* token, int32_t* parent, int32_t* depth, uint64_t* mask, int32_t* count, const DevErr& err,
                          cudaStream_t st) {
    ProfScope ps("draft_tree", st);
    // a tree of B rows is at most B - 1 deep, and its rows have at most B - 1 children
    const int g = G < B - 1 ? G : B - 1, k = K < B - 1 ? K : B - 1;
    return launch_pdl(draft_tree_kernel, N, 32, (size_t)g * k * 4, st, anchor, top_ids, top_logp, N, G, K, g, k, B, token, parent,
                      depth, mask, count, err);
}

dfl_status tree_accept_run(const int32_t* token, const int32_t* parent, const int32_t* target, int N, int B, int32_t* path,
                           int32_t* accept_len, int32_t* n_rows, int32_t* bonus, const DevErr& err, cudaStream_t st) {
    ProfScope ps("tree_accept", st);
    return launch_pdl(tree_accept_kernel, (N + TA_WARPS - 1) / TA_WARPS, TA_WARPS * 32, 0, st, token, parent, target, N, B, path,
                      accept_len, n_rows, bonus, err);
}

}  // namespace dfl
