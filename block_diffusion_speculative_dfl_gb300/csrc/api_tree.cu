// C-ABI entry points of the drafted-token trees: argument checks.
#include <cmath>

#include "internal.h"
#include "paged.h"
#include "tree.h"

using namespace dfl;

extern "C" dfl_status dfl_token_logprobs(const void* logits, int32_t dt, int64_t rows, int32_t V, int64_t row_stride, float T,
                                         const int32_t* ids, int32_t M, float* logp, float* entropy, int32_t K, int32_t* top_ids,
                                         float* top_logp, dfl_stream stream) {
    const dfl::ApiRange nvtx_range("dfl_token_logprobs");
    if (!logits || (dt != DFL_F32 && dt != DFL_BF16) || rows < 1 || V < 1 || row_stride < V || M < 0 || K < 0 || K > LP_MAX_TOP)
        return DFL_ERR_INVALID_ARG;
    if (!(T >= 1e-6f && T <= 1e6f)) return DFL_ERR_INVALID_ARG;
    if ((M > 0 && (!ids || !logp)) || (K > 0 && (!top_ids || !top_logp)) || (M == 0 && K == 0 && !entropy)) return DFL_ERR_INVALID_ARG;
    if (!rows_fit(rows) || V > 1 << 30 || row_stride > (int64_t)1 << 40) return DFL_ERR_UNSUPPORTED_SHAPE;
    if (!aligned16(logits) || !aligned4(ids) || !aligned4(logp) || !aligned4(entropy) || !aligned4(top_ids) || !aligned4(top_logp))
        return DFL_ERR_MISALIGNED;
    DeviceCtx* ctx = current_ctx();
    if (!ctx) return DFL_ERR_NO_DEVICE;
    const LpArgs a{logits, rows, row_stride, V, M, K, (float)(1.4426950408889634 / (double)T), ids, logp, entropy, top_ids, top_logp};
    return token_logprobs_run(ctx, a, dt, static_cast<cudaStream_t>(stream));
}

extern "C" dfl_status dfl_draft_tree(const int32_t* anchor, const int32_t* top_ids, const float* top_logp, int32_t N, int32_t G,
                                     int32_t K, int32_t B, int32_t* token, int32_t* parent, int32_t* depth, uint64_t* mask,
                                     int32_t* count, dfl_stream stream) {
    const dfl::ApiRange nvtx_range("dfl_draft_tree");
    if (!anchor || !top_ids || !top_logp || !token || !parent || !depth || !mask || !count || N < 1 || G < 1 || K < 1 || B < 1)
        return DFL_ERR_INVALID_ARG;
    if (B > TREE_MAX_ROWS || (int64_t)G * K >= (int64_t)1 << 31) return DFL_ERR_UNSUPPORTED_SHAPE;
    const int32_t* words[] = {anchor, top_ids, token, parent, depth, count};
    for (const int32_t* p : words) if (!aligned4(p)) return DFL_ERR_MISALIGNED;
    if (!aligned4(top_logp) || (reinterpret_cast<uintptr_t>(mask) & 7u)) return DFL_ERR_MISALIGNED;
    DeviceCtx* ctx = current_ctx();
    if (!ctx) return DFL_ERR_NO_DEVICE;
    return draft_tree_run(anchor, top_ids, top_logp, N, G, K, B, token, parent, depth, mask, count, dev_err(ctx),
                          static_cast<cudaStream_t>(stream));
}

extern "C" dfl_status dfl_tree_accept(const int32_t* token, const int32_t* parent, const int32_t* target, int32_t N, int32_t B,
                                      int32_t* path, int32_t* accept_len, int32_t* n_rows, int32_t* bonus, dfl_stream stream) {
    const dfl::ApiRange nvtx_range("dfl_tree_accept");
    if (!token || !parent || !target || !path || !accept_len || !bonus || N < 1 || B < 1) return DFL_ERR_INVALID_ARG;
    if (B > TREE_MAX_ROWS) return DFL_ERR_UNSUPPORTED_SHAPE;
    const int32_t* words[] = {token, parent, target, path, accept_len, n_rows, bonus};
    for (const int32_t* p : words) if (!aligned4(p)) return DFL_ERR_MISALIGNED;
    DeviceCtx* ctx = current_ctx();
    if (!ctx) return DFL_ERR_NO_DEVICE;
    return tree_accept_run(token, parent, target, N, B, path, accept_len, n_rows, bonus, dev_err(ctx),
                           static_cast<cudaStream_t>(stream));
}
