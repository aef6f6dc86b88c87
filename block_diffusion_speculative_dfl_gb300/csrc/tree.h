// Host launchers of the drafted-token trees and of the log probabilities they are built from.
#pragma once

#include "internal.h"

namespace dfl {

constexpr int TREE_MAX_ROWS = 64;    // rows of a tree: the bits of its masks
constexpr int LP_MAX_TOP = 64;       // alternatives of a row

struct LpArgs {
    const void* logits;      // [rows] rows of V elements, `stride` elements apart
    int64_t rows, stride;
    int V, M, K;
    float c;                 // log2(e) / T
    const int32_t* ids;      // [rows][M]
    float* logp;             // [rows][M]
    float* entropy;          // [rows] (nullable)
    int32_t* top_ids;        // [rows][K]
    float* top_logp;         // [rows][K]
};

dfl_status token_logprobs_run(DeviceCtx* ctx, const LpArgs& a, int dt, cudaStream_t st);

dfl_status draft_tree_run(const int32_t* anchor, const int32_t* top_ids, const float* top_logp, int N, int G, int K, int B,
                          int32_t* token, int32_t* parent, int32_t* depth, uint64_t* mask, int32_t* count, const DevErr& err,
                          cudaStream_t st);
dfl_status tree_accept_run(const int32_t* token, const int32_t* parent, const int32_t* target, int N, int B, int32_t* path,
                           int32_t* accept_len, int32_t* n_rows, int32_t* bonus, const DevErr& err, cudaStream_t st);

}  // namespace dfl
