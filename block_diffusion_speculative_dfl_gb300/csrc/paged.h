// Host launchers of the paged 4-bit context cache.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/dfl.h"
#include "internal.h"
#include "kv4.cuh"

namespace dfl {

inline int64_t kv4_page_bytes(int page, int Hkv, int hd) { return (int64_t)page / 16 * Hkv * 18 * hd; }

inline Kv4Slab kv4_slab(const dfl_kv4_pool& p, int layer) {
    return Kv4Slab{static_cast<uint8_t*>(p.data) + layer * p.layer_stride, p.num_pages, p.page, p.Hkv, p.page / 16};
}

inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Page counts are summed over sequences in 32 bits.
inline bool pages_fit(const dfl_pages& pg) { return (int64_t)pg.N * pg.max_pages < (int64_t)1 << 31; }

// Host-side checks of a pool, a layer of it and (nullable) its page tables.
dfl_status kv4_check(const dfl_kv4_pool* pool, int layer, const dfl_pages* pg);

// Rows n*R + i (i < n_new[n]; with `rows` n*R + rows[n*R + i]) of K / V [N*R][Hkv][hd] to / from positions start[n] + i.
dfl_status kv4_append_run(DeviceCtx* ctx, const dfl_kv4_pool& pool, int layer, const dfl_pages& pg,
                          const int32_t* start, const int32_t* n_new, const int32_t* rows, int R, const void* K,
                          const void* V, cudaStream_t st);
dfl_status kv4_read_run(DeviceCtx* ctx, const dfl_kv4_pool& pool, int layer, const dfl_pages& pg, const int32_t* start,
                        const int32_t* count, int R, void* K, void* V, cudaStream_t st);

// Attention over the cache and the block's own keys (kv4_attn.cu).  mask (nullable), window (0: none), sinks: what
// its rows see.
constexpr int KV4_MAX_HEAD_ROWS = 65536;   // query rows of a K/V head: B * Hq / Hkv
// Tokens of a sequence that attention takes: its positions are 32-bit and are
// looked up as much as 32 units of 128 ahead.
constexpr int64_t KV4_ATTN_TOKENS = ((int64_t)1 << 31) - 8192;
// kv4_attn_check: the sizes that attention takes beyond kv4_check's.
dfl_status kv4_attn_check(const dfl_kv4_pool& pool, const dfl_pages& pg, int B, int Hq, bool masked = false);
size_t kv4_attn_ws_bytes(int N, int B, int Hq, int Hkv, int hd);
dfl_status kv4_attn_run(DeviceCtx* ctx, const dfl_kv4_pool& pool, int layer, const dfl_pages& pg, const void* Q,
                        const void* Kb, const void* Vb, int B, int Hq, const uint64_t* mask, int window, int sinks, void* O,
                        void* ws, cudaStream_t st);

// Page operations (pages.cu).  max_new: a larger n_new is out of range.
size_t pages_reserve_ws(int64_t N, int64_t num_pages);
size_t pages_remap_ws(int64_t N, int64_t max_pages);
size_t pages_compact_ws(int64_t num_pages);
dfl_status pages_reserve_run(DeviceCtx* ctx, const dfl_kv4_pool& pool, const dfl_pages& pg, const int32_t* n_new,
                             int max_new, int32_t* start, void* ws, cudaStream_t st);
dfl_status pages_remap_run(DeviceCtx* ctx, const dfl_kv4_pool& pool, const dfl_pages& pg, const int32_t* parent,
                           const int32_t* keep_len, void* ws, cudaStream_t st);
dfl_status pages_compact_run(DeviceCtx* ctx, const dfl_kv4_pool& pool, const dfl_pages& pg, int32_t* map,
                             int32_t* live, void* ws, cudaStream_t st);

}  // namespace dfl
