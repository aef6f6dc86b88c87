// C-ABI entry points of the paged 4-bit context cache: argument checks.
#include "internal.h"
#include "paged.h"

using namespace dfl;

namespace dfl {

dfl_status kv4_check(const dfl_kv4_pool* pool, int layer, const dfl_pages* pg) {
    if (!pool || !pool->data || pool->layers < 1 || pool->num_pages < 1 || pool->page < 1 || pool->Hkv < 1 ||
        pool->hd < 1 || layer < 0 || layer >= pool->layers)
        return DFL_ERR_INVALID_ARG;
    if (pool->k_exp < -60 || pool->k_exp > 60 || pool->v_exp < -60 || pool->v_exp > 60) return DFL_ERR_INVALID_ARG;
    const int64_t bytes = dfl_kv4_page_bytes(pool->page, pool->Hkv, pool->hd);
    if (bytes == 0) return DFL_ERR_UNSUPPORTED_SHAPE;
    if ((int64_t)pool->num_pages * pool->Hkv * (pool->page / 16) >= (int64_t)1 << 31) return DFL_ERR_UNSUPPORTED_SHAPE;
    if ((int64_t)pool->Hkv * pool->hd >= (int64_t)1 << 31) return DFL_ERR_UNSUPPORTED_SHAPE;
    if (pool->layer_stride < bytes * pool->num_pages) return DFL_ERR_INVALID_ARG;
    if (!aligned16(pool->data) || pool->layer_stride % 16 != 0) return DFL_ERR_MISALIGNED;
    if (!pg) return DFL_OK;
    if (!pg->table || !pg->len || pg->N < 1 || pg->max_pages < 1) return DFL_ERR_INVALID_ARG;
    if ((int64_t)pg->max_pages * pool->page >= (int64_t)1 << 31) return DFL_ERR_UNSUPPORTED_SHAPE;
    if (!aligned4(pg->table) || !aligned4(pg->len) || !aligned4(pg->ref)) return DFL_ERR_MISALIGNED;
    return DFL_OK;
}

namespace {

dfl_status rows_check(const dfl_kv4_pool* pool, int layer, const dfl_pages* pg, const int32_t* start,
                      const int32_t* count, int R, const void* K, const void* V) {
    if (!pg || !start || !count || !K || !V || R < 1) return DFL_ERR_INVALID_ARG;
    const dfl_status rc = kv4_check(pool, layer, pg);
    if (rc != DFL_OK) return rc;
    if (!rows_fit((int64_t)pg->N * R)) return DFL_ERR_UNSUPPORTED_SHAPE;
    if (!aligned16(K) || !aligned16(V) || !aligned4(start) || !aligned4(count)) return DFL_ERR_MISALIGNED;
    return DFL_OK;
}

// Checks shared by the page operations; `need` bytes of ws.
dfl_status pages_check(const dfl_kv4_pool* pool, const dfl_pages* pg, const void* ws, size_t ws_bytes, size_t need) {
    if (!pg || !pg->ref || !ws) return DFL_ERR_INVALID_ARG;
    const dfl_status rc = kv4_check(pool, 0, pg);
    if (rc != DFL_OK) return rc;
    if (!pages_fit(*pg)) return DFL_ERR_UNSUPPORTED_SHAPE;
    if (!aligned16(ws)) return DFL_ERR_MISALIGNED;
    return ws_bytes < need ? DFL_ERR_WORKSPACE : DFL_OK;
}

}  // namespace
}  // namespace dfl

extern "C" size_t dfl_kv4_page_bytes(int32_t page, int32_t Hkv, int32_t hd) {
    if (page < 16 || page > 1024 || page % 16 != 0 || Hkv < 1 || (hd != 64 && hd != 128)) return 0;
    return (size_t)kv4_page_bytes(page, Hkv, hd);
}

extern "C" dfl_status dfl_kv4_append(const dfl_kv4_pool* pool, int32_t layer, const dfl_pages* pages,
                                     const int32_t* start, const int32_t* n_new, int32_t R, const void* K,
                                     const void* V, dfl_stream stream) {
    const dfl::ApiRange nvtx_range("dfl_kv4_append");
    const dfl_status rc = rows_check(pool, layer, pages, start, n_new, R, K, V);
    if (rc != DFL_OK) return rc;
    DeviceCtx* ctx = current_ctx();
    if (!ctx) return DFL_ERR_NO_DEVICE;
    return kv4_append_run(ctx, *pool, layer, *pages, start, n_new, nullptr, R, K, V, static_cast<cudaStream_t>(stream));
}

extern "C" dfl_status dfl_kv4_append_rows(const dfl_kv4_pool* pool, int32_t layer, const dfl_pages* pages,
                                          const int32_t* start, const int32_t* n_new, const int32_t* rows, int32_t R,
                                          const void* K, const void* V, dfl_stream stream) {
    const dfl::ApiRange nvtx_range("dfl_kv4_append_rows");
    if (!rows) return DFL_ERR_INVALID_ARG;
    const dfl_status rc = rows_check(pool, layer, pages, start, n_new, R, K, V);
    if (rc != DFL_OK) return rc;
    if (!aligned4(rows)) return DFL_ERR_MISALIGNED;
    DeviceCtx* ctx = current_ctx();
    if (!ctx) return DFL_ERR_NO_DEVICE;
    return kv4_append_run(ctx, *pool, layer, *pages, start, n_new, rows, R, K, V, static_cast<cudaStream_t>(stream));
}

extern "C" dfl_status dfl_kv4_read(const dfl_kv4_pool* pool, int32_t layer, const dfl_pages* pages,
                                   const int32_t* start, const int32_t* count, int32_t R, void* K, void* V,
                                   dfl_stream stream) {
    const dfl::ApiRange nvtx_range("dfl_kv4_read");
    const dfl_status rc = rows_check(pool, layer, pages, start, count, R, K, V);
    if (rc != DFL_OK) return rc;
    DeviceCtx* ctx = current_ctx();
    if (!ctx) return DFL_ERR_NO_DEVICE;
    return kv4_read_run(ctx, *pool, layer, *pages, start, count, R, K, V, static_cast<cudaStream_t>(stream));
}

namespace {

dfl_status attn_call(const dfl_kv4_pool* pool, int layer, const dfl_pages* pages, const void* Q, const void* Kb, const void* Vb,
                     int B, int Hq, const uint64_t* mask, int window, int sinks, void* O, void* ws, size_t ws_bytes,
                     dfl_stream stream) {
    if (!pages || !Q || !Kb || !Vb || !O || !ws || B < 1 || Hq < 1 || window < 0 || sinks < 0) return DFL_ERR_INVALID_ARG;
    dfl_status rc = kv4_check(pool, layer, pages);
    if (rc != DFL_OK) return rc;
    if (Hq % pool->Hkv != 0) return DFL_ERR_INVALID_ARG;
    if ((rc = kv4_attn_check(*pool, *pages, B, Hq, mask || window > 0)) != DFL_OK) return rc;
    const void* ptrs[] = {Q, Kb, Vb, O, ws};
    for (const void* p : ptrs) if (!aligned16(p)) return DFL_ERR_MISALIGNED;
    if (reinterpret_cast<uintptr_t>(mask) & 7u) return DFL_ERR_MISALIGNED;
    if (ws_bytes < kv4_attn_ws_bytes(pages->N, B, Hq, pool->Hkv, pool->hd)) return DFL_ERR_WORKSPACE;
    DeviceCtx* ctx = current_ctx();
    if (!ctx) return DFL_ERR_NO_DEVICE;
    return kv4_attn_run(ctx, *pool, layer, *pages, Q, Kb, Vb, B, Hq, mask, window, sinks, O, ws,
                        static_cast<cudaStream_t>(stream));
}

}  // namespace

extern "C" dfl_status dfl_kv4_attn(const dfl_kv4_pool* pool, int32_t layer, const dfl_pages* pages, const void* Q,
                                   const void* Kb, const void* Vb, int32_t B, int32_t Hq, void* O, void* ws,
                                   size_t ws_bytes, dfl_stream stream) {
    const dfl::ApiRange nvtx_range("dfl_kv4_attn");
    return attn_call(pool, layer, pages, Q, Kb, Vb, B, Hq, nullptr, 0, 0, O, ws, ws_bytes, stream);
}

extern "C" dfl_status dfl_kv4_attn_masked(const dfl_kv4_pool* pool, int32_t layer, const dfl_pages* pages, const void* Q,
                                          const void* Kb, const void* Vb, int32_t B, int32_t Hq, const uint64_t* mask,
                                          int32_t window, int32_t sinks, void* O, void* ws, size_t ws_bytes,
                                          dfl_stream stream) {
    const dfl::ApiRange nvtx_range("dfl_kv4_attn_masked");
    return attn_call(pool, layer, pages, Q, Kb, Vb, B, Hq, mask, window, sinks, O, ws, ws_bytes, stream);
}

extern "C" dfl_status dfl_pages_reserve(const dfl_kv4_pool* pool, const dfl_pages* pages, const int32_t* n_new,
                                        int32_t* start, void* ws, size_t ws_bytes, dfl_stream stream) {
    const dfl::ApiRange nvtx_range("dfl_pages_reserve");
    if (!pages || !pool || !n_new || !start) return DFL_ERR_INVALID_ARG;
    const dfl_status rc = pages_check(pool, pages, ws, ws_bytes, pages_reserve_ws(pages->N, pool->num_pages));
    if (rc != DFL_OK) return rc;
    if (!aligned4(n_new) || !aligned4(start)) return DFL_ERR_MISALIGNED;
    DeviceCtx* ctx = current_ctx();
    if (!ctx) return DFL_ERR_NO_DEVICE;
    return pages_reserve_run(ctx, *pool, *pages, n_new, INT32_MAX, start, ws, static_cast<cudaStream_t>(stream));
}

extern "C" dfl_status dfl_pages_remap(const dfl_kv4_pool* pool, const dfl_pages* pages, const int32_t* parent,
                                      const int32_t* keep_len, void* ws, size_t ws_bytes, dfl_stream stream) {
    const dfl::ApiRange nvtx_range("dfl_pages_remap");
    if (!pages || !parent) return DFL_ERR_INVALID_ARG;
    const dfl_status rc = pages_check(pool, pages, ws, ws_bytes, pages_remap_ws(pages->N, pages->max_pages));
    if (rc != DFL_OK) return rc;
    if (!aligned4(parent) || !aligned4(keep_len)) return DFL_ERR_MISALIGNED;
    DeviceCtx* ctx = current_ctx();
    if (!ctx) return DFL_ERR_NO_DEVICE;
    return pages_remap_run(ctx, *pool, *pages, parent, keep_len, ws, static_cast<cudaStream_t>(stream));
}

extern "C" dfl_status dfl_pages_compact(const dfl_kv4_pool* pool, const dfl_pages* pages, int32_t* map, int32_t* live,
                                        void* ws, size_t ws_bytes, dfl_stream stream) {
    const dfl::ApiRange nvtx_range("dfl_pages_compact");
    if (!pages || !pool || !map || !live) return DFL_ERR_INVALID_ARG;
    const dfl_status rc = pages_check(pool, pages, ws, ws_bytes, pages_compact_ws(pool->num_pages));
    if (rc != DFL_OK) return rc;
    if (!aligned4(map) || !aligned4(live)) return DFL_ERR_MISALIGNED;
    DeviceCtx* ctx = current_ctx();
    if (!ctx) return DFL_ERR_NO_DEVICE;
    return pages_compact_run(ctx, *pool, *pages, map, live, ws, static_cast<cudaStream_t>(stream));
}
