// C ABI of the paged key-value cache: host-side validation, then launches on
// the caller's stream.  Every check runs before any HIP call.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "libspecverify.h"
#include "sv_cache_check.h"
#include "sv_launch.h"
#include "sv_serve.h"

namespace {

hipStream_t as_stream(void* s) { return static_cast<hipStream_t>(s); }

}  // namespace

using namespace sv;

extern "C" {

size_t sv_cache_attend_workspace_bytes(int32_t n_req, int32_t k_max, int32_t n_heads,
                                       int32_t n_kv_heads, int32_t head_dim, int32_t max_pages,
                                       int32_t page_size) {
    if (max_pages < 0 || page_size < 1) return 0;
    const int64_t capacity = (int64_t)max_pages * page_size;
    if (check_attend_sizes(n_req, k_max, n_heads, n_kv_heads, head_dim, capacity) != SV_OK)
        return 0;
    // two-byte caches are cut into no fewer parts than one-byte ones
    const sv::AttendPlan p(n_req, k_max, n_heads, n_kv_heads, head_dim, 2, capacity);
    return p.bytes(n_req, k_max, n_heads, head_dim);
}

sv_status sv_cache_append(const sv_cache* cache, const int32_t* page_table, int32_t max_pages,
                          const void* k, const void* v, int64_t kv_ld, const int32_t* row_req,
                          const int32_t* row_pos, int32_t n_rows, const int32_t* ctx_len,
                          int32_t n_req, int32_t* dev_error, void* stream) {
    const sv_status cs = check_cache(cache, max_pages);
    if (cs != SV_OK) return cs;
    if (n_rows < 0 || n_req < 0) return SV_ERR_SHAPE;
    const int64_t width = (int64_t)cache->n_kv_heads * cache->head_dim;
    if (width > INT32_MAX || (int64_t)n_rows * width > SV_MAX_APPEND_VALUES) return SV_ERR_SHAPE;
    if (n_rows == 0 || n_req == 0) return SV_OK;
    if (k == nullptr || v == nullptr || row_req == nullptr || row_pos == nullptr ||
        ctx_len == nullptr || page_table == nullptr || cache->k == nullptr || cache->v == nullptr)
        return SV_ERR_NULL;
    if (!row_layout_ok(k, kv_ld, width) || !row_layout_ok(v, kv_ld, width)) return SV_ERR_SHAPE;
    if ((double)n_rows * (double)kv_ld > 2.0e18) return SV_ERR_SHAPE;
    const sv::AppendArgs a{*cache, page_table, max_pages, k,     v,        kv_ld, row_req,
                           row_pos, n_rows,    ctx_len,   n_req, dev_error};
    const hipError_t e = sv::launch_cache_append(a, as_stream(stream));
    return sv::finish_launch(e, as_stream(stream));
}

sv_status sv_cache_attend(const sv_cache* cache, const int32_t* page_table, int32_t max_pages,
                          const void* q, int64_t q_ld, int64_t q_rows, int32_t n_heads,
                          const int32_t* cu_rows, const int32_t* ctx_len, int32_t n_req,
                          int32_t k_max, float scale, void* out, int64_t out_ld, float* out_lse,
                          int32_t* dev_error, void* ws, size_t ws_bytes, void* stream) {
    const sv_status cs = check_cache(cache, max_pages);
    if (cs != SV_OK) return cs;
    const int64_t capacity = (int64_t)max_pages * cache->page_size;
    const sv_status ss = check_attend_sizes(n_req, k_max, n_heads, cache->n_kv_heads,
                                            cache->head_dim, capacity);
    if (ss != SV_OK) return ss;
    if (q_rows < 0 || q_rows > INT32_MAX) return SV_ERR_SHAPE;
    if (!std::isfinite(scale)) return SV_ERR_VALUE;
    if (n_req == 0) return SV_OK;
    if (q == nullptr || out == nullptr || cu_rows == nullptr || ctx_len == nullptr ||
        page_table == nullptr || cache->k == nullptr || cache->v == nullptr)
        return SV_ERR_NULL;
    const int64_t width = (int64_t)n_heads * cache->head_dim;
    if (!row_layout_ok(q, q_ld, width) || !row_layout_ok(out, out_ld, width)) return SV_ERR_SHAPE;
    if ((double)q_rows * (double)q_ld > 2.0e18 || (double)q_rows * (double)out_ld > 2.0e18)
        return SV_ERR_SHAPE;
    if (cache->n_pages == 0) return SV_ERR_SHAPE;  // a bad page id reads page 0 instead
    const sv::AttendPlan p(n_req, k_max, n_heads, cache->n_kv_heads, cache->head_dim,
                           cache->dtype == SV_E4M3 ? 1 : 2, capacity);
    const size_t need = p.bytes(n_req, k_max, n_heads, cache->head_dim);
    if (need > 0 && (ws == nullptr || ws_bytes < need)) return SV_ERR_WORKSPACE;
    if (!aligned16(ws)) return SV_ERR_WORKSPACE;
    float* part_out = static_cast<float*>(ws);
    float* part_ml = nullptr;
    if (need > 0)
        part_ml = part_out +
                  (size_t)n_req * n_heads * (k_max + 1) * p.parts * cache->head_dim;
    const sv::AttendArgs a{*cache,  page_table, max_pages, q,       q_ld,
                           q_rows,  n_heads,    n_heads / cache->n_kv_heads,
                           cu_rows, ctx_len,    n_req,     k_max,   scale,
                           out,     out_ld,     out_lse,   dev_error, xcd_run(*cache),
                           n_req > 1 && n_req <= 256 && p.grid(n_req, cache->n_kv_heads) > 1024,
                           log2_exact(cache->page_size),
                           p.slot_tiles, p.slot_blocks, p.parts, p.part_min, part_out, part_ml};
    const hipError_t e = sv::launch_cache_attend(a, as_stream(stream));
    return sv::finish_launch(e, as_stream(stream));
}

}  // extern "C"
