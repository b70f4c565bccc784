// C ABI of attention over shared prefixes: host-side validation, then launches on
// the caller's stream.  Every check runs before any HIP call.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "libspecverify.h"
#include "sv_cache_check.h"
#include "sv_launch.h"
#include "sv_shared.h"

namespace {

hipStream_t as_stream(void* s) { return static_cast<hipStream_t>(s); }

// Sizes a call may have; SV_OK means a plan can be made.
sv_status check_sizes(int32_t n_req, int32_t n_groups, int32_t k_max, int32_t n_heads,
                      int32_t n_kv_heads, int32_t head_dim, int64_t capacity) {
    const sv_status s =
        sv::check_attend_sizes(n_req, k_max, n_heads, n_kv_heads, head_dim, capacity);
    if (s != SV_OK) return s;
    if (n_groups < 0 || n_groups > n_req) return SV_ERR_SHAPE;
    // the launch stays below 2^32 work-items
    const sv::SharedPlan p(n_req, n_groups, k_max, n_heads, n_kv_heads, head_dim, 2, capacity);
    return p.chunks + p.own.grid(n_req, n_kv_heads) > SV_MAX_ATTEND_SLOTS ? SV_ERR_SHAPE : SV_OK;
}

}  // namespace

extern "C" {

size_t sv_cache_attend_shared_workspace_bytes(int32_t n_req, int32_t n_groups, int32_t k_max,
                                              int32_t n_heads, int32_t n_kv_heads,
                                              int32_t head_dim, int32_t max_pages,
                                              int32_t page_size) {
    if (max_pages < 0 || page_size < 1) return 0;
    const int64_t capacity = (int64_t)max_pages * page_size;
    if (check_sizes(n_req, n_groups, k_max, n_heads, n_kv_heads, head_dim, capacity) != SV_OK)
        return 0;
    // two-byte caches are cut into no fewer parts than one-byte ones
    const sv::SharedPlan p(n_req, n_groups, k_max, n_heads, n_kv_heads, head_dim, 2, capacity);
    return p.bytes(n_req, n_groups, k_max, n_heads, head_dim);
}

sv_status sv_cache_attend_shared(const sv_cache* cache, const int32_t* page_table,
                                 int32_t max_pages, const void* q, int64_t q_ld, int64_t q_rows,
                                 int32_t n_heads, const int32_t* cu_rows, const int32_t* ctx_len,
                                 int32_t n_req, int32_t k_max, const int32_t* group_start,
                                 const int32_t* prefix_len, int32_t n_groups, float scale,
                                 void* out, int64_t out_ld, float* out_lse, int32_t* dev_error,
                                 void* ws, size_t ws_bytes, void* stream) {
    const sv_status cs = sv::check_cache(cache, max_pages);
    if (cs != SV_OK) return cs;
    const int64_t capacity = (int64_t)max_pages * cache->page_size;
    const sv_status ss = check_sizes(n_req, n_groups, k_max, n_heads, cache->n_kv_heads,
                                     cache->head_dim, capacity);
    if (ss != SV_OK) return ss;
    if (q_rows < 0 || q_rows > INT32_MAX) return SV_ERR_SHAPE;
    if (!std::isfinite(scale)) return SV_ERR_VALUE;
    if (n_req == 0) return SV_OK;
    if (q == nullptr || out == nullptr || cu_rows == nullptr || ctx_len == nullptr ||
        page_table == nullptr || cache->k == nullptr || cache->v == nullptr)
        return SV_ERR_NULL;
    if (n_groups > 0 && (group_start == nullptr || prefix_len == nullptr)) return SV_ERR_NULL;
    const int64_t width = (int64_t)n_heads * cache->head_dim;
    if (!sv::row_layout_ok(q, q_ld, width) || !sv::row_layout_ok(out, out_ld, width))
        return SV_ERR_SHAPE;
    if ((double)q_rows * (double)q_ld > 2.0e18 || (double)q_rows * (double)out_ld > 2.0e18)
        return SV_ERR_SHAPE;
    if (cache->n_pages == 0) return SV_ERR_SHAPE;  // a bad page id reads page 0 instead
    const sv::SharedPlan p(n_req, n_groups, k_max, n_heads, cache->n_kv_heads, cache->head_dim,
                           cache->dtype == SV_E4M3 ? 1 : 2, capacity);
    const size_t need = p.bytes(n_req, n_groups, k_max, n_heads, cache->head_dim);
    if (ws == nullptr || ws_bytes < need || !sv::aligned16(ws)) return SV_ERR_WORKSPACE;
    // what is stored 16 bytes at a time first, then what has 8-byte members
    const size_t segment = (size_t)p.segments() * sv::SharedPlan::kSlots;
    const size_t own = p.own_records(n_req, k_max, n_heads);
    float* prefix_out = static_cast<float*>(ws);
    float* own_out = prefix_out + segment * cache->head_dim;
    float* prefix_ml = own_out + own * cache->head_dim;
    float* own_ml = prefix_ml + segment * 2;
    sv::SharedGroup* group = reinterpret_cast<sv::SharedGroup*>(own_ml + own * 2);
    sv::SharedTotals* totals = reinterpret_cast<sv::SharedTotals*>(group + n_groups + 1);
    sv::SharedSpan* span = reinterpret_cast<sv::SharedSpan*>(totals + 1);
    sv::SharedRequest* request = reinterpret_cast<sv::SharedRequest*>(span + p.blocks);
    int32_t* first = reinterpret_cast<int32_t*>(request + n_req);
    const sv::SharedArgs a{
        {*cache, page_table, max_pages, q, q_ld, q_rows, n_heads, n_heads / cache->n_kv_heads,
         cu_rows, ctx_len, n_req, k_max, scale, out, out_ld, out_lse, dev_error,
         sv::xcd_run(*cache),
         n_req > 1 && n_req <= 256 && p.own.grid(n_req, cache->n_kv_heads) > 1024,
         sv::log2_exact(cache->page_size), p.own.slot_tiles, p.own.slot_blocks, p.own.parts,
         p.own.part_min, own_out, own_ml, first},
        group_start, prefix_len, n_groups, p.chunks, first, request, group, totals, span,
        prefix_out, prefix_ml};
    const hipError_t e = sv::launch_cache_attend_shared(a, as_stream(stream));
    return sv::finish_launch(e, as_stream(stream));
}

}  // extern "C"
