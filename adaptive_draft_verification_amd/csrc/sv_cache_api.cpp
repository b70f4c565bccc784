// C ABI of the paged key-value cache: host-side validation, then launches on
// the caller's stream.  Every check runs before any HIP call.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "libspecverify.h"
#include "sv_launch.h"
#include "sv_serve.h"

namespace {

hipStream_t as_stream(void* s) { return static_cast<hipStream_t>(s); }

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Layout of a cache: 16-byte loads need every row start on 16 bytes.
sv_status check_cache(const sv_cache* c, int32_t max_pages) {
    if (c == nullptr) return SV_ERR_NULL;
    if (c->dtype != SV_BF16 && c->dtype != SV_E4M3) return SV_ERR_DTYPE;
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return SV_ERR_SHAPE;
    if (c->n_pages < 0 || c->page_size < 1 || c->n_kv_heads < 1 || max_pages < 0)
        return SV_ERR_SHAPE;
    if ((int64_t)max_pages * c->page_size > SV_MAX_CONTEXT) return SV_ERR_SHAPE;
    const int64_t per16 = c->dtype == SV_E4M3 ? 16 : 8;
    for (const int64_t s : {c->page_stride, c->token_stride, c->head_stride})
        if (s < 0 || s % per16 != 0) return SV_ERR_SHAPE;
    // the largest byte offset a kernel may form must fit int64
    if ((double)c->page_stride * c->n_pages + (double)c->token_stride * c->page_size +
            (double)c->head_stride * c->n_kv_heads > 2.0e18)
        return SV_ERR_SHAPE;
    if (!aligned16(c->k) || !aligned16(c->v)) return SV_ERR_SHAPE;
    return SV_OK;
}

int log2_exact(int32_t n) {
    for (int i = 0; i < 31; ++i)
        if (n == (int32_t)1 << i) return i;
    return -1;
}

// How many neighbouring heads' rows of a position lie in a 128-byte line.
int xcd_run(const sv_cache& c) {
    const int64_t row = (int64_t)c.head_dim * (c.dtype == SV_E4M3 ? 1 : 2);
    if (c.head_stride != c.head_dim || row >= 128) return 1;
    return (int)std::min<int64_t>(128 / row, c.n_kv_heads);
}

// Heads of one row are contiguous; rows start on 16 bytes.
bool row_layout_ok(const void* p, int64_t ld, int64_t width) {
    return ld >= width && ld % 8 == 0 && aligned16(p);
}

// Sizes an attend call may have; SV_OK means a plan can be made.
sv_status check_attend_sizes(int32_t n_req, int32_t k_max, int32_t n_heads, int32_t n_kv_heads,
                             int32_t head_dim, int64_t capacity) {
    if (n_req < 0 || k_max < 0 || k_max > SV_MAX_DRAFT) return SV_ERR_SHAPE;
    if (n_kv_heads < 1 || n_heads < n_kv_heads || n_heads % n_kv_heads != 0) return SV_ERR_SHAPE;
    if (head_dim != 64 && head_dim != 128 && head_dim != 256) return SV_ERR_SHAPE;
    if (capacity < 0 || capacity > SV_MAX_CONTEXT) return SV_ERR_SHAPE;
    // every grid stays below 2^32 work-items, every count of slots in 32 bits
    if (std::max<int64_t>(n_req, 1) * n_heads * (k_max + 1) > SV_MAX_ATTEND_SLOTS)
        return SV_ERR_SHAPE;
    return SV_OK;
}

}  // namespace

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
