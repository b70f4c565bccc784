// C ABI of the latent cache: host-side validation, then launches on the caller's
// stream.  Every check runs before any HIP call.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "libspecverify.h"
#include "sv_cache_check.h"
#include "sv_latent.h"
#include "sv_launch.h"

namespace {

using sv::aligned16;
using sv::log2_exact;
using sv::row_layout_ok;

hipStream_t as_stream(void* s) { return static_cast<hipStream_t>(s); }

bool latent_dim_ok(int32_t d) { return d == 256 || d == 512; }

// Layout of a cache: 16-byte loads need every position to start on 16 bytes.
sv_status check_cache(const sv_latent_cache* c, int32_t max_pages) {
    if (c == nullptr) return SV_ERR_NULL;
    if (c->dtype != SV_BF16 && c->dtype != SV_E4M3) return SV_ERR_DTYPE;
    if (!latent_dim_ok(c->latent_dim)) return SV_ERR_SHAPE;
    if (c->n_pages < 0 || c->page_size < 1 || max_pages < 0) return SV_ERR_SHAPE;
    if ((int64_t)max_pages * c->page_size > SV_MAX_CONTEXT) return SV_ERR_SHAPE;
    const int64_t per16 = c->dtype == SV_E4M3 ? 16 : 8;
    for (const int64_t s : {c->page_stride, c->token_stride})
        if (s < 0 || s % per16 != 0) return SV_ERR_SHAPE;
    // the largest byte offset a kernel may form must fit int64
    if ((double)c->page_stride * c->n_pages + (double)c->token_stride * c->page_size > 2.0e18)
        return SV_ERR_SHAPE;
    if (!aligned16(c->kv)) return SV_ERR_SHAPE;
    return SV_OK;
}

sv_status check_attend_sizes(int32_t n_req, int32_t k_max, int32_t n_heads, int32_t latent_dim,
                             int64_t capacity) {
    if (n_req < 0 || k_max < 0 || k_max > SV_MAX_DRAFT || n_heads < 1) return SV_ERR_SHAPE;
    if (!latent_dim_ok(latent_dim)) return SV_ERR_SHAPE;
    if (capacity < 0 || capacity > SV_MAX_CONTEXT) return SV_ERR_SHAPE;
    // every grid stays below 2^32 work-items, every count of slots in 32 bits
    if (std::max<int64_t>(n_req, 1) * n_heads * (k_max + 1) > SV_MAX_ATTEND_SLOTS)
        return SV_ERR_SHAPE;
    return SV_OK;
}

}  // namespace

extern "C" {

size_t sv_latent_attend_workspace_bytes(int32_t n_req, int32_t k_max, int32_t n_heads,
                                        int32_t latent_dim, int32_t max_pages,
                                        int32_t page_size) {
    if (max_pages < 0 || page_size < 1) return 0;
    const int64_t capacity = (int64_t)max_pages * page_size;
    if (check_attend_sizes(n_req, k_max, n_heads, latent_dim, capacity) != SV_OK) return 0;
    return sv::LatentPlan(n_req, k_max, n_heads, capacity)
        .bytes(n_req, k_max, n_heads, latent_dim);
}

sv_status sv_latent_append(const sv_latent_cache* cache, const int32_t* page_table,
                           int32_t max_pages, const void* latent, int64_t latent_ld,
                           const void* rope, int64_t rope_ld, const int32_t* row_req,
                           const int32_t* row_pos, int32_t n_rows, const int32_t* ctx_len,
                           int32_t n_req, int32_t* dev_error, void* stream) {
    const sv_status cs = check_cache(cache, max_pages);
    if (cs != SV_OK) return cs;
    if (n_rows < 0 || n_req < 0) return SV_ERR_SHAPE;
    if ((int64_t)n_rows * (cache->latent_dim + SV_LATENT_ROPE) > SV_MAX_APPEND_VALUES)
        return SV_ERR_SHAPE;
    if (n_rows == 0 || n_req == 0) return SV_OK;
    if (latent == nullptr || rope == nullptr || row_req == nullptr || row_pos == nullptr ||
        ctx_len == nullptr || page_table == nullptr || cache->kv == nullptr)
        return SV_ERR_NULL;
    if (!row_layout_ok(latent, latent_ld, cache->latent_dim) ||
        !row_layout_ok(rope, rope_ld, SV_LATENT_ROPE))
        return SV_ERR_SHAPE;
    if ((double)n_rows * (double)latent_ld > 2.0e18 || (double)n_rows * (double)rope_ld > 2.0e18)
        return SV_ERR_SHAPE;
    const sv::LatentAppendArgs a{*cache,  page_table, max_pages, latent,  latent_ld, rope,    rope_ld,
                                 row_req, row_pos,    n_rows,    ctx_len, n_req,     dev_error};
    const hipError_t e = sv::launch_latent_append(a, as_stream(stream));
    return sv::finish_launch(e, as_stream(stream));
}

sv_status sv_latent_attend(const sv_latent_cache* cache, const int32_t* page_table,
                           int32_t max_pages, const void* q, int64_t q_ld, int64_t q_rows,
                           int32_t n_heads, const int32_t* cu_rows, const int32_t* ctx_len,
                           int32_t n_req, int32_t k_max, float scale, void* out, int64_t out_ld,
                           float* out_lse, int32_t* dev_error, void* ws, size_t ws_bytes,
                           void* stream) {
    const sv_status cs = check_cache(cache, max_pages);
    if (cs != SV_OK) return cs;
    const int64_t capacity = (int64_t)max_pages * cache->page_size;
    const sv_status ss = check_attend_sizes(n_req, k_max, n_heads, cache->latent_dim, capacity);
    if (ss != SV_OK) return ss;
    if (q_rows < 0 || q_rows > INT32_MAX) return SV_ERR_SHAPE;
    if (!std::isfinite(scale)) return SV_ERR_VALUE;
    if (n_req == 0) return SV_OK;
    if (q == nullptr || out == nullptr || cu_rows == nullptr || ctx_len == nullptr ||
        page_table == nullptr || cache->kv == nullptr)
        return SV_ERR_NULL;
    if (!row_layout_ok(q, q_ld, (int64_t)n_heads * (cache->latent_dim + SV_LATENT_ROPE)) ||
        !row_layout_ok(out, out_ld, (int64_t)n_heads * cache->latent_dim))
        return SV_ERR_SHAPE;
    if ((double)q_rows * (double)q_ld > 2.0e18 || (double)q_rows * (double)out_ld > 2.0e18)
        return SV_ERR_SHAPE;
    if (cache->n_pages == 0) return SV_ERR_SHAPE;
    const sv::LatentPlan p(n_req, k_max, n_heads, capacity);
    const size_t need = p.bytes(n_req, k_max, n_heads, cache->latent_dim);
    if (need > 0 && (ws == nullptr || ws_bytes < need)) return SV_ERR_WORKSPACE;
    if (!aligned16(ws)) return SV_ERR_WORKSPACE;
    float* part_out = static_cast<float*>(ws);
    float* part_ml = nullptr;
    if (need > 0)
        part_ml = part_out + (size_t)n_req * n_heads * (k_max + 1) * p.parts * cache->latent_dim;
    const sv::LatentAttendArgs a{*cache, page_table, max_pages, q, q_ld, q_rows, n_heads, cu_rows,
                                 ctx_len, n_req, k_max, scale, out, out_ld, out_lse, dev_error,
                                 n_req > 1 && n_req <= 256 && p.grid(n_req) > 256,
                                 log2_exact(cache->page_size), p.slot_blocks, p.parts,
                                 p.part_min, part_out, part_ml};
    const hipError_t e = sv::launch_latent_attend(a, as_stream(stream));
    return sv::finish_launch(e, as_stream(stream));
}

}  // extern "C"
