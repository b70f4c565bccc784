// Host-side checks that the calls of the paged cache share (internal).
#pragma once

#include <algorithm>
#include <cstdint>

#include "libspecverify.h"

namespace sv {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Layout of a cache: 16-byte loads need every row start on 16 bytes.
inline sv_status check_cache(const sv_cache* c, int32_t max_pages) {
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

inline int log2_exact(int32_t n) {
    for (int i = 0; i < 31; ++i)
        if (n == (int32_t)1 << i) return i;
    return -1;
}

// How many neighbouring heads' rows of a position lie in a 128-byte line.
inline int xcd_run(const sv_cache& c) {
    const int64_t row = (int64_t)c.head_dim * (c.dtype == SV_E4M3 ? 1 : 2);
    if (c.head_stride != c.head_dim || row >= 128) return 1;
    return (int)std::min<int64_t>(128 / row, c.n_kv_heads);
}

// Heads of one row are contiguous; rows start on 16 bytes.
inline bool row_layout_ok(const void* p, int64_t ld, int64_t width) {
    return ld >= width && ld % 8 == 0 && aligned16(p);
}

// Sizes an attend call may have; SV_OK means a plan can be made.
inline sv_status check_attend_sizes(int32_t n_req, int32_t k_max, int32_t n_heads, int32_t n_kv_heads,
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

}  // namespace sv
