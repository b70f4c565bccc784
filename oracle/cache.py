"""Paged key-value cache of the packed batch — oracle side (test infrastructure).

agentlens page, section "기술적 구현 및 CUDA Graphs", item Graph Capture: one
decode shape holds 1 .. k+1 query tokens per request.  The pages do not spell
out attention over the cache; this is the textbook softmax attention of those
rows, row j of request r at position ctx_len[r] + j seeing positions up to its
own, position by position, in fp64.
"""

import numpy as np


def e4m3_round(x):
    """Nearest e4m3 value (ties to even), held at +-448; NaN stays NaN.  fp64 in and out.

    Steps of 2^-9 below 2^-6 (subnormals), 2^(e-3) in [2^e, 2^(e+1)) above."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(x), 448.0)
    with np.errstate(divide="ignore", invalid="ignore"):
        e = np.floor(np.log2(np.where(a > 0, a, 1.0)))
    step = np.exp2(np.maximum(e, -6.0) - 3.0)
    y = np.minimum(np.round(a / step) * step, 448.0)  # np.round: ties to even
    return np.where(np.isnan(x), np.nan, np.copysign(y, x))


def cache_append(cache, page_table, new, row_req, row_pos, ctx_len, scale=None):
    """Writes rows new [rows, heads, dim] into cache [pages, page_size, heads, dim] in place.

    scale [heads]: an 8-bit cache, which keeps fp32(x / scale) rounded to e4m3."""
    size = cache.shape[1]
    for i, (r, j) in enumerate(zip(row_req, row_pos)):
        if r < 0:
            continue
        t = int(ctx_len[r]) + int(j)
        x = new[i].astype(np.float32)
        if scale is not None:
            x = e4m3_round((x / np.asarray(scale, np.float32)[:, None]).astype(np.float32))
        cache[page_table[r, t // size], t % size] = x
    return cache


def cache_attend(q, k_cache, v_cache, page_table, cu_rows, ctx_len, scale):
    """(out, lse, spread): softmax attention of the packed rows, fp64.

    q [rows, heads, dim]; caches [pages, page_size, kv_heads, dim] as values.
    A page id outside the cache holds no positions; a row that sees none, or only
    scores of -inf, gives 0 and lse -inf.  spread is the weighted mean of |v|, the
    scale in which rounding of the weights shows.  Rows outside every request: NaN.
    """
    q = np.asarray(q, np.float64)
    rows, heads, dim = q.shape
    pages, size, kv_heads, _ = k_cache.shape
    out = np.full(q.shape, np.nan)
    spread = np.full(q.shape, np.nan)
    lse = np.full((rows, heads), np.nan)
    for r in range(len(ctx_len)):
        for row in range(int(cu_rows[r]), int(cu_rows[r + 1])):
            last = int(ctx_len[r]) + row - int(cu_rows[r])
            t = np.arange(last + 1)
            page = np.asarray(page_table[r])[t // size]
            seen = (page >= 0) & (page < pages)
            page, slot = page[seen], (t % size)[seen]
            for h in range(heads):
                g = h // (heads // kv_heads)
                k = np.asarray(k_cache[page, slot, g], np.float64)
                v = np.asarray(v_cache[page, slot, g], np.float64)
                with np.errstate(invalid="ignore", over="ignore"):
                    s = (k * q[row, h]).sum(-1) * scale
                    if len(s) == 0 or np.all(np.isneginf(s)):
                        out[row, h] = spread[row, h] = 0.0
                        lse[row, h] = -np.inf
                        continue
                    m = np.nanmax(s)
                    w = np.exp(s - m)
                    out[row, h] = (w[:, None] * v).sum(0) / w.sum()
                    spread[row, h] = (w[:, None] * np.abs(v)).sum(0) / w.sum()
                    lse[row, h] = m + np.log(w.sum())
    return out, lse, spread
