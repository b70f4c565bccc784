"""Attention to latent vectors — oracle side (test infrastructure).

The absorbed form of attention whose keys and values are up-projected from one
latent vector a token: keys are (latent, rope), values the latent vector, every
head sees the same ones.  That is softmax attention with one kv head, so the
positions, pages and masks are oracle.cache's; fp64.
"""

import numpy as np

from .cache import cache_append, cache_attend


def latent_append(cache, page_table, latent, rope, row_req, row_pos, ctx_len, scale=None):
    """Writes rows (latent, rope) into cache [pages, page_size, dim] in place; scale: 8 bits."""
    new = np.concatenate([latent, rope], -1)[:, None]
    cache_append(cache[:, :, None], page_table, new, row_req, row_pos, ctx_len,
                 None if scale is None else [scale])
    return cache


def latent_attend(q, cache, latent_dim, page_table, cu_rows, ctx_len, scale):
    """(out, lse, spread) of q [rows, heads, dim] over cache [pages, page_size, dim] as values.

    A step's own vector (behind the context) that is not finite makes NaN of the rows
    that see it."""
    cache = np.array(cache, np.float64)
    size = cache.shape[1]
    hurt = np.zeros((q.shape[0], q.shape[1]), bool)
    for r in range(len(ctx_len)):
        for j in range(1, int(cu_rows[r + 1]) - int(cu_rows[r])):
            t = int(ctx_len[r]) + j
            page = int(page_table[r][t // size])
            if 0 <= page < len(cache) and not np.isfinite(cache[page, t % size]).all():
                cache[page, t % size] = 0.0
                hurt[int(cu_rows[r]) + j:int(cu_rows[r + 1])] = True
    v = np.zeros(cache.shape)
    v[..., :latent_dim] = cache[..., :latent_dim]
    out, lse, spread = cache_attend(q, cache[:, :, None], v[:, :, None], page_table, cu_rows,
                                    ctx_len, scale)
    out[hurt], lse[hurt] = np.nan, np.nan
    return out[..., :latent_dim], lse, spread[..., :latent_dim]
