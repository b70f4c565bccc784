"""Pins of the paged-cache oracle (CPU)."""

import numpy as np
import pytest
import torch

from oracle.cache import cache_append, cache_attend, e4m3_round


def test_e4m3_round_matches_the_type():
    """Every e4m3 value is a fixed point; between neighbours the rounding is torch's."""
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    finite = codes[np.isfinite(codes)]
    np.testing.assert_array_equal(e4m3_round(finite), finite)
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.standard_normal(4000) * s for s in (1e-3, 0.05, 1, 30, 200)])
    mid = np.sort(np.unique(finite))
    x = np.concatenate([x, (mid[1:] + mid[:-1]) / 2]).astype(np.float32)
    want = torch.from_numpy(x).clamp(-448, 448).to(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(e4m3_round(x), want)
    assert np.isnan(e4m3_round(np.nan)) and e4m3_round(np.inf) == 448 and e4m3_round(-1e9) == -448


def test_attend_matches_dense_softmax():
    """Against torch's matrix form on one request whose pages are scattered."""
    g = torch.Generator().manual_seed(1)
    ctx, rows, heads, kv, dim, size = 11, 3, 4, 2, 8, 5
    pages = 4
    table = np.array([[2, 0, 3]], np.int32)
    k = torch.randn(pages, size, kv, dim, generator=g, dtype=torch.float64)
    v = torch.randn(pages, size, kv, dim, generator=g, dtype=torch.float64)
    q = torch.randn(rows, heads, dim, generator=g, dtype=torch.float64)
    out, lse, _ = cache_attend(q.numpy(), k.numpy(), v.numpy(), table, [0, rows], [ctx], 0.3)
    kk = k[table[0]].reshape(-1, kv, dim)[:ctx + rows].repeat_interleave(2, 1)
    vv = v[table[0]].reshape(-1, kv, dim)[:ctx + rows].repeat_interleave(2, 1)
    s = torch.einsum("rhd,thd->rht", q, kk) * 0.3
    mask = torch.arange(ctx + rows)[None] <= ctx + torch.arange(rows)[:, None]
    s = s.masked_fill(~mask[:, None], -np.inf)
    np.testing.assert_allclose(out, torch.einsum("rht,thd->rhd", s.softmax(-1), vv).numpy(),
                               rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(lse, s.logsumexp(-1).numpy(), rtol=1e-12)


def test_attend_edges():
    one = np.ones((1, 1, 1, 4))
    # a single position: its value, whatever the score
    out, lse, _ = cache_attend(np.full((1, 1, 4), 2.0), one, one * 7, [[0]], [0, 1], [0], 1.0)
    assert (out == 7).all() and lse[0, 0] == 8
    # no page: nothing seen
    out, lse, _ = cache_attend(np.ones((1, 1, 4)), one, one, [[9]], [0, 1], [0], 1.0)
    assert (out == 0).all() and lse[0, 0] == -np.inf
    # rows of no request stay unset
    out, _, _ = cache_attend(np.ones((3, 1, 4)), one, one, [[0]], [1, 2], [0], 1.0)
    assert np.isnan(out[[0, 2]]).all() and (out[1] == 1).all()


@pytest.mark.parametrize("scale", [None, [0.5, 2.0]])
def test_append_then_read_back(scale):
    rng = np.random.default_rng(2)
    cache = np.full((3, 4, 2, 8), -999.0)
    table = np.array([[2, 1], [0, 0]], np.int32)
    new = rng.standard_normal((4, 2, 8)).astype(np.float32)
    cache_append(cache, table, new, [0, 0, -1, 1], [0, 1, -1, 0], [3, 0], scale)
    want = new.astype(np.float64)
    if scale is not None:
        want = e4m3_round(new / np.array(scale, np.float32)[:, None])
    np.testing.assert_array_equal(cache[2, 3], want[0])   # position 3: page 2, slot 3
    np.testing.assert_array_equal(cache[1, 0], want[1])   # position 4: the next page
    np.testing.assert_array_equal(cache[0, 0], want[3])
    assert (cache == -999).sum() == cache.size - 3 * 16
