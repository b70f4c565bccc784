"""sv_cache_attend where every position counts, and at parts and pages that the
oracle's comparisons of random batches cannot tell apart or do not reach.

With q = 0 every visible position has the same weight, a power of two: sums of
weights are whole multiples of it below 2^24, exact in fp32 in any order, and the
merges' factors are powers of two.  A value row that is zero but for one position's C then gives
C / n for n visible positions: one division and the rounding to bf16 (2^-8 of the
value, and 2^-22 for the fp32 steps).  lse is ln n within 2^-21 of it (the
logarithm's rounding, the product with ln 2), where one position more or less
makes 1 / n: 2^-17 at the longest length here, against 2^-21 * 11.8.
"""

import math

import numpy as np
import pytest
import torch

import adaptive_draft_verification_amd as sv
from test_gpu_cache import BF, F8, Batch, values

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def parts_of(b):
    """Parts the length is cut into, from the workspace: head_dim + 2 floats a row and head."""
    size = sv.sv_cache_attend_workspace_bytes(b.n, b.k_max, b.heads, b.kv, b.dim,
                                              b.table.shape[1], b.page)
    return size // (b.n * b.heads * (b.k_max + 1) * (b.dim + 2) * 4)


def probes(ctx, rows, dim, seed):
    """Up to as many positions as there are dims: the first, those around the context's end
    and past it, and both sides of borders of 32, 128 and 1024 positions."""
    rng = np.random.default_rng(seed)
    last = ctx + rows - 1
    at = [0, ctx - 1, ctx, ctx + 1, last, last + 1]
    for _ in range(dim):
        step = int(rng.choice([32, 128, 128, 1024]))
        at.append(int(rng.integers(0, last // step + 1)) * step - int(rng.integers(0, 2)))
        at.append(int(rng.integers(0, last + 1)))
    return list(dict.fromkeys(t for t in at if t >= 0))[:dim]


def plant(b, seed):
    """Zero queries and values but for 256 at each probe of each request, in a dim of its own."""
    b.q.zero_()
    b.v.view(torch.uint8 if b.v.dtype == F8 else torch.int16).zero_()
    if b.scales:
        b.scales[1].fill_(0.5)
    where = []
    for r in range(b.n):
        at = probes(int(b.ctx[r]), b.rows[r], b.dim, seed + r)
        at = [t for t in at if t < b.table.shape[1] * b.page]
        for d, t in enumerate(at):
            row = b.v[int(b.table[r, t // b.page]), t % b.page]
            row[:, d] = torch.full((b.kv,), 256.0).to(b.v.dtype)
        where.append(at)
    return where


def check_planted(b, seed=0):
    where = plant(b, seed)
    c = 128.0 if b.scales else 256.0
    out, lse, err = b.device().attend()
    assert err == 0
    got, got_lse = values(out), values(lse)
    for r in range(b.n):
        at = np.array(where[r])
        for j in range(b.rows[r]):
            i = int(b.cu[r]) + j
            n = int(b.ctx[r]) + j + 1
            want = np.zeros(b.dim)
            want[:len(at)] = np.where(at < n, c / n, 0.0)
            tol = (2.0 ** -8 + 2.0 ** -22) * want
            bad = np.abs(got[i] - want) > tol
            assert not bad.any(), (r, j, [int(at[d]) for d in np.nonzero(bad)[1] if d < len(at)])
            assert (np.abs(got_lse[i] - math.log(n)) <= 2.0 ** -21 * math.log(n) + 1e-30).all(), \
                (r, j, n, got_lse[i])


@pytest.mark.parametrize("dtype", [BF, F8])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("ctx", [64 * 128 - 1, 64 * 128, 64 * 128 + 1, 100 * 128 - 3, 128 * 128 - 1,
                                 128 * 128 + 5, 131069])
def test_every_position_counts_in_many_parts(dtype, dim, ctx):
    """One request and one head: the length is cut into up to 128 parts, more than the
    join's waves have lanes."""
    b = Batch(50, [2], [ctx], 1, 1, dim, 64, dtype, extra=0)
    assert parts_of(b) == min(128, -(-b.table.shape[1] * 64 // 128))
    check_planted(b, ctx)


@pytest.mark.parametrize("dtype", [BF, F8])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("heads,kv,rows", [(1, 1, 1), (8, 2, 4), (8, 1, 5), (4, 4, 65)])
@pytest.mark.parametrize("page", [1, 8, 16, 17, 48])
def test_every_position_counts(dtype, dim, heads, kv, rows, page):
    """One to four slot tiles, a short and a split length, pages of every kind."""
    check_planted(Batch(51, [rows, 1, rows], [1500, 31, 640], heads, kv, dim, page, dtype), page)


@pytest.mark.parametrize("dtype", [BF, F8])
@pytest.mark.parametrize("ctx", [0, 1, 31, 32, 127, 128, 129, 383, 384])
def test_every_position_counts_in_one_part(dtype, ctx):
    """Enough requests that no length is split."""
    n = 300
    b = Batch(52, [1 + i % 3 for i in range(n)], [max(0, ctx - i % 2) for i in range(n)], 8, 8, 64,
              16, dtype)
    assert b.ws() is None
    check_planted(b, ctx)


@pytest.mark.parametrize("dtype", [BF, F8])
@pytest.mark.parametrize("dim,page", [(64, 16), (128, 64), (128, 8), (256, 32), (256, 3)])
def test_one_key_takes_everything(dtype, dim, page):
    """Each request's scores are 0 but for one position's, of 448: the rows that see it
    give its value, exactly (the other weights are below 2^-500)."""
    rng = np.random.default_rng(dim + page)
    n, G = 40, 2
    rows = [int(x) for x in rng.integers(1, 5, n)]
    ctx = [int(x) for x in rng.integers(0, 700, n)]
    b = Batch(53, rows, ctx, 2 * G, 2, dim, page, dtype)
    b.k.view(torch.uint8 if dtype == F8 else torch.int16).zero_()
    b.q.zero_()
    b.q[:, :, 3] = 448.0 / 16 / b.scale
    if b.scales:
        for s in b.scales:
            s.fill_(1.0)
    at = [int(rng.integers(0, c + m)) for c, m in zip(ctx, rows)]
    for r, t in enumerate(at):
        b.k[int(b.table[r, t // page]), t % page][:, 3] = torch.full((2,), 16.0).to(dtype)
    out, _, err = b.device().attend()
    assert err == 0
    got, v = values(out), values(b.v)
    for r, t in enumerate(at):
        want = v[int(b.table[r, t // page]), t % page].repeat(G, 0)
        for j in range(rows[r]):
            if t <= ctx[r] + j:
                np.testing.assert_array_equal(got[int(b.cu[r]) + j], want, err_msg=f"{r} {j} {t}")


@pytest.mark.parametrize("dtype", [BF, F8])
@pytest.mark.parametrize("dim", [128, 256])
@pytest.mark.parametrize("page", [1, 3, 8, 17, 48])
@pytest.mark.parametrize("heads,kv,rows", [(4, 4, 1), (8, 1, 4), (8, 1, 7)])
def test_pages_at_wide_heads(dtype, dim, page, heads, kv, rows):
    """Pages that hold no multiple of 16 positions, at one, two and four slot tiles."""
    Batch(54, [rows, 1, 2], [15, 64, 203], heads, kv, dim, page, dtype).device().check()


@pytest.mark.parametrize("dtype", [BF, F8])
@pytest.mark.parametrize("dim", [64, 256])
@pytest.mark.parametrize("ctx", [2500, 9001])
def test_parts_at_narrow_and_wide_heads(dtype, dim, ctx):
    """Few parts and many (the two forms of the join) at 64 and 256 dims."""
    b = Batch(55, [3, 1], [ctx, 77], 4, 2, dim, 32, dtype)
    assert 1 < parts_of(b)
    b.device().check()


@pytest.mark.parametrize("dtype", [BF, F8])
def test_parts_beyond_a_wave(dtype):
    """More parts than lanes, random scores."""
    b = Batch(56, [2], [12000], 1, 1, 128, 64, dtype)
    assert parts_of(b) > 64
    b.device().check()
