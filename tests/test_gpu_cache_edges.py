"""sv_cache_attend at values near the types' limits, and the bits its weights keep."""

import math

import numpy as np
import pytest
import torch

from test_gpu_cache import BF, F8, Batch, values

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("ctx", [3, 40, 1000, 9000])
def test_values_at_the_largest(dim, ctx):
    """Equal scores over values of the bf16 maximum: their mean is that maximum, while
    their sum is far past fp32."""
    for n in (1, 300):          # the length split, and not
        if n * ctx * dim > 3e7:
            continue
        b = Batch(57, [2] * n, [ctx] * n, 4, 2, dim, 16)
        b.q.zero_()
        most = torch.finfo(BF).max
        b.v.fill_(most)
        b.v[..., 1::2] = -most
        out, lse, _ = b.device().attend()
        got = values(out)[:2 * n]
        assert (got[..., ::2] == most).all() and (got[..., 1::2] == -most).all()
        assert torch.isfinite(lse[:2 * n]).all()


@pytest.mark.parametrize("ctx", [3, 1000, 9000])
def test_values_at_the_smallest(ctx):
    """Equal scores over values of 2^-104: their mean, with nothing lost on the way."""
    b = Batch(62, [2], [ctx], 4, 2, 128, 16)
    b.q.zero_()
    b.v.fill_(2.0 ** -104)
    out, _, _ = b.device().attend()
    assert (values(out)[:2] == 2.0 ** -104).all()


def test_sums_that_fill_up():
    """One part of 300,000 positions a request, of equal scores, then of rising ones: m is
    raised on the way."""
    b = Batch(63, [1] * 2, [300000, 299990], 1, 1, 64, 64, extra=0)
    b.table = b.table.repeat(1024, 1)[:2048].contiguous()      # so many that no length is split
    b.n, b.rows, b.k_max = 2048, [1] * 2048, 0
    b.ctx = torch.full((b.n,), 20, dtype=torch.int32)
    b.ctx[:2] = torch.tensor([300000, 299990])
    b.cu = torch.arange(b.n + 1, dtype=torch.int32)
    b.q = torch.zeros(b.n, 1, 64, dtype=BF)
    assert b.ws() is None
    b.v.zero_()
    most = torch.finfo(BF).max
    b.v[:, :, 0, 0] = 1.0
    b.v[:, :, 0, 1] = most
    out, lse, _ = b.device().attend()
    got = values(out)
    assert (got[:, 0, 0] == 1.0).all() and (got[:, 0, 1] == most).all()
    for r, n in ((0, 300001), (1, 299991), (2, 21)):
        assert abs(float(lse[r]) - math.log(n)) <= 2.0 ** -21 * math.log(n)
    # position t scores t / 2^14 (18 nats over the length), in steps of 1 / 16
    b.q[:, 0, 0] = 1.0 / b.scale / 16
    t = torch.arange(300032)
    for r in range(2):
        page = b.table[r, :300032 // 64].long().repeat_interleave(64)
        b.k[page, t % 64, 0, 0] = (t // 1024).to(BF)
    b.k[..., 1:] = 0
    out, lse, _ = b.device().attend()
    s = (t // 1024).to(BF).double() / 16
    # a lane adds a sixteenth of the weights one by one: n / 16 roundings of 2^-24
    added = 300001 / 16 * 2.0 ** -24
    for r in range(2):
        want = torch.logsumexp(s[:int(b.ctx[r]) + 1], 0)
        assert abs(float(lse[r]) - float(want)) <= added + 2.0 ** -21 * float(want)
    got = values(out)
    # the weights' rounding and the output's, 2^-8 each
    assert (np.abs(got[:2, 0, 0] - 1) <= 2 * 2.0 ** -8 + added).all() and np.isfinite(got).all()


@pytest.mark.parametrize("heads,kv,rows", [(4, 4, 1), (8, 1, 4), (8, 1, 7)])
@pytest.mark.parametrize("ctx", [20, 900, 9000])
def test_large_values_and_uneven_scores(heads, kv, rows, ctx):
    """Values of 2^124: a few weights more than one and their sum passes fp32."""
    b = Batch(58, [rows, 1], [ctx, 5], heads, kv, 128, 16)
    b.v = (b.v.float().clamp(-7, 7) * 2.0 ** 124).to(BF)
    out, _ = b.device().check()
    assert torch.isfinite(out).all()


def test_large_values_beside_faulty_ones():
    """Values near the maximum while a later row's value, NaN, is not seen by all rows."""
    b = Batch(59, [4, 1], [60, 900], 4, 2, 64, 16)
    b.v = (b.v.float().clamp(-7, 7) * 2.0 ** 124).to(BF)
    b.v[int(b.table[0, 3]), 62 % 16, :, 5] = float("nan")
    out, _ = b.device().check()
    assert torch.isfinite(out[:2]).all() and torch.isnan(out[2:4, :, 5]).all()


@pytest.mark.parametrize("ctx", [50, 9000])
def test_large_value_scale(ctx):
    """An 8-bit cache whose value scale is 2^115: only the mean has to be in range."""
    b = Batch(60, [2, 1], [ctx, 20], 4, 2, 128, 16, F8)
    b.scales[1].fill_(2.0 ** 115)
    b.q.zero_()
    b.v.copy_(torch.full(b.v.shape, 448.0))
    out, _, _ = b.device().attend()
    assert (values(out)[:3] == 448.0 * 2.0 ** 115).all()


@pytest.mark.parametrize("ctx", [0, 40, 3000])
def test_rows_of_minus_infinity_over_faulty_values(ctx):
    """All of a row's scores are -inf: it gives 0 and lse -inf whatever the values hold."""
    b = Batch(61, [1, 1], [ctx, 20], 2, 1, 64, 16)
    b.q = b.q.abs() + 1
    for t in range(ctx + 1):
        b.k[int(b.table[0, t // 16]), t % 16] = -float("inf")
    b.v[int(b.table[0, 0]), 0, 0, :3] = torch.tensor([float("nan"), float("inf"), -float("inf")])
    out, lse, err = b.device().attend()
    assert err == 0
    assert (out[0] == 0).all() and torch.isneginf(lse[0]).all()
    assert torch.isfinite(out[1]).all() and torch.isfinite(lse[1]).all()


@pytest.mark.parametrize("dtype", [BF, F8])
@pytest.mark.parametrize("dim,heads,rows", [(64, 1, 1), (128, 8, 4), (128, 8, 7), (256, 4, 2)])
@pytest.mark.parametrize("gap", [0.3, 1.1, 2.7])
def test_weights_keep_sixteen_bits(dtype, dim, heads, rows, gap):
    """Two scores `gap` apart over values of +1 and -1 that nearly cancel: every weight of the
    smaller score is rounded the same way, so their rounding shows in the output (2^-15 of each
    for two bf16 terms, and they are half of the weighted mean of |v|; the scores' own rounding
    is below 2^-20 of it)."""
    ctx = 900
    b = Batch(64, [rows], [ctx], heads, 1, dim, 16, dtype)
    if b.scales:
        for s in b.scales:
            s.fill_(1.0)
    b.q.zero_()
    b.q[:, :, 0] = 1.0
    b.scale = float(np.float32(gap / 16))
    bits = lambda t: t.view(torch.uint8 if dtype == F8 else torch.int16)  # noqa: E731
    bits(b.k).zero_()
    one = torch.tensor([1.0, -1.0, -16.0]).to(dtype)
    low = round(math.exp(gap) / (1 + math.exp(gap)) * ctx)      # so many of the smaller weight
    for t in range(ctx + rows):
        p, s = int(b.table[0, t // 16]), t % 16
        bits(b.v)[p, s] = bits(one)[1 if t < low else 0]
        if t < low:
            bits(b.k)[p, s, 0, 0] = bits(one)[2]
    out, _, _ = b.device().attend()
    (o, _, spread), _ = b.expect()
    got = values(out)[:rows]
    # of the inputs alone: nearly balanced, and each later row adds one more value of +1
    assert (np.abs(o[:rows]) < 0.02 * rows).all()
    tol = 2.0 ** -8 * np.abs(o[:rows]) + (2.0 ** -16 + 2.0 ** -20) * spread[:rows]
    assert (np.abs(got - o[:rows]) <= tol).all(), np.max(np.abs(got - o[:rows]) / tol)


@pytest.mark.parametrize("scores", ["equal", "random"])
@pytest.mark.parametrize("dim,heads,rows", [(64, 1, 1), (128, 8, 4), (128, 8, 7), (256, 4, 2)])
@pytest.mark.parametrize("ctx", [100, 5000])
def test_infinite_values_that_every_row_sees(scores, dim, heads, rows, ctx):
    """A value of inf or -inf far inside the context goes into every row's output as itself,
    one of each sign in one dim as NaN."""
    b = Batch(65, [rows, 1], [ctx, 40], heads, 1, dim, 16, qscale=0.3)
    if scores == "equal":
        b.q.zero_()
    inf = float("inf")
    for t, d, x in ((3, 0, inf), (37, 1, -inf), (38, 2, inf), (39, 2, -inf), (ctx - 40, 3, inf)):
        b.v[int(b.table[0, t // 16]), t % 16, 0, d] = x
    got = values(b.device().attend()[0])
    assert (got[:rows, :, [0, 3]] == inf).all() and (got[:rows, :, 1] == -inf).all()
    assert np.isnan(got[:rows, :, 2]).all()
    assert np.isfinite(got[:rows, :, 4:]).all() and np.isfinite(got[rows]).all()
