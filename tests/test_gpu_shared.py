"""Attention over shared prefixes on the GPU: sv_cache_attend_shared against the fp64 oracle
of plain attention.

Tolerances, from the arithmetic (bf16 rounding is off by at most 2^-8, fp32 by 2^-24
relative):
* scores: fp32 sums of dim products (an error of at most (dim + 8) 2^-24 times the sum of
  |q k| scale, the products of bf16 values being exact), and the exponent's own rounding and
  exp2's ulp (2^-21 of a score's size at most): together `delta`, absolute in the score,
  relative in each weight;
* out: 2^-15 of each weight (two bf16 terms), the sums' roundings (n 2^-24 at most) and 2
  delta, all in units of the weighted mean of |v|, then 2^-8 of the output;
* lse: delta, the sum's own rounding (n 2^-24 of it at most) and 2^-22 of the result.
"""

import numpy as np
import pytest
import torch

import adaptive_draft_verification_amd as sv
from oracle.cache import cache_attend

pytestmark = pytest.mark.gpu

BF, F8 = torch.bfloat16, torch.float8_e4m3fn
NAN = float("nan")


@pytest.fixture(autouse=True, scope="module")
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def values(t):
    return t.cpu().float().double().numpy()


class Batch:
    """groups: (prefix, [(rows, own context), ...]) each; before and after: requests without.

    Pages in random order, a table wider than needed.  What the call has no business with is
    spoilt on the device: the table's entries of whole pages of the prefix in the rows of a
    group's later requests (a page id outside the cache), and the prefix's positions on their
    own copy of its last page (NaN)."""

    def __init__(self, seed, groups, heads, kv_heads, dim, page, dtype=BF, k_max=None, extra=2,
                 qscale=1.0, before=(), after=(), head_major=False):
        g = torch.Generator().manual_seed(seed)
        rows, ctx, self.first = [], [], []
        self.start, self.prefix = [len(before)], [p for p, _ in groups]
        for r, c in before:
            rows.append(r), ctx.append(c), self.first.append(0)
        for p, members in groups:
            for r, c in members:
                rows.append(r), ctx.append(p + c), self.first.append(p)
            self.start.append(len(rows))
        for r, c in after:
            rows.append(r), ctx.append(c), self.first.append(0)
        self.n, self.heads, self.kv_heads, self.dim, self.page = len(rows), heads, kv_heads, dim, page
        self.k_max = max(max(rows) - 1, 0) if k_max is None else k_max
        self.ctx = torch.tensor(ctx, dtype=torch.int32)
        self.cu = torch.zeros(self.n + 1, dtype=torch.int32)
        self.cu[1:] = torch.cumsum(torch.tensor(rows), 0)
        width = max(-(-(c + r) // page) for c, r in zip(ctx, rows)) + extra
        pages = self.n * width + 1
        self.table = torch.randperm(pages, generator=g)[:self.n * width].int().view(self.n, width)
        shape = (pages, kv_heads, page, dim) if head_major else (pages, page, kv_heads, dim)
        self.k, self.v = (torch.randn(shape, generator=g).to(dtype) for _ in range(2))
        if head_major:
            self.k, self.v = self.k.transpose(1, 2), self.v.transpose(1, 2)
        self.scales = [None, None] if dtype == BF else [0.5 + torch.rand(kv_heads, generator=g)
                                                        for _ in range(2)]
        self.spoilt = self.table.clone()
        self.holes = []  # (page, positions) of a later request's own copy
        for i, (p, members) in enumerate(groups):
            for r in range(self.start[i] + 1, self.start[i + 1]):
                whole = p // page
                self.table[r, :whole] = self.table[self.start[i], :whole]
                self.spoilt[r, :whole] = 2 ** 31 - 1 if r % 2 else -1
                if p % page:
                    own, of = int(self.table[r, whole]), int(self.table[self.start[i], whole])
                    for c in (self.k, self.v):
                        c[own, :p % page] = c[of, :p % page]
                    self.holes.append((own, p % page))
        self.q = (torch.randn(int(self.cu[-1]) + 3, heads, dim, generator=g) * qscale).to(BF)
        self.scale = dim ** -0.5

    def device(self):
        self.dev = []
        for c in (self.k, self.v):
            d = torch.empty_strided(c.shape, c.stride(), dtype=c.dtype, device="cuda").copy_(c)
            for page, upto in self.holes:
                d[page, :upto] = NAN
            self.dev.append(d)
        self.cache = sv.PagedCache(*self.dev, *[None if s is None else s.cuda() for s in self.scales])
        return self

    def ws(self):
        b = sv.sv_cache_attend_shared_workspace_bytes(
            self.n, len(self.prefix), self.k_max, self.heads, self.kv_heads, self.dim,
            self.table.shape[1], self.page)
        return torch.full((b,), 0xFF, dtype=torch.uint8, device="cuda")

    def arguments(self):
        return (self.cache, self.spoilt.cuda(), self.q.cuda(), self.cu.cuda(), self.ctx.cuda(),
                torch.tensor(self.start, dtype=torch.int32, device="cuda"),
                torch.tensor(self.prefix, dtype=torch.int32, device="cuda"), self.k_max, self.scale)

    def attend(self, stream=None):
        out = torch.full(self.q.shape, -7.0, dtype=BF, device="cuda")
        lse = torch.full(self.q.shape[:2], -7.0, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        sv.sv_cache_attend_shared(*self.arguments(), out, self.ws(), lse, err, stream)
        torch.cuda.synchronize()
        return out, lse, int(err)

    def expect(self):
        k, v = values(self.k), values(self.v)
        if self.scales[0] is not None:
            k = k * self.scales[0].double().numpy()[:, None]
            v = v * self.scales[1].double().numpy()[:, None]
        return cache_attend(values(self.q), k, v, self.table.numpy(), self.cu.numpy(),
                            self.ctx.numpy(), self.scale), k

    def check(self, want_err=0, untouched=()):
        out, lse, err = self.attend()
        assert err == want_err
        (o, e, spread), k = self.expect()
        got, got_lse = values(out), values(lse)
        tail = np.arange(len(e)) >= int(self.cu[-1])
        for r in untouched:
            tail[int(self.cu[r]):int(self.cu[r + 1])] = True
        assert (got[tail] == -7).all() and (got_lse[tail] == -7).all()
        head = ~tail
        kmax = np.abs(k[np.isfinite(k)]).max()
        qsum = np.abs(values(self.q)).sum(-1)[head]
        delta = qsum * kmax * abs(self.scale) * ((self.dim + 8) * 2.0 ** -24 + 2.0 ** -21)
        o, e, spread, got, got_lse = o[head], e[head], spread[head], got[head], got_lse[head]
        np.testing.assert_array_equal(np.isnan(got), np.isnan(o))
        np.testing.assert_array_equal(np.isneginf(got_lse), np.isneginf(e))
        fine = np.isfinite(o)
        n = int(self.ctx.max()) + self.k_max + 1
        tol = 2.0 ** -8 * np.abs(o) + 1e-30
        tol += (2.0 ** -15 + n * 2.0 ** -24 + 2 * delta[..., None]) * spread
        assert (np.abs(got - o) <= tol)[fine].all(), np.max((np.abs(got - o) / tol)[fine])
        f = np.isfinite(e)
        etol = delta + n * 2.0 ** -24 + 2.0 ** -22 * np.abs(e)
        assert (np.abs(got_lse - e) <= etol)[f].all(), np.max((np.abs(got_lse - e) / etol)[f])
        return out, lse


@pytest.mark.parametrize("dtype", [BF, F8])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("heads,kv", [(1, 1), (4, 4), (8, 2), (7, 1), (16, 2)])
def test_heads_and_types(dtype, dim, heads, kv):
    Batch(1, [(37, [(1, 0), (3, 5), (4, 30)]), (64, [(2, 1), (1, 0)])], heads, kv, dim, 16,
          dtype).device().check()


@pytest.mark.parametrize("dtype", [BF, F8])
@pytest.mark.parametrize("page", [1, 3, 8, 16, 17, 64])
def test_pages(dtype, page):
    Batch(2, [(70, [(2, 3), (1, 0), (4, 90)]), (33, [(1, 1), (3, 2)])], 4, 2, 128, page,
          dtype).device().check()


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("prefix", [0, 1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 96, 97, 255, 256])
def test_prefixes_around_tiles(prefix, dim):
    Batch(prefix, [(prefix, [(1, 0), (5, 3), (2, 17)])], 4, 2, dim, 16).device().check()


@pytest.mark.parametrize("own", [0, 1, 14, 15, 16, 31, 32, 47, 127, 128, 200])
def test_own_positions_around_tiles(own):
    Batch(own, [(45, [(1, own), (2, own), (1, 0)])], 4, 1, 64, 16).device().check()


@pytest.mark.parametrize("dtype", [BF, F8])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_a_prefix_in_parts(dtype, dim):
    """Longer than a part, and longer than the positions whose places are kept."""
    Batch(3, [(2400, [(2, 3), (1, 0)])], 4, 2, dim, 16, dtype).device().check()
    Batch(4, [(20000, [(1, 300)]), (1100, [(3, 1)])], 2, 1, dim, 32, dtype, extra=0).device().check()


@pytest.mark.parametrize("dtype", [BF, F8])
def test_small_calls_with_long_tables(dtype):
    """The workspace does not depend on the type; few slots, a table of 8192 positions."""
    Batch(24, [(1000, [(2, i)]) for i in range(8)], 1, 1, 64, 16, dtype, k_max=3,
          extra=448).device().check()


def test_a_part_longer_than_the_places_kept():
    """Room for many rows, so few parts, each of more than 1024 positions."""
    Batch(5, [(4100, [(1 + i % 2, i) for i in range(11)])], 64, 8, 64, 64, extra=0,
          k_max=64).device().check()


@pytest.mark.parametrize("dtype", [BF, F8])
def test_blocks_of_slots(dtype):
    """Groups of more than 128 slots a kv head, of odd counts; requests without rows."""
    members = [(r, c) for r, c in zip([8, 0, 3, 5, 8, 1, 0, 7, 8, 8, 2, 8], range(12))]
    Batch(6, [(90, members), (40, [(0, 4)]), (65, members[:5])], 10, 2, 64, 16,
          dtype).device().check()


def test_requests_outside_of_groups():
    Batch(7, [(50, [(2, 3), (1, 9)]), (0, [(1, 0), (2, 40)])], 8, 2, 128, 16,
          before=[(3, 20), (1, 0)], after=[(1, 200), (2, 3), (0, 5)]).device().check()


def test_no_groups():
    """The same as sv_cache_attend's rows then."""
    b = Batch(8, [], 8, 2, 128, 16, before=[(3, 20), (1, 0), (2, 300)]).device()
    b.check()
    b.start, b.prefix = [0], []
    b.check()


def test_groups_without_requests():
    b = Batch(9, [(50, [(2, 3), (1, 9)]), (20, [(1, 4)])], 8, 2, 128, 16).device()
    b.start, b.prefix = [0, 2, 2, 3], [50, 7, 20]
    b.check()
    b.prefix[1] = 1000  # past the page table, though of no request
    b.check(want_err=sv.SV_DEV_BAD_CTX)


@pytest.mark.parametrize("n", [255, 256, 257, 1300])
def test_many_groups(n):
    """More than the layout has threads; more requests than are ordered."""
    Batch(10, [(33 + i % 3, [(1, i % 5)] * (1 + i % 2)) for i in range(n)], 2, 1, 64, 16,
          extra=0).device().check()


def test_head_major_cache():
    Batch(11, [(70, [(2, 3), (1, 40)])], 8, 4, 128, 16, head_major=True).device().check()


def test_scores_that_rise_and_fall():
    """Maxima in the prefix, at its end, among the own positions."""
    for at in (3, 40, 299, 305):
        b = Batch(12, [(300, [(2, 8), (1, 20)])], 4, 1, 128, 16)
        for r in range(b.n):
            page = int(b.table[r, at // 16])
            b.k[page, at % 16] = (values_like(b.k, 8.0))
        b.q.abs_()
        b.device().check()


def values_like(t, x):
    return torch.full(t.shape[2:], x, dtype=t.dtype)


def test_large_scores():
    Batch(13, [(300, [(2, 8), (1, 20)])], 4, 2, 128, 16, qscale=40.0).device().check()


@pytest.mark.parametrize("scale", [0.0, -0.07, 1e-3, 0.9])
def test_scales(scale):
    b = Batch(14, [(300, [(2, 8), (1, 20)])], 4, 2, 128, 16)
    b.scale = scale
    b.device().check()


def test_large_and_small_values():
    b = Batch(15, [(3000, [(2, 80), (1, 20)])], 4, 2, 64, 16)
    b.v = (b.v.float() * torch.tensor([3e37, 1e-24])[:, None]).to(BF)
    b.device().check()


def test_equal_scores_over_a_long_prefix():
    """Sums of a part that fill up: m is raised on their account."""
    b = Batch(16, [(1120000, [(2, 80), (1, 20)])], 1, 1, 64, 64, extra=0)
    b.k.fill_(0.5)
    b.v = b.v.abs()
    b.device().check()


def test_scores_of_minus_infinity():
    """A prefix of nothing but scores of -inf leaves the own positions; all of them, 0."""
    b = Batch(17, [(40, [(1, 0), (1, 6)])], 4, 2, 64, 16)
    b.q.fill_(1.0)
    for r in range(2):
        for t in range(40):
            b.k[int(b.table[r, t // 16]), t % 16, :, 0] = -float("inf")
    b.k[int(b.table[0, 2]), 40 % 16, 1, 0] = -float("inf")
    out, lse = b.device().check()
    assert (out[0, 2:] == 0).all() and torch.isneginf(lse[0, 2:]).all()


@pytest.mark.parametrize("value", [NAN, float("inf"), -float("inf")])
def test_rows_do_not_touch_each_other(value):
    """A query of one row, a value past another's position, the other group's keys."""
    b = Batch(18, [(40, [(2, 3), (2, 9)]), (33, [(1, 0)])], 4, 2, 128, 16)
    b.q[1, 2, 5] = value
    b.k[int(b.table[1, 3]), 49 % 16 + 1] = value   # the second row's own position
    b.v[int(b.table[1, 3]), 49 % 16 + 1] = value
    b.v[int(b.table[4 - 2, 0]), 7] = value          # the second group's prefix
    b.device().check()


def test_pages_that_are_not_there():
    """Of the prefix, of the own positions; all of them."""
    for holes in ([(0, 1)], [(0, 2), (1, 4)], [(0, i) for i in range(3)], [(1, 3), (1, 4), (1, 5)]):
        b = Batch(19, [(48, [(2, 13), (1, 20)])], 4, 2, 64, 16, extra=1)
        for r, j in holes:
            for table in (b.table, b.spoilt):
                table[r, j] = -1
                if r == 0 and j < 3 and table is b.table:
                    table[1, j] = -1
        b.device().check(want_err=sv.SV_DEV_BAD_PAGE)


def test_faulty_groups_and_requests():
    make = lambda: Batch(20, [(48, [(2, 13), (1, 20)]), (20, [(1, 4), (2, 5)])], 4, 2, 64, 16)
    for prefix in (-1, 10 ** 6, -2 ** 31, 2 ** 31 - 1):
        b = make().device()
        b.prefix[0] = prefix
        b.check(sv.SV_DEV_BAD_CTX, untouched=(0, 1))
    b = make().device()  # a context that the prefix passes
    b.prefix[1] = 25
    for c in (b.k, b.v):
        c[int(b.table[3, 1]), :9] = c[int(b.table[2, 1]), :9]
    b.holes = []
    b.device().ctx[3] = 26
    b.check(sv.SV_DEV_BAD_CTX, untouched=(2,))
    for start in ([0, 2, 5], [-1, 2, 4], [0, 3, 2], [2, 1, 4], [0, 2 ** 31 - 1, 4]):
        b = make().device()
        b.start = start
        b.check(sv.SV_DEV_BAD_CU_ROWS, untouched=range(4))
    for bad in (-1, 100, 2):  # cu_rows[2]: of requests 1 and 2, so of both groups
        b = make()
        cu = b.cu.clone()
        cu[2] = bad
        b.device()
        good, b.cu = b.cu, cu
        out, lse, err = b.attend()
        if bad == 2:  # request 1 without rows, request 2 one more than it had
            continue
        assert err == sv.SV_DEV_BAD_CU_ROWS
        assert (out == -7).all() and (lse == -7).all()


def test_offsets_past_32_bits():
    """A cache of more than 2^32 values; the pages in use at its ends."""
    pages, page, kv, dim = 70000, 64, 8, 128
    b = Batch(21, [(130, [(2, 13), (1, 70)])], 8, kv, dim, page, extra=0)
    old = b.table.clone()
    k = torch.empty(pages, page, kv, dim, dtype=BF, device="cuda")
    v = torch.empty_like(k)
    place = {int(p): pages - 1 - i if i % 2 else i for i, p in enumerate(old.unique())}
    for p, to in place.items():
        k[to], v[to] = b.k[p].cuda(), b.v[p].cuda()
    b.device()
    spoilt = b.spoilt.clone()
    for p, to in place.items():
        spoilt[b.spoilt == p] = to
    b.spoilt = spoilt
    b.cache = sv.PagedCache(k, v)
    b.check()


def test_repeats_two_streams_and_graphs():
    """Repeats agree bit for bit, on two streams at once and replayed from a graph whose
    inputs change between the replays."""
    b = Batch(22, [(300, [(2, 8), (1, 20)]), (1000, [(3, 5), (4, 0)])], 8, 2, 128, 16).device()
    c = Batch(23, [(300, [(2, 8), (1, 20)]), (1000, [(3, 5), (4, 0)])], 8, 2, 128, 16).device()
    want = [x.attend()[:2] for x in (b, c)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    sets = [(x.arguments(), torch.empty_like(w[0]).fill_(-7), torch.empty_like(w[1]).fill_(-7),
             x.ws()) for x, w in zip((b, c), want)]
    torch.cuda.synchronize()
    for _ in range(3):
        for (args, out, lse, ws), s in zip(sets, streams):
            sv.sv_cache_attend_shared(*args, out, ws, lse, None, s)
    torch.cuda.synchronize()
    for (_, out, lse, _), w in zip(sets, want):
        assert torch.equal(out, w[0]) and torch.equal(lse, w[1])
    args, out, lse, ws = sets[0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sv.sv_cache_attend_shared(*args, out, ws, lse)
    start, prefix, table, ctx = args[5], args[6], args[1], args[4]
    for k in range(3):
        out.fill_(-7)
        if k == 1:  # without groups: what was spoilt is needed then
            table.copy_(b.table)
            for d, c in zip(b.dev, (b.k, b.v)):
                d.copy_(c)
            prefix.zero_()
        if k == 2:
            table.copy_(b.spoilt)
            prefix.copy_(torch.tensor(b.prefix, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        if k == 1:  # rounded in other places
            w = want[0][0].float()
            assert bool(((out.float() - w).abs() <= 2.0 ** -7 * w.abs() + 2.0 ** -6).all())
        else:
            assert torch.equal(out, want[0][0]) and torch.equal(lse, want[0][1])
