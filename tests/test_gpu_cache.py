"""The paged cache on the GPU: sv_cache_append and sv_cache_attend against the
fp64 oracle.

Tolerances, from the arithmetic (bf16 rounding is off by at most 2^-8, fp32 by
2^-24 relative):
* scores: fp32 sums of dim products (an error of at most (dim + 8) 2^-24 times
  the sum of |q k| scale, the products of bf16 values being exact), and the
  exponent's own rounding and exp2's ulp (2^-21 of a score's size at most):
  together `delta`, absolute in the score, relative in each weight;
* out: 2^-8 of each weight (rounded to bf16 for the product) and 2 delta, both
  in units of the weighted mean of |v|, then 2^-8 of the output;
* lse: delta, the sum's own rounding (n 2^-24 of it at most) and 2^-22 of the
  result.
"""

import numpy as np
import pytest
import torch

import adaptive_draft_verification_amd as sv
from oracle.cache import cache_append, cache_attend, e4m3_round

pytestmark = pytest.mark.gpu

BF, F8 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(autouse=True, scope="module")
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def values(t):
    return t.cpu().double().numpy() if t.dtype != F8 else t.cpu().float().double().numpy()


class Batch:
    """A batch of requests: pages in random order, a table wider than needed."""

    def __init__(self, seed, rows, ctx, heads, kv, dim, page, dtype=BF, k_max=None, extra=2,
                 layout="nhd", qscale=1.5):
        g = torch.Generator().manual_seed(seed)
        self.n, self.kv, self.heads, self.dim, self.page = len(rows), kv, heads, dim, page
        self.k_max = max(max(rows) - 1, 0) if k_max is None else k_max
        self.rows, self.ctx = rows, torch.tensor(ctx, dtype=torch.int32)
        self.cu = torch.zeros(self.n + 1, dtype=torch.int32)
        self.cu[1:] = torch.cumsum(torch.tensor(rows), 0)
        need = max(-(-(c + r) // page) for c, r in zip(ctx, rows))
        width = need + extra
        pages = self.n * width + 1
        self.table = torch.randperm(pages, generator=g)[:self.n * width].int().view(self.n, width)
        shape = (pages, page, kv, dim) if layout == "nhd" else (pages, kv, page, dim)
        self.scales = None
        if dtype == F8:
            self.scales = [0.5 + torch.rand(kv, generator=g) for _ in range(2)]
        self.k, self.v = [torch.randn(shape, generator=g).to(dtype) for _ in range(2)]
        if layout == "hnd":
            self.k, self.v = self.k.transpose(1, 2), self.v.transpose(1, 2)
        total = int(self.cu[-1])
        self.q = (torch.randn(total + 3, heads, dim, generator=g) * qscale).to(BF)
        self.scale = dim ** -0.5

    def device(self):
        self.kd, self.vd = self.k.cuda(), self.v.cuda()
        if not self.k.is_contiguous():
            self.kd = self.k.transpose(1, 2).contiguous().cuda().transpose(1, 2)
            self.vd = self.v.transpose(1, 2).contiguous().cuda().transpose(1, 2)
        self.cache = sv.PagedCache(self.kd, self.vd,
                                   *([s.cuda() for s in self.scales] if self.scales else []))
        return self

    def ws(self):
        b = sv.sv_cache_attend_workspace_bytes(self.n, self.k_max, self.heads, self.kv, self.dim,
                                               self.table.shape[1], self.page)
        return torch.full((b,), 0xFF, dtype=torch.uint8, device="cuda") if b else None

    def attend(self, q=None, stream=None):
        q = self.q.cuda() if q is None else q
        out = torch.full(q.shape, -7.0, dtype=BF, device="cuda")
        lse = torch.full(q.shape[:2], -7.0, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        sv.sv_cache_attend(self.cache, self.table.cuda(), q, self.cu.cuda(), self.ctx.cuda(),
                           self.k_max, self.scale, out, self.ws(), lse, err, stream)
        torch.cuda.synchronize()
        return out, lse, int(err)

    def expect(self):
        k, v = values(self.k), values(self.v)
        if self.scales:
            k = k * self.scales[0].double().numpy()[:, None]
            v = v * self.scales[1].double().numpy()[:, None]
        return cache_attend(values(self.q), k, v, self.table.numpy(), self.cu.numpy(),
                            self.ctx.numpy(), self.scale), k

    def check(self, want_err=0):
        out, lse, err = self.attend()
        assert err == want_err
        (o, e, spread), k = self.expect()
        live = ~np.isnan(e) | (np.arange(len(e)) < int(self.cu[-1]))[:, None]
        got, got_lse = values(out), values(lse)
        tail = np.arange(len(e)) >= int(self.cu[-1])
        assert (got[tail] == -7).all() and (got_lse[tail] == -7).all()
        head = ~tail
        kmax = np.abs(k[np.isfinite(k)]).max()
        qsum = np.abs(values(self.q)).sum(-1)[head]
        delta = qsum * kmax * abs(self.scale) * ((self.dim + 8) * 2.0 ** -24 + 2.0 ** -21)
        o, e, spread, got, got_lse = o[head], e[head], spread[head], got[head], got_lse[head]
        np.testing.assert_array_equal(np.isnan(got), np.isnan(o))
        np.testing.assert_array_equal(np.isneginf(got_lse), np.isneginf(e))
        fine = np.isfinite(o)
        np.testing.assert_array_equal(got[~fine & ~np.isnan(o)], o[~fine & ~np.isnan(o)])
        tol = 2.0 ** -8 * np.abs(o) + (2.0 ** -8 + 2 * delta[..., None]) * spread + 1e-30
        assert (np.abs(got - o) <= tol)[fine].all(), np.max((np.abs(got - o) / tol)[fine])
        n = int(self.ctx.max()) + self.k_max + 1
        f = np.isfinite(e)
        etol = delta + n * 2.0 ** -24 + 2.0 ** -22 * np.abs(e)
        assert (np.abs(got_lse - e) <= etol)[f].all(), np.max((np.abs(got_lse - e) / etol)[f])
        assert live.any()
        return out, lse


@pytest.mark.parametrize("dtype", [BF, F8])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("heads,kv", [(1, 1), (4, 4), (8, 2), (7, 1), (16, 2)])
def test_attend_heads_and_types(dtype, dim, heads, kv):
    Batch(1, [1, 3, 4], [0, 37, 130], heads, kv, dim, 16, dtype).device().check()


@pytest.mark.parametrize("page", [1, 3, 8, 16, 17, 32, 48, 128])
@pytest.mark.parametrize("dtype", [BF, F8])
def test_attend_page_sizes(page, dtype):
    """Pages that end inside a tile, hold one position, or are no power of two."""
    Batch(2, [2, 1, 5], [15, 64, 203], 8, 2, 64, page, dtype).device().check()


@pytest.mark.parametrize("ctx", [0, 1, 14, 15, 16, 31, 32, 33, 127, 128, 129, 255, 1000])
def test_attend_single_token(ctx):
    Batch(3, [1], [ctx], 8, 2, 128, 16).device().check()


@pytest.mark.parametrize("rows", [1, 2, 8, 16, 33, 65])
@pytest.mark.parametrize("heads", [1, 3, 8])
def test_attend_many_rows(rows, heads):
    """Up to 65 rows of 8 heads: several slot blocks, tiles with a partly empty end."""
    Batch(4, [rows, 1], [50, 3], heads, 1, 64, 32).device().check()


def test_attend_ragged_batch_with_empty_requests():
    rng = np.random.default_rng(5)
    rows = [int(x) for x in rng.integers(0, 9, 24)]
    ctx = [int(x) for x in rng.integers(0, 400, 24)]
    Batch(5, rows, ctx, 8, 2, 128, 64, k_max=8).device().check()


@pytest.mark.parametrize("dtype", [BF, F8])
def test_attend_long_context_in_parts(dtype):
    b = Batch(6, [3, 1], [9001, 77], 4, 2, 128, 64, dtype)
    assert sv.sv_cache_attend_workspace_bytes(b.n, b.k_max, 4, 2, 128, b.table.shape[1], 64) > 0
    b.device().check()


def test_attend_one_part():
    """Enough requests that the length is not split: no workspace."""
    b = Batch(7, [1] * 300, [5 + i % 40 for i in range(300)], 8, 8, 64, 16)
    assert b.ws() is None
    b.device().check()


def test_attend_layouts_agree():
    """Heads before positions within a page, and query rows that are part of wider ones."""
    b = Batch(8, [4, 2], [70, 9], 8, 2, 128, 16, layout="hnd").device()
    out, lse = b.check()
    wide = torch.zeros(b.q.shape[0], 3, 8, 128, dtype=BF, device="cuda")
    wide[:, 1] = b.q.cuda()
    out2, lse2, _ = b.attend(wide[:, 1])
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


def test_attend_large_scores():
    """Scores in the hundreds: one position takes almost everything."""
    Batch(9, [4, 1], [300, 40], 4, 1, 128, 16, qscale=60.0).device().check()


def test_attend_ignores_what_it_does_not_see():
    """NaN and infinities past each row's position: in unwritten slots and in the
    keys and values of the request's own later rows."""
    for dtype in (BF, F8):
        b = Batch(10, [1, 5, 3], [40, 66, 128], 8, 2, 64, 16, dtype)
        nan = torch.tensor(float("nan")).to(dtype)
        inf = torch.tensor(float("inf")).to(BF) if dtype == BF else nan
        as_int = lambda t: t.view(torch.uint8) if dtype == F8 else t  # noqa: E731
        for r in range(3):
            for t in range(int(b.ctx[r]) + b.rows[r], b.table.shape[1] * 16):
                p = b.table[r, t // 16]
                as_int(b.k)[p, t % 16] = as_int(nan.reshape(1))[0]
                as_int(b.v)[p, t % 16] = as_int(nan.reshape(1))[0]
        used = set(b.table.flatten().tolist())
        for p in range(b.k.shape[0]):
            if p not in used:
                as_int(b.v)[p] = as_int(nan.reshape(1))[0]
        # request 1's row 3 (position 69): rows 0..2 must not see it, rows 3, 4 do
        p, s = b.table[1, 69 // 16], 69 % 16
        as_int(b.v)[p, s, 0, 5] = as_int(nan.reshape(1))[0]
        as_int(b.v)[p, s, 1, 63] = as_int(inf.reshape(1))[0]
        # request 2's row 2 (position 130): its key
        p, s = b.table[2, 130 // 16], 130 % 16
        as_int(b.k)[p, s, 0, 0] = as_int(nan.reshape(1))[0]
        out, _ = b.device().check()
        o = out.float().cpu()
        assert torch.isfinite(o[:4]).all() and not torch.isfinite(o[4:6]).all()


def test_attend_scores_of_minus_infinity():
    """A key of -inf takes its position out; a row with nothing else gives 0 and -inf."""
    b = Batch(11, [1, 1], [0, 20], 2, 1, 64, 16)
    b.q = b.q.abs() + 1
    b.k[b.table[0, 0], 0] = -float("inf")
    b.k[b.table[1, 0], 3] = -float("inf")
    out, lse = b.device().check()
    assert (out[0] == 0).all() and torch.isneginf(lse[0]).all() and torch.isfinite(lse[1]).all()


def test_attend_bad_pages_are_absent():
    b = Batch(12, [2, 1, 2], [90, 10, 40], 4, 2, 64, 16)
    b.table[0, 1], b.table[0, 3], b.table[1, 0] = -1, b.k.shape[0], 2 ** 31 - 1
    b.k[0], b.v[0] = float("nan"), float("nan")     # page 0 must not leak in
    b.table[b.table == 0] = 1
    out, lse = b.device().check(want_err=sv.SV_DEV_BAD_PAGE)
    assert (out[2] == 0).all() and torch.isneginf(lse[2]).all()
    b = Batch(13, [2], [30], 4, 2, 64, 5)
    b.table[0, 2] = -3
    b.device().check(want_err=sv.SV_DEV_BAD_PAGE)


def test_attend_faulty_requests_write_nothing():
    b = Batch(14, [2, 2, 2, 2], [20, 20, 20, 20], 4, 2, 64, 16).device()
    good, good_lse, _ = b.attend()
    b.ctx[1] = -1
    b.ctx[2] = b.table.shape[1] * 16 - 1     # its second row is past the table
    out, lse, err = b.attend()
    assert err == sv.SV_DEV_BAD_CTX
    assert (out[2:6] == -7).all() and (lse[2:6] == -7).all()
    assert torch.equal(out[:2], good[:2]) and torch.equal(out[6:8], good[6:8])
    b = Batch(14, [2, 2, 2, 2], [20, 20, 20, 20], 4, 2, 64, 16).device()
    b.cu = torch.tensor([0, 2, 1, 9, 8 + 4], dtype=torch.int32)  # backwards; too many; past the end
    out, _, err = b.attend()
    assert err == sv.SV_DEV_BAD_CU_ROWS
    assert torch.equal(out[:2], good[:2]) and (out[2:] == -7).all()


def test_attend_offsets_past_32_bits():
    """Pages far enough apart that byte and value offsets pass 2^32."""
    page, kv, dim = 16, 2, 128
    base = torch.empty(3, 1 << 31, dtype=BF, device="cuda")     # 4 GiB between pages, in bytes
    k = base[:, :page * kv * dim].view(3, page, kv, dim)
    v = base[:, 1 << 30:(1 << 30) + page * kv * dim].view(3, page, kv, dim)
    b = Batch(15, [2], [30], 4, kv, dim, page, extra=0)
    b.k, b.v = b.k[:3], b.v[:3]
    b.table = torch.tensor([[2, 0]], dtype=torch.int32)
    b.kd, b.vd = k, v
    k.copy_(b.k)
    v.copy_(b.v)
    b.cache = sv.PagedCache(k, v)
    b.check()


def test_attend_repeats_and_streams_agree():
    b = Batch(16, [3, 1, 8], [2000, 5, 700], 8, 2, 128, 16, F8).device()
    out, lse, _ = b.attend()
    side = torch.cuda.Stream()
    for stream in (None, side, None):
        o, e, _ = b.attend(stream=stream)
        assert torch.equal(o, out) and torch.equal(e, lse)


def test_append_attend_replay_from_a_graph():
    """A captured append and attend follow the buffers' contents at every replay."""
    b = Batch(17, [2, 4], [100, 33], 8, 2, 128, 16).device()
    cap = 8
    req = torch.tensor([0, 0, 1, 1, 1, 1, -1, -1], dtype=torch.int32, device="cuda")
    pos = torch.tensor([0, 1, 0, 1, 2, 3, -1, -1], dtype=torch.int32, device="cuda")
    nk, nv = [torch.randn(cap, 2, 128, device="cuda").to(BF) for _ in range(2)]
    q, table, cu, ctx = b.q.cuda(), b.table.cuda(), b.cu.cuda(), b.ctx.cuda()
    out, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], device="cuda")
    ws = b.ws()

    def step():
        sv.sv_cache_append(b.cache, table, nk, nv, req, pos, ctx)
        sv.sv_cache_attend(b.cache, table, q, cu, ctx, b.k_max, b.scale, out, ws, lse)

    step()
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        step()
    for i in range(4):
        nk.normal_()
        nv.normal_()
        q.normal_()
        ctx.copy_(torch.tensor([100 - 7 * i, 33 + 11 * i], dtype=torch.int32))
        out.fill_(-3)
        graph.replay()
        torch.cuda.synchronize()
        got, got_lse = out.clone(), lse.clone()
        out.fill_(-3)
        step()
        torch.cuda.synchronize()
        assert torch.equal(got, out) and torch.equal(got_lse, lse)


# -------------------------------------------------------------------- append

@pytest.mark.parametrize("dtype", [BF, F8])
@pytest.mark.parametrize("dim,kv,page,layout", [(64, 1, 1, "nhd"), (128, 8, 16, "nhd"),
                                                (256, 3, 7, "hnd"), (128, 2, 64, "hnd")])
def test_append_matches_oracle(dtype, dim, kv, page, layout):
    rows = [1, 4, 0, 3]
    b = Batch(20, rows, [0, 13, 5, 63], kv, kv, dim, page, dtype, layout=layout).device()
    g = torch.Generator().manual_seed(3)
    cap = 16
    req = torch.full((cap,), -1, dtype=torch.int32)
    pos = torch.full((cap,), -1, dtype=torch.int32)
    pairs = [(r, j) for r, m in enumerate(rows) for j in range(m)]
    for i, (r, j) in enumerate(pairs):
        req[i], pos[i] = r, j
    new = [(torch.randn(cap, kv, dim, generator=g) * s).to(BF) for s in (1.0, 150.0)]
    new[1][0, 0, :3] = torch.tensor([float("nan"), float("inf"), -float("inf")])
    want = [cache_append(values(c), b.table.numpy(), x.float().numpy(), req.numpy(), pos.numpy(),
                         b.ctx.numpy(), None if b.scales is None else s.numpy())
            for c, x, s in zip((b.k, b.v), new, b.scales or (None, None))]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    sv.sv_cache_append(b.cache, b.table.cuda(), new[0].cuda(), new[1].cuda(), req.cuda(),
                       pos.cuda(), b.ctx.cuda(), err)
    torch.cuda.synchronize()
    assert int(err) == 0
    np.testing.assert_array_equal(values(b.kd), want[0])
    np.testing.assert_array_equal(values(b.vd), want[1])


def test_append_rounds_every_tie_and_border():
    """Values on and between all e4m3 values, through a scale of 1."""
    codes = torch.arange(256, dtype=torch.uint8).view(F8).double()
    fin = codes[torch.isfinite(codes)].unique()
    x = torch.cat([fin, (fin[1:] + fin[:-1]) / 2, torch.tensor([1e9, -1e9, 464.0, 2.0 ** -10])])
    x = x.to(BF)    # every tie has at most 5 significant bits: exact in bf16
    x = torch.cat([x, torch.zeros(-len(x) % 64, dtype=BF)]).view(-1, 1, 64)
    k = torch.zeros(len(x), 1, 1, 64, dtype=F8, device="cuda")
    v = torch.zeros_like(k)
    table = torch.arange(len(x), dtype=torch.int32, device="cuda")[:, None].contiguous()
    i32 = dict(dtype=torch.int32, device="cuda")
    sv.sv_cache_append(sv.PagedCache(k, v), table, x.cuda(), (-x).cuda(),
                       torch.arange(len(x), **i32), torch.zeros(len(x), **i32),
                       torch.zeros(len(x), **i32))
    torch.cuda.synchronize()
    np.testing.assert_array_equal(values(k)[:, 0], e4m3_round(values(x)))
    np.testing.assert_array_equal(values(v)[:, 0], e4m3_round(-values(x)))


def test_append_faults_leave_the_cache_alone():
    b = Batch(21, [1, 1, 1], [4, 4, 4], 2, 2, 64, 16).device()
    b.table[1, 0] = b.k.shape[0]
    new = torch.ones(3, 2, 64, dtype=BF, device="cuda")
    before = b.kd.clone(), b.vd.clone()
    cases = [([3, -2, 0], [0, 0, -1], [4, 4, 4], sv.SV_DEV_BAD_CU_ROWS),
             ([0, 0, 2], [0, 0, 0], [-1, 4, b.table.shape[1] * 16], sv.SV_DEV_BAD_CTX),
             ([1, -1, -1], [0, -1, -1], [4, 4, 4], sv.SV_DEV_BAD_PAGE)]
    for req, pos, ctx, bit in cases:
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        t = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        sv.sv_cache_append(b.cache, b.table.cuda(), new, new, t(req), t(pos), t(ctx), err)
        torch.cuda.synchronize()
        assert int(err) == bit
        assert torch.equal(b.kd, before[0]) and torch.equal(b.vd, before[1])


@pytest.mark.parametrize("n,heads,kv,dim,dtype", [(200, 16, 8, 64, F8), (257, 8, 8, 64, BF),
                                                  (40, 32, 32, 128, BF)])
def test_attend_many_workgroups(n, heads, kv, dim, dtype):
    """More workgroups than the CUs take at once: requests served longest first
    (up to 256 of them), heads that share cache lines kept together."""
    rng = np.random.default_rng(n)
    rows = [int(x) for x in rng.integers(0, 3, n)]
    ctx = [int(x) for x in rng.integers(0, 60, n)]
    ctx[3], ctx[n // 2] = 700, 700
    Batch(30 + n, rows, ctx, heads, kv, dim, 16, dtype, k_max=2).device().check()


@pytest.mark.parametrize("dtype", [BF, F8])
def test_attend_requests_that_share_pages(dtype):
    """A common prefix: the requests' tables hold the same pages, and one page twice."""
    b = Batch(41, [2, 1, 3], [40, 63, 20], 8, 2, 128, 16, dtype)
    b.table[1, :2] = b.table[0, :2]
    b.table[2, :2] = b.table[0, :2]
    b.table[2, 0] = b.table[2, 1]
    b.device().check()


def test_attend_two_calls_at_once():
    """Two streams, each with a workspace of its own, their launches interleaved."""
    b = Batch(42, [2, 1], [9000, 4000], 8, 2, 128, 16).device()
    q, table, cu, ctx = b.q.cuda(), b.table.cuda(), b.cu.cuda(), b.ctx.cuda()
    want, want_lse, _ = b.attend()
    streams, outs = [torch.cuda.Stream() for _ in range(2)], []
    torch.cuda.synchronize()
    for i in range(8):
        outs.append((torch.zeros_like(q), torch.zeros(q.shape[:2], device="cuda"), b.ws()))
    torch.cuda.synchronize()
    for i, (out, lse, ws) in enumerate(outs):
        sv.sv_cache_attend(b.cache, table, q, cu, ctx, b.k_max, b.scale, out, ws, lse,
                           stream=streams[i % 2])
    torch.cuda.synchronize()
    rows = int(b.cu[-1])
    for out, lse, _ in outs:
        assert torch.equal(out[:rows], want[:rows]) and torch.equal(lse[:rows], want_lse[:rows])


def test_attend_head_groups_wider_than_a_block():
    """More query slots than one workgroup takes, at 256 dims and at 64."""
    Batch(43, [5, 1], [70, 3], 24, 1, 256, 16).device().check()
    Batch(44, [9, 2], [70, 3], 24, 1, 64, 16, F8).device().check()
