"""Histories and adjusted logits on the GPU against the fp64 oracle.

Tolerance, from the arithmetic: a quotient or product, the product with the
count, two differences and the bias, each rounded to fp32 (2^-24 of a value not
above the sum of sizes the oracle returns), then the row type's own rounding
(bf16 2^-8 of the result, fp32 none beyond the last difference).
"""

import numpy as np
import pytest
import torch

import adaptive_draft_verification_amd as sv
from oracle.logits import (DEV_BAD_CU_ROWS, DEV_BAD_PARAM, DEV_BAD_SLOT, DEV_BAD_TOKEN, adjust_row,
                           bits_of, history_add)

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True, scope="module")
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def dev(a, dtype=None):
    return torch.as_tensor(np.asarray(a)).to("cuda", dtype)


def listed(h, slot):
    """The slot's listed ids, sorted."""
    n = int(h.n_seen[slot])
    return sorted(h.seen[slot, :min(n, h.seen.shape[1])].tolist()), n


# ------------------------------------------------------------------- history

@pytest.mark.parametrize("n,width,vocab", [(1, 1, 1), (1, 64, 7), (3, 65, 1000), (5, 257, 50),
                                           (2, 1000, 129280), (70, 300, 333)])
@pytest.mark.parametrize("cap", ["all", "few", 0])
def test_history(n, width, vocab, cap):
    rng = np.random.default_rng(n * width)
    slots = rng.permutation(n + 2)[:n]
    cap = {"all": vocab, "few": max(1, min(vocab, width) // 3), 0: 0}[cap]
    h = sv.TokenHistory.empty(n + 2, vocab, cap)
    want = np.zeros((n + 2, vocab), np.int32)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for in_prompt in (True, False, False, True):
        toks = rng.integers(-1, vocab, (n, width)).astype(np.int32)
        toks[:, width // 2:] = np.minimum(toks[:, width // 2:], 3)
        sv.sv_history_add(h, dev(slots, torch.int32), dev(toks), in_prompt, err)
        assert history_add(want, slots, toks, in_prompt) == 0
    np.testing.assert_array_equal(h.counts.cpu().numpy(), want)
    for s in range(n + 2):
        ids, count = listed(h, s)
        true = np.flatnonzero(want[s]).tolist()
        assert count == len(true)
        assert len(set(ids)) == len(ids) == min(count, cap) and set(ids) <= set(true)
    gone = slots[::2]
    sv.sv_history_clear(h, dev(gone, torch.int32), err)
    want[gone] = 0
    np.testing.assert_array_equal(h.counts.cpu().numpy(), want)
    assert (h.n_seen.cpu().numpy() == (want > 0).sum(-1)).all() and int(err) == 0


def test_history_of_one_slot_in_many_rows():
    """Rows of one slot in one call add up, and each id is listed once."""
    rng = np.random.default_rng(0)
    h = sv.TokenHistory.empty(2, 500)
    toks = rng.integers(0, 40, (64, 100)).astype(np.int32)
    slots = np.ones(64, np.int64)
    sv.sv_history_add(h, dev(slots, torch.int32), dev(toks))
    want = np.zeros((2, 500), np.int32)
    history_add(want, slots, toks, False)
    np.testing.assert_array_equal(h.counts.cpu().numpy(), want)
    ids, count = listed(h, 1)
    assert ids == np.flatnonzero(want[1]).tolist() and count == len(ids)
    # the same slot named twice is cleared
    sv.sv_history_clear(h, dev([1, 1], torch.int32))
    assert int(h.counts.abs().sum()) == 0 and h.n_seen.tolist() == [0, 0]


def test_history_errors_and_strided_rows():
    h = sv.TokenHistory.empty(2, 10)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    toks = dev([[1, 10, -2, 2, 9, 9], [3, 3, 3, 3, 9, 9], [4, 4, 4, 4, 9, 9]], torch.int32)
    sv.sv_history_add(h, dev([1, 2, -1], torch.int32), toks[:, :4], False, err)
    assert int(err) == DEV_BAD_TOKEN | DEV_BAD_SLOT
    assert h.counts.tolist() == [[0] * 10, [0, 2, 2] + [0] * 7]
    err.zero_()
    sv.sv_history_clear(h, dev([5, 1], torch.int32), err)
    assert int(err) == DEV_BAD_SLOT and int(h.counts.sum()) == 0


# -------------------------------------------------------------------- adjust

class Case:
    """A packed batch with histories, drafts, penalties, biases and masks."""

    def __init__(self, seed, n, k, vocab, dtype, said=60, bias=5, masks=True, cap=None, pad=0):
        rng = np.random.default_rng(seed)
        self.n, self.k, self.V, self.dtype = n, k, vocab, dtype
        rows = rng.integers(1, k + 2, n)
        cap_rows = n * (k + 1)
        self.req = np.full(cap_rows, -1, np.int32)
        self.pos = np.full(cap_rows, -1, np.int32)
        self.req[:rows.sum()] = np.repeat(np.arange(n), rows)
        self.pos[:rows.sum()] = np.concatenate([np.arange(x) for x in rows])
        z = torch.from_numpy((3 * rng.standard_normal((cap_rows, vocab + pad))).astype(np.float32))
        self.z = z.to(dtype).cuda()[:, :vocab]
        self.slots = rng.permutation(n + 1)[:n].astype(np.int32)
        self.counts = np.zeros((n + 1, vocab), np.int32)
        self.h = sv.TokenHistory.empty(n + 1, vocab, cap)
        for in_prompt in (True, False):
            toks = (vocab * rng.random((n, said)) ** 2).astype(np.int32)
            history_add(self.counts, self.slots, toks, in_prompt)
            sv.sv_history_add(self.h, dev(self.slots), dev(toks), in_prompt)
        # drafts: some said before, some twice in a row, some new
        self.drafts = rng.integers(0, vocab, (n, k)).astype(np.int32)
        if k > 1:
            self.drafts[::2, 1] = self.drafts[::2, 0]
            self.drafts[:, k - 1] = toks[:, 0]
        self.pen = np.stack([1 + 0.5 * rng.random(n), rng.standard_normal(n),
                             rng.standard_normal(n)]).astype(np.float32)
        self.bias = []
        for r in range(n):
            m = int(rng.integers(0, min(bias, vocab) + 1))
            ids = rng.choice(vocab, m, replace=False)
            if m > 1:  # one that was said, one that is drafted
                ids[0] = toks[r, 0]
                ids[1] = self.drafts[r, 0] if k else ids[1]
            ids = np.unique(ids)
            self.bias.append(list(zip(ids.tolist(), (2 * rng.standard_normal(len(ids))))))
        if self.bias[0]:
            self.bias[0][-1] = (self.bias[0][-1][0], -np.inf)
        self.allowed, self.row_mask = [], np.full(cap_rows, -1, np.int32)
        if masks:
            for i in range(0, int(rows.sum()), 2):
                self.row_mask[i] = len(self.allowed)
                share = (0.0, 1.0, 0.5, 0.05)[(i // 2) % 4]
                self.allowed.append(rng.random(vocab) < share)

    def args(self):
        start = np.cumsum([0] + [len(b) for b in self.bias]).astype(np.int32)
        flat = [e for b in self.bias for e in b]
        bias = sv.Bias(dev(start), dev([i for i, _ in flat], torch.int32),
                       dev([v for _, v in flat], F32)) if flat else None
        mask = None
        if self.allowed:
            mask = sv.TokenMask(dev(np.stack([bits_of(a) for a in self.allowed])),
                                dev(self.row_mask))
        return dict(history=self.h, slots=dev(self.slots),
                    penalties=sv.Penalties(*(dev(p) for p in self.pen)),
                    draft_tokens=dev(self.drafts), bias=bias, mask=mask)

    def expect(self):
        z = self.z.double().cpu().numpy()
        want, size = np.full(z.shape, np.nan), np.zeros(z.shape)
        for i, (r, j) in enumerate(zip(self.req, self.pos)):
            if r < 0:
                continue
            allowed = self.allowed[self.row_mask[i]] if self.row_mask[i] >= 0 else None
            want[i], size[i] = adjust_row(z[i], self.counts[self.slots[r]], self.drafts[r, :j],
                                          *self.pen[:, r], self.bias[r], allowed)
        return want, size

    def compare(self, out):
        want, size = self.expect()
        got = out.double().cpu().numpy()
        live = self.req >= 0
        got, want, size = got[live], want[live], size[live]
        same = np.isinf(want) | np.isnan(want)
        np.testing.assert_array_equal(got[same], want[same])
        half = 2.0 ** -8 if self.dtype == BF else 0.0
        tol = half * np.abs(want) + (1 + half) * 6 * 2.0 ** -24 * size
        ok = np.abs(got - want) <= tol
        assert ok[~same].all(), np.max(np.abs(got - want)[~same] / tol[~same])

    def check(self):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.full_like(self.z, 7.0)
        sv.sv_adjust_logits(self.z, out, dev(self.req), dev(self.pos), dev_error=err, **self.args())
        assert int(err) == 0
        self.compare(out)
        dead = self.req < 0
        assert bool((out[dev(dead)] == 7.0).all())
        # in place: the same values
        inplace = self.z.clone()
        sv.sv_adjust_logits(inplace, inplace, dev(self.req), dev(self.pos), dev_error=err,
                            **self.args())
        live = dev(~dead)
        assert torch.equal(inplace[live].view(torch.int16 if self.dtype == BF else torch.int32),
                           out[live].view(torch.int16 if self.dtype == BF else torch.int32))
        assert torch.equal(inplace[dev(dead)], self.z[dev(dead)]) and int(err) == 0
        return out


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,k,vocab", [(1, 0, 1), (1, 0, 31), (2, 3, 33), (3, 7, 1000), (4, 2, 4097),
                                       (2, 1, 32003), (40, 3, 517), (1, 64, 600)])
def test_adjust(dtype, n, k, vocab):
    Case(n + vocab, n, k, vocab, dtype).check()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_adjust_large_rows(dtype):
    Case(5, 3, 2, 256000, dtype, said=3000, bias=300).check()


def test_adjust_more_rows_than_parts():
    """Above 2048 rows a row is one workgroup's."""
    Case(6, 700, 3, 5000, BF, said=20, bias=2).check()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("pad", [1, 3, 8])
def test_adjust_rows_apart(dtype, pad):
    """Rows that start at any multiple of the type's size, in a wider matrix that stays as it is."""
    c = Case(7, 4, 3, 2051, dtype, pad=pad)
    wide = torch.full((c.z.shape[0], 2051 + pad), 9.0, dtype=dtype, device="cuda")
    sv.sv_adjust_logits(c.z, wide[:, :2051], dev(c.req), dev(c.pos), **c.args())
    c.compare(wide[:, :2051])
    assert bool((wide[:, 2051:] == 9.0).all())


@pytest.mark.parametrize("cap", [0, 1, 40])
def test_adjust_lists_that_do_not_hold_every_id(cap):
    Case(8, 5, 3, 700, F32, said=100, cap=cap).check()


@pytest.mark.parametrize("without", ["history", "penalties", "bias", "mask", "draft_tokens"])
def test_adjust_without(without):
    c = Case(9, 6, 0 if without == "draft_tokens" else 3, 900, F32)
    args = c.args()
    args[without] = None
    if without == "history":
        c.counts[:] = 0
    elif without == "penalties":
        c.pen = np.stack([np.ones(6), np.zeros(6), np.zeros(6)]).astype(np.float32)
        args["draft_tokens"] = None
    elif without == "bias":
        c.bias = [[]] * 6
    elif without == "mask":
        c.row_mask[:] = -1
    out = torch.zeros_like(c.z)
    sv.sv_adjust_logits(c.z, out, dev(c.req), dev(c.pos), n_req=6, **args)
    c.compare(out)
    if without == "penalties":  # drafts without penalties change nothing
        again = torch.zeros_like(c.z)
        args["draft_tokens"] = dev(c.drafts)
        sv.sv_adjust_logits(c.z, again, dev(c.req), dev(c.pos), **args)
        assert torch.equal(out, again)


def test_adjust_plain_decoding_rows():
    """No maps: row i is request i; mask i where no row_mask is given; no penalty arrays."""
    rng = np.random.default_rng(3)
    z = torch.randn(4, 77, device="cuda")
    allowed = rng.random((4, 77)) < 0.5
    out = torch.empty_like(z)
    sv.sv_adjust_logits(z, out, None, None, mask=sv.TokenMask(dev(np.stack([bits_of(a) for a in allowed]))),
                        penalties=sv.Penalties())
    want = torch.where(dev(allowed), z, -torch.inf)
    assert torch.equal(out, want)
    # nothing to adjust: a copy; in place: nothing
    sv.sv_adjust_logits(z, out, None, None)
    assert torch.equal(out, z)
    sv.sv_adjust_logits(out, out, None, None)
    assert torch.equal(out, z)


def test_adjust_values_that_are_not_finite():
    z = torch.tensor([[float("inf"), -float("inf"), float("nan"), 1.0, float("nan"), float("nan")]],
                     device="cuda")
    h = sv.TokenHistory.empty(1, 6)
    sv.sv_history_add(h, None, dev([[0, 1, 2]], torch.int32))
    out = torch.empty_like(z)
    allowed = np.array([1, 1, 1, 1, 1, 0])
    sv.sv_adjust_logits(z, out, None, None, h, None,
                        sv.Penalties(dev([1.5], F32), dev([0.5], F32), dev([0.5], F32)),
                        bias=sv.Bias(dev([0, 1], torch.int32), dev([3], torch.int32), dev([-np.inf], F32)),
                        mask=sv.TokenMask(dev(bits_of(allowed)[None])))
    got = out[0].tolist()
    assert got[0] == np.inf and got[1] == -np.inf and np.isnan(got[2]) and got[3] == -np.inf
    assert np.isnan(got[4]) and got[5] == -np.inf


BAD = [("req", 3, DEV_BAD_CU_ROWS), ("req", -2, DEV_BAD_CU_ROWS), ("pos", 4, DEV_BAD_CU_ROWS),
       ("pos", -1, DEV_BAD_CU_ROWS), ("slot", 4, DEV_BAD_SLOT), ("slot", -1, DEV_BAD_SLOT),
       ("draft", 500, DEV_BAD_TOKEN), ("draft", -1, DEV_BAD_TOKEN), ("rho", 0.0, DEV_BAD_PARAM),
       ("rho", -1.0, DEV_BAD_PARAM), ("rho", np.inf, DEV_BAD_PARAM), ("rho", np.nan, DEV_BAD_PARAM),
       ("phi", np.nan, DEV_BAD_PARAM), ("pi", np.inf, DEV_BAD_PARAM), ("bias_id", 500, DEV_BAD_TOKEN),
       ("bias_id", -1, DEV_BAD_TOKEN), ("bias_twice", 0, DEV_BAD_TOKEN), ("bias", np.nan, DEV_BAD_PARAM),
       ("bias", np.inf, DEV_BAD_PARAM), ("start", 99, DEV_BAD_PARAM), ("mask", 2, DEV_BAD_PARAM),
       ("mask", -2, DEV_BAD_PARAM)]


@pytest.mark.parametrize("what,value,bit", BAD)
@pytest.mark.parametrize("inplace", [False, True])
def test_adjust_faulty_rows_become_nan(what, value, bit, inplace):
    """Request 1 (rows 2 .. 5) or one of its rows is faulty: those rows are NaN, the rest fine."""
    V, k = 500, 3
    z = torch.randn(8, V, device="cuda")
    req, pos = [0, 0, 1, 1, 1, 1, 2, -1], [0, 1, 0, 1, 2, 3, 0, -1]
    slots, pen = [0, 1, 2], [[1.2] * 3, [0.1] * 3, [0.2] * 3]
    drafts, start = [[5, 6, 7]] * 3, [0, 1, 3, 4]
    drafts = [list(d) for d in drafts]
    ids, values, row_mask = [4, 8, 9, 4], [1.0] * 4, [-1, 0, 1, 0, 1, 0, -1, -1]
    bad = [2, 3, 4, 5]
    if what in ("req", "pos"):
        (req if what == "req" else pos)[4] = value
        bad = [4]
    elif what == "slot":
        slots[1] = value
    elif what == "draft":
        drafts[1][1] = value
        bad = [4, 5]  # the rows behind it
    elif what in ("rho", "phi", "pi"):
        pen[("rho", "phi", "pi").index(what)][1] = value
    elif what == "bias_id":
        ids[1 if value < 0 else 2] = value
    elif what == "bias_twice":
        ids[2] = ids[1]
    elif what == "bias":
        values[2] = value
    elif what == "start":
        start[2] = value
        bad = [2, 3, 4, 5, 6]  # request 2 begins there
    elif what == "mask":
        row_mask[3] = value
        bad = [3]
    h = sv.TokenHistory.empty(4, V)
    sv.sv_history_add(h, None, torch.arange(12, dtype=torch.int32, device="cuda").view(4, 3))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    bits = dev(np.stack([bits_of(np.arange(V) % 3 == i) for i in range(2)]))
    src = z.clone()
    out = src if inplace else torch.full_like(z, 7.0)
    sv.sv_adjust_logits(src, out, dev(req, torch.int32), dev(pos, torch.int32), h,
                        dev(slots, torch.int32), sv.Penalties(*(dev(p, F32) for p in pen)),
                        dev(drafts, torch.int32),
                        sv.Bias(dev(start, torch.int32), dev(ids, torch.int32), dev(values, F32)),
                        sv.TokenMask(bits, dev(row_mask, torch.int32)), err)
    assert int(err) == bit
    nan = torch.isnan(out).all(-1).tolist()
    assert [i for i in range(8) if nan[i]] == bad
    assert not torch.isnan(out[[i for i in range(8) if i not in bad]]).any()
    assert torch.equal(out[7], z[7] if inplace else torch.full_like(z[7], 7.0))
    # and a draw from them is refused
    tok = torch.empty(8, dtype=torch.int32, device="cuda")
    sv.sv_sample(out, torch.full((8,), 0.5, device="cuda"), None, tok)
    assert [i for i in range(8) if int(tok[i]) < 0] == bad


def test_adjust_on_another_stream_and_in_a_graph():
    c = Case(11, 6, 3, 3001, BF)
    args, req, pos = c.args(), dev(c.req), dev(c.pos)
    out = torch.zeros_like(c.z)
    sv.sv_adjust_logits(c.z, out, req, pos, **args)
    side, other = torch.cuda.Stream(), torch.zeros_like(out)
    side.wait_stream(torch.cuda.current_stream())
    sv.sv_adjust_logits(c.z, other, req, pos, stream=side, **args)
    side.synchronize()
    assert torch.equal(out, other)
    # captured: what was said is added, then the rows adjusted; replayed over new inputs
    toks = torch.full((6, 4), -1, dtype=torch.int32, device="cuda")
    slots, z = dev(c.slots), c.z.contiguous().clone()
    graph = torch.cuda.CUDAGraph()
    got = torch.zeros_like(z)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        sv.sv_history_add(c.h, slots, toks)
        sv.sv_adjust_logits(z, got, req, pos, **args)
    rng = np.random.default_rng(1)
    for _ in range(4):
        new = rng.integers(-1, 3001, (6, 4)).astype(np.int32)
        toks.copy_(dev(new))
        z.copy_(torch.randn(z.shape, device="cuda") * 2)
        graph.replay()
        torch.cuda.synchronize()
        history_add(c.counts, c.slots, new, False)
        c.z = z
        c.compare(got)
        np.testing.assert_array_equal(c.h.counts.cpu().numpy(), c.counts)


def test_verified_tokens_go_into_the_history_as_they_are():
    """sv_verify's emitted ids (-1 behind them, or everywhere for a faulty request)."""
    h = sv.TokenHistory.empty(3, 50)
    emitted = dev([[4, 4, -1, -1], [9, -1, -1, -1], [-1, -1, -1, -1]], torch.int32)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    sv.sv_history_add(h, None, emitted, dev_error=err)
    assert h.counts[0, 4] == 4 and h.counts[1, 9] == 2 and int(h.counts.sum()) == 6 and int(err) == 0
