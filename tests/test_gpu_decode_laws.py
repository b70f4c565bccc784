"""Decode steps with the calls in a run: a token history that penalises what prompts and
answers said, biases and grammar masks on the drafter's and on the target's logits, the packed
rows attending to a cache of latent vectors or to one whose requests share a prefix, drafts
drawn and verified under the adjusted logits' truncated laws, the accepted tokens added to the
history.  Every stage against its oracle, on the device's own inputs of that stage; the
tolerances are the stages' own."""

import numpy as np
import pytest
import torch

import adaptive_draft_verification_amd as sv
from oracle.cache import cache_append, cache_attend
from oracle.latent import latent_append, latent_attend
from oracle.logits import adjust_row, bits_of
from oracle.truncate import sample_row, verify_truncated

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(autouse=True, scope="module")
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def values(t):
    return t.cpu().float().double().numpy()


class Latent:
    """One latent vector a position, read in the absorbed form."""
    heads, rank = 4, 256
    q_dim, out_dim = 320, 256
    scale = 0.07

    def __init__(self, pages, page, g):
        self.kv = torch.randn(pages, page, 320, generator=g).cuda().to(BF)
        self.cache = sv.LatentCache(self.kv, self.rank)

    def append(self, x, table, req, pos, ctx, err):
        rows = x[:, :320].to(BF)
        want = latent_append(values(self.kv), table.cpu().numpy(), values(rows)[:, :256],
                             values(rows)[:, 256:], req.tolist(), pos.tolist(), ctx.tolist())
        sv.sv_latent_append(self.cache, table, rows[:, :256], rows[:, 256:], req, pos, ctx, err)
        np.testing.assert_array_equal(values(self.kv), want)

    def attend(self, q, table, cu, ctx, k, err):
        out = torch.zeros(*q.shape[:2], self.rank, dtype=BF, device="cuda")
        ws = torch.empty(max(16, sv.sv_latent_attend_workspace_bytes(
            len(ctx), k, self.heads, self.rank, table.shape[1], self.kv.shape[1])),
            dtype=torch.uint8, device="cuda")
        sv.sv_latent_attend(self.cache, table, q, cu, ctx, k, self.scale, out, ws, None, err)
        return out, latent_attend(values(q), values(self.kv), self.rank, table.cpu().numpy(),
                                  cu.tolist(), ctx.tolist(), self.scale)


class Shared:
    """Requests 0 .. 3 share their first positions, the others nothing."""
    heads, kv, dim = 4, 2, 64
    q_dim = out_dim = 64
    scale = 0.125

    def __init__(self, pages, page, g):
        self.k, self.v = (torch.randn(pages, page, self.kv, self.dim, generator=g).cuda().to(BF)
                          for _ in range(2))
        self.cache = sv.PagedCache(self.k, self.v)
        self.start = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
        self.prefix = torch.tensor([2 * page], dtype=torch.int32, device="cuda")

    def append(self, x, table, req, pos, ctx, err):
        k, v = (x[:, i * 128:(i + 1) * 128].reshape(-1, 2, 64).to(BF) for i in range(2))
        want = [cache_append(values(c), table.cpu().numpy(), values(new), req.tolist(), pos.tolist(),
                             ctx.tolist()) for c, new in ((self.k, k), (self.v, v))]
        sv.sv_cache_append(self.cache, table, k, v, req, pos, ctx, err)
        np.testing.assert_array_equal(values(self.k), want[0])
        np.testing.assert_array_equal(values(self.v), want[1])

    def attend(self, q, table, cu, ctx, k, err):
        out = torch.zeros_like(q)
        ws = torch.empty(sv.sv_cache_attend_shared_workspace_bytes(
            len(ctx), 1, k, self.heads, self.kv, self.dim, table.shape[1], self.k.shape[1]),
            dtype=torch.uint8, device="cuda")
        sv.sv_cache_attend_shared(self.cache, table, q, cu, ctx, self.start, self.prefix, k,
                                  self.scale, out, ws, None, err)
        return out, cache_attend(values(q), values(self.k), values(self.v), table.cpu().numpy(),
                                 cu.tolist(), ctx.tolist(), self.scale)


@pytest.mark.parametrize("kind", [Latent, Shared])
def test_decode_steps_under_adjusted_laws(kind):
    g = torch.Generator().manual_seed(3)
    n, k, V, page, pages = 6, 3, 331, 16, 40
    dev = dict(device="cuda")
    rn = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    model = kind(pages, page, g)
    H = model.heads
    emb, wq = rn(V, 320), rn(320, H * model.q_dim) / 18
    head = rn(H * model.out_dim, V) / (H * model.out_dim) ** 0.5 * 8
    table = torch.randperm(pages, generator=g)[:n * 6].int().view(n, 6).cuda()
    if kind is Shared:
        table[1:4, :2] = table[0, :2]
    ctx = torch.tensor([32, 35, 47, 40, 1, 20], dtype=torch.int32, **dev)
    settings = [(0.0, 0, 1.0, 0.0), (0.8, 40, 0.95, 0.0), (1.0, 0, 1.0, 0.0), (0.7, 0, 0.9, 0.0),
                (1.0, 0, 1.0, 0.05), (1.2, 7, 0.8, 0.01)]
    t, kk, p, s = (torch.tensor(x).cuda() for x in zip(*settings))
    law = sv.Sampling(t.float(), kk.int(), p.float(), s.float())
    # every request's slot, its penalties, its biases; half of the requests under a grammar
    slots = torch.tensor([5, 0, 7, 2, 3, 6], dtype=torch.int32, **dev)
    hist = sv.TokenHistory(torch.zeros(8, V, dtype=torch.int32, **dev),  # as they have to start
                           torch.zeros(8, 64, dtype=torch.int32, **dev),
                           torch.zeros(8, dtype=torch.int32, **dev))
    law_of = [(1.3, 0.2, 0.1), (1.0, 0.0, 0.0), (0.8, 0.5, 0.0), (1.1, 0.0, 0.7), (2.0, 0.1, 0.1),
              (1.0, -0.3, 0.0)]
    pen = sv.Penalties(*(torch.tensor(x).cuda() for x in zip(*law_of)))
    bias_of = [[(3, 1.5), (17, -2.0)], [], [(0, -float("inf"))], [], [(V - 1, 4.0)], [(5, 0.25)]]
    flat = [b for x in bias_of for b in x]
    bias = sv.Bias(torch.tensor(np.cumsum([0] + [len(x) for x in bias_of]), dtype=torch.int32, **dev),
                   torch.tensor([b[0] for b in flat], dtype=torch.int32, **dev),
                   torch.tensor([b[1] for b in flat], **dev))
    allowed = (torch.rand(3, V, generator=g) < 0.6).numpy()
    bits = torch.from_numpy(np.stack([bits_of(a) for a in allowed])).cuda()
    mask_of = [0, -1, 1, -1, 2, -1]
    err = torch.zeros(1, dtype=torch.int32, **dev)

    sv.sv_history_clear(hist, torch.arange(8, dtype=torch.int32, **dev), err)
    prompt = torch.randint(0, V, (n, 9), generator=g).int()
    prompt[2, 4:] = -1
    sv.sv_history_add(hist, slots, prompt.cuda(), True, err)
    held = np.zeros((8, V), np.int64)
    for r in range(n):
        for x in prompt[r].tolist():
            if x >= 0:
                held[slots[r], x] |= 1

    def adjusted(logits, req, pos, drafts):
        """On the device, held against the oracle's rows."""
        rows = len(logits)
        masks = torch.tensor([mask_of[r] if r >= 0 else -1 for r in req.tolist()],
                             dtype=torch.int32, **dev)
        out = torch.full_like(logits, -7.0)
        sv.sv_adjust_logits(logits, out, req, pos, hist, slots, pen, drafts, bias,
                            sv.TokenMask(bits, masks), err)
        for i in range(rows):
            r, j = int(req[i]), int(pos[i])
            if r < 0:
                assert (out[i] == -7).all()
                continue
            want, size = adjust_row(values(logits[i]), held[int(slots[r])],
                                    drafts[r, :j].tolist(), *law_of[r], bias=bias_of[r],
                                    allowed=None if mask_of[r] < 0 else allowed[mask_of[r]])
            got = values(out[i])
            np.testing.assert_array_equal(np.isneginf(got), np.isneginf(want))
            f = np.isfinite(want)  # what a mask or a bias of -inf leaves
            # five fp32 roundings at most of what is added up
            assert (np.abs(got[f] - want[f]) <= 5 * 2.0 ** -24 * size[f]).all()
        return out

    last = torch.randint(0, V, (n,), generator=g).int().cuda()
    for step in range(3):
        # the drafter, a position at a time: what it drafted before counts as said
        toks = torch.full((n, k), -1, dtype=torch.int32, **dev)
        u, v = torch.empty(n, k, **dev), torch.empty(n, k, **dev)
        sv.sv_philox_uniforms(77, step, u, v)
        each = torch.arange(n, dtype=torch.int32, **dev)
        laws = torch.empty(n, k, V, **dev)
        for j in range(k):
            laws[:, j] = adjusted((rn(n, V) * 2).contiguous(), each, torch.full_like(each, j),
                                  toks.clamp(min=0))
            new = torch.empty(n, dtype=torch.int32, **dev)
            sv.sv_sample(laws[:, j].contiguous(), u[:, j].contiguous(), law, new, None, None, err)
            for r in range(n):
                want = sample_row(laws[r, j].cpu().numpy(), float(u[r, j]), *settings[r])
                assert int(new[r]) == want[0]
            toks[:, j] = new
        kept = torch.tensor([3, 2, 3, 0, 1, 3], dtype=torch.int32, **dev)
        pk = sv.pack_varlen(kept, last, toks)
        cu, req, pos = pk["cu_rows"], pk["row_req"], pk["row_pos"]
        rows = int(cu[-1])

        x = emb[pk["packed_tokens"].clamp(min=0).long()]
        model.append(x, table, req, pos, ctx, err)
        q = (x @ wq).view(-1, H, model.q_dim).to(BF)
        out, (o, _, spread) = model.attend(q, table, cu, ctx, k, err)
        diff = np.abs(values(out)[:rows] - o[:rows])
        # weights and output rounded to bf16 (2^-8 each), scores in fp32
        assert (diff <= 2.0 ** -8 * np.abs(o[:rows]) + 1.01 * 2.0 ** -8 * spread[:rows]).all()
        assert (out[rows:] == 0).all()

        raw = (out.float().view(len(q), -1) @ head).contiguous()
        target = adjusted(raw, req, pos, toks)
        tokens = torch.empty(n, k + 1, dtype=torch.int32, **dev)
        accepted = torch.empty(n, dtype=torch.int32, **dev)
        ws = torch.empty(sv.sv_verify_truncated_workspace_bytes(n, k), dtype=torch.uint8, **dev)
        draft = laws.view(n * k, V)
        sv.sv_verify_truncated(target, draft, toks, cu, law, law, 5, step, tokens, accepted, ws,
                               dev_error=err)
        want = verify_truncated(target.cpu().numpy(), draft.cpu().numpy(), toks.cpu().numpy(),
                                cu.tolist(), k, V, settings, settings, 5, step)
        np.testing.assert_array_equal(tokens.cpu().numpy(), want["tokens"])
        np.testing.assert_array_equal(accepted.cpu().numpy(), want["accepted"])
        # what a grammar forbids is never emitted
        for r in range(n):
            if mask_of[r] >= 0:
                assert allowed[mask_of[r]][tokens[r, :int(accepted[r]) + 1].tolist()].all()

        sv.sv_history_add(hist, slots, tokens, False, err)
        for r in range(n):
            for y in tokens[r].tolist():
                if y >= 0:
                    held[int(slots[r]), y] += 2
        np.testing.assert_array_equal(hist.counts.cpu().numpy(), held)
        assert int(err) == 0
        last = tokens.gather(1, accepted.long()[:, None])[:, 0].contiguous()
        ctx = ctx + accepted + 1
