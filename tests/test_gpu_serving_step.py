"""The serving calls in a run, as a decode step uses them: drafts drawn from the
drafter's truncated laws, the budget sized and the rows packed, their keys and
values written into the paged cache, the packed rows attending to it, logits
from that, and verification under the same laws; then the next step on the
contexts the accepted tokens made.  Every stage against its oracle, on the
device's own inputs of that stage."""

import numpy as np
import pytest
import torch

import adaptive_draft_verification_amd as sv
from oracle.cache import cache_append, cache_attend
from oracle.truncate import sample_row, verify_truncated

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def test_decode_steps():
    g = torch.Generator().manual_seed(0)
    n, k, V, H, KV, D, page, pages = 6, 3, 501, 4, 2, 64, 16, 40
    dev = dict(device="cuda")
    rn = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    settings = [(0.0, 0, 1.0, 0.0), (0.8, 40, 0.95, 0.0), (1.0, 0, 1.0, 0.0), (0.7, 0, 0.9, 0.0),
                (1.0, 0, 1.0, 0.05), (1.2, 7, 0.8, 0.01)]
    t, kk, p, s = (torch.tensor(x).cuda() for x in zip(*settings))
    law = sv.Sampling(t.float(), kk.int(), p.float(), s.float())
    # a toy model: token embeddings make queries, keys and values; the attended rows make logits
    emb = rn(V, H * D) * 0.5
    wk, wv = rn(H * D, KV * D) / (H * D) ** 0.5, rn(H * D, KV * D) / (H * D) ** 0.5
    head = rn(H * D, V) / (H * D) ** 0.5 * 6
    kc = torch.zeros(pages, page, KV, D, dtype=torch.bfloat16, **dev)
    vc = torch.zeros_like(kc)
    cache = sv.PagedCache(kc, vc)
    table = torch.randperm(pages, generator=g)[:n * 5].int().view(n, 5).cuda()
    ctx = torch.tensor([0, 3, 17, 31, 32, 40], dtype=torch.int32, **dev)
    kc.view(-1, KV, D)[:] = rn(pages * page, KV, D).bfloat16()
    vc.view(-1, KV, D)[:] = rn(pages * page, KV, D).bfloat16()
    cost = torch.from_numpy(sv.sv_cost_table_prepare(
        np.maximum(1.0, np.arange(n * (k + 1) + 1) / 12.0), 1, n + n * k + 1)).cuda()
    last = torch.randint(0, V, (n,), generator=g).int().cuda()
    err = torch.zeros(1, dtype=torch.int32, **dev)
    emitted = 0
    for step in range(3):
        # the drafter: logits of its own, a token a position
        draft = (rn(n * k, V) * 2).contiguous()
        u = torch.empty(n, k, **dev)
        v = torch.empty(n, k, **dev)
        sv.sv_philox_uniforms(99, step, u, v)
        toks = torch.empty(n * k, dtype=torch.int32, **dev)
        conf = torch.empty(n * k, **dev)
        wide = sv.Sampling(*(x.repeat_interleave(k) for x in law))
        sv.sv_sample(draft, u.view(-1), wide, toks, conf, None, err)
        for i in range(n * k):
            want = sample_row(draft[i].cpu().numpy(), float(u.view(-1)[i]), *settings[i // k])
            assert int(toks[i]) == want[0] and abs(float(conf[i]) - want[1]) < 1e-6
        toks, conf = toks.view(n, k), conf.view(n, k)

        dl = torch.tensor([k, k, k - 1, k, 1, k], dtype=torch.int32, **dev)
        b = sv.budget_select(conf, dl, cost, n, n)
        pk = sv.pack_varlen(b["kept"], last, toks)
        cu, req, pos = pk["cu_rows"], pk["row_req"], pk["row_pos"]
        rows = int(cu[-1])

        x = emb[pk["packed_tokens"].clamp(min=0).long()]
        q = x.view(-1, H, D).bfloat16()
        nk, nv = (x @ wk).view(-1, KV, D).bfloat16(), (x @ wv).view(-1, KV, D).bfloat16()
        before = kc.float().cpu().numpy(), vc.float().cpu().numpy()
        sv.sv_cache_append(cache, table, nk, nv, req, pos, ctx, err)
        out = torch.zeros_like(q)
        b_ws = sv.sv_cache_attend_workspace_bytes(n, k, H, KV, D, 5, page)
        ws = torch.empty(max(16, b_ws), dtype=torch.uint8, **dev)
        sv.sv_cache_attend(cache, table, q, cu, ctx, k, D ** -0.5, out, ws, None, err)
        for c, was, new in ((kc, before[0], nk), (vc, before[1], nv)):
            want = cache_append(was, table.cpu().numpy(), new.float().cpu().numpy(),
                                req.tolist(), pos.tolist(), ctx.tolist())
            np.testing.assert_array_equal(c.float().cpu().numpy(), want)
        o, _, spread = cache_attend(q.double().cpu().numpy(), kc.double().cpu().numpy(),
                                    vc.double().cpu().numpy(), table.cpu().numpy(), cu.tolist(),
                                    ctx.tolist(), D ** -0.5)
        diff = np.abs(out.double().cpu().numpy() - o)[:rows]
        # weights and output rounded to bf16 (2^-8 each), scores in fp32
        assert (diff <= 2.0 ** -8 * np.abs(o[:rows]) + 1.01 * 2.0 ** -8 * spread[:rows]).all()
        assert (out[rows:] == 0).all()

        target = (out.float().view(-1, H * D) @ head).contiguous()
        tokens = torch.empty(n, k + 1, dtype=torch.int32, **dev)
        accepted = torch.empty(n, dtype=torch.int32, **dev)
        vws = torch.empty(sv.sv_verify_truncated_workspace_bytes(n, k), dtype=torch.uint8, **dev)
        sv.sv_verify_truncated(target, draft, toks, cu, law, law, 5, step, tokens, accepted, vws,
                               dev_error=err)
        want = verify_truncated(target.cpu().numpy(), draft.cpu().numpy(), toks.cpu().numpy(),
                                cu.tolist(), k, V, settings, settings, 5, step)
        np.testing.assert_array_equal(tokens.cpu().numpy(), want["tokens"])
        np.testing.assert_array_equal(accepted.cpu().numpy(), want["accepted"])
        assert int(err) == 0
        # the accepted drafts' rows stay cached; the token at L starts the next step
        last = tokens.gather(1, accepted.long()[:, None])[:, 0].contiguous()
        ctx = ctx + accepted + 1
        emitted += int(accepted.sum()) + n
    assert emitted >= 3 * n
