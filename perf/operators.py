"""What is measured of the serving operators around the verify step.

Four operators: the draw of a token under temperature, top-k, top-p and min-p
(sample), verification under such truncated laws (verify), writing a packed
step's keys and values into a paged cache (append), and the packed rows'
attention over that cache (attend).  Where ``own`` is false ``run`` computes
them in plain torch operations; where it is true, through the library."""

import math

import torch

own = False

DEV = "cuda"


def listed():
    return [
        # one user, one token: latency
        dict(name="sample_1x32000_bf16", op="sample", rows=1, vocab=32000, dtype="bf16",
             law="topk"),
        # a few users, nucleus sampling, an odd vocabulary (rows not aligned to 16 bytes)
        dict(name="sample_16x128255_bf16", op="sample", rows=16, vocab=128255, dtype="bf16",
             law="nucleus"),
        # the library's headline batch: every request with its own settings, greedy ones among them
        dict(name="sample_256x129280_bf16", op="sample", rows=256, vocab=129280, dtype="bf16",
             law="mixed"),
        # its largest vocabulary, fp32 logits, nucleus sampling
        dict(name="sample_256x256000_f32", op="sample", rows=256, vocab=256000, dtype="f32",
             law="nucleus"),
        # a small batch's verification, fp32
        dict(name="verify_4x3x32000_f32", op="verify", n=4, k=3, vocab=32000, dtype="f32",
             law="topk"),
        # the headline batch's, with each request's own settings
        dict(name="verify_256x7x129280_bf16", op="verify", n=256, k=7, vocab=129280, dtype="bf16",
             law="mixed"),
        # one new token of one request into the cache
        dict(name="append_1x1_bf16", op="append", n=1, k=0, heads=8, kv_heads=8, dim=128, page=16,
             ctx=1000, ragged=False, cache="bf16"),
        # a full verify step's rows into an 8-bit cache
        dict(name="append_256x8_e4m3", op="append", n=256, k=7, heads=8, kv_heads=8, dim=128,
             page=64, ctx=120, ragged=True, cache="e4m3"),
        # one new token of one request: latency
        dict(name="attend_1x1_ctx1023_bf16", op="attend", n=1, k=0, heads=32, kv_heads=8, dim=128,
             page=16, ctx=1023, ragged=False, cache="bf16"),
        # many short chats, a head of its own for every query, narrow heads
        dict(name="attend_64x8_ctx1500_e4m3", op="attend", n=64, k=7, heads=16, kv_heads=16,
             dim=64, page=32, ctx=1500, ragged=True, cache="e4m3"),
        # the headline batch verified: 1..8 rows a request, contexts up to 4096
        dict(name="attend_256x8_ctx4096_bf16", op="attend", n=256, k=7, heads=32, kv_heads=8,
             dim=128, page=64, ctx=4096, ragged=True, cache="bf16"),
        # few long documents, 8-bit cache: the length has to be split
        dict(name="attend_3x4_ctx100001_e4m3", op="attend", n=3, k=3, heads=64, kv_heads=8,
             dim=128, page=64, ctx=100001, ragged=False, cache="e4m3"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["sample", "verify", "append", "attend"])
    if op == "sample":
        dtype = rng.choice(["bf16", "f32"])
        vocab = _log(rng, 1000, 256000)
        most = 256 * 256000 * 4 // (vocab * (2 if dtype == "bf16" else 4))
        return dict(op=op, rows=_log(rng, 1, min(most, 512)), vocab=vocab, dtype=dtype,
                    law=rng.choice(["topk", "nucleus", "minp", "mixed"]))
    if op == "verify":
        vocab, k = _log(rng, 1000, 129280), rng.randint(1, 7)
        most = max(1, 256 * 7 * 129280 // (2 * vocab * k))
        return dict(op=op, n=_log(rng, 1, min(most, 256)), k=k, vocab=vocab,
                    dtype=rng.choice(["bf16", "f32"]),
                    law=rng.choice(["topk", "nucleus", "minp", "mixed"]))
    dim, kv = rng.choice([64, 128, 256]), rng.choice([1, 2, 4, 8, 16])
    group, k = rng.choice([1, 2, 4, 7, 8]), rng.choice([0, 0, 1, 3, 5, 7])
    page = rng.choice([1, 8, 16, 17, 32, 64, 128])
    cache = rng.choice(["bf16", "e4m3"])
    if op == "append":
        return dict(op=op, n=_log(rng, 1, 256), k=k, heads=kv, kv_heads=kv, dim=dim, page=page,
                    ctx=_log(rng, 1, 500), ragged=rng.random() < 0.7, cache=cache)
    n = _log(rng, 1, 256)
    most = 256 * 4096 * 8 * 128 // (2 * n * kv * dim)
    ctx = _log(rng, 1, max(2, min(131072, most)))
    return dict(op=op, n=n, k=k, heads=kv * group, kv_heads=kv, dim=dim, page=page, ctx=ctx,
                ragged=rng.random() < 0.7, cache=cache)


# --------------------------------------------------------------------- inputs

def _law(kind, n, g):
    """Per-row settings, as a server holds them: temperature, top_k, top_p, min_p."""
    r = torch.rand(4, n, generator=g, device=DEV)
    t = 0.6 + 0.6 * r[0]
    k = torch.zeros(n, dtype=torch.int32, device=DEV)
    p = torch.ones(n, device=DEV)
    s = torch.zeros(n, device=DEV)
    if kind == "topk":
        k += 20 + (r[1] * 60).int()
        p = 0.8 + 0.19 * r[2]
    elif kind == "nucleus":
        p = 0.85 + 0.1 * r[2]
    elif kind == "minp":
        s = 0.02 + 0.1 * r[3]
    else:
        # a fifth each: greedy, temperature alone, top-k with top-p, nucleus, min-p
        i = torch.arange(n, device=DEV) % 5
        t = torch.where(i == 0, 0.0, t)
        k = torch.where(i == 2, 20 + (r[1] * 60).int(), k).int()
        p = torch.where((i == 2) | (i == 3), 0.85 + 0.1 * r[2], p)
        s = torch.where(i == 4, 0.02 + 0.1 * r[3], s)
    return t, k, p, s


def _ragged_rows(n, k, ragged, g):
    rows = torch.full((n,), k + 1, dtype=torch.int32, device=DEV)
    if ragged:
        rows = torch.randint(1, k + 2, (n,), generator=g, device=DEV, dtype=torch.int32)
    cu = torch.zeros(n + 1, dtype=torch.int32, device=DEV)
    cu[1:] = torch.cumsum(rows, 0)
    return rows, cu


def _maps(rows, n, k):
    """(request, position) of every packed row, -1 behind the last one."""
    cap = n * (k + 1)
    r = torch.repeat_interleave(torch.arange(n, device=DEV), rows.long())
    first = torch.repeat_interleave(torch.cumsum(rows.long(), 0) - rows.long(), rows.long())
    req = torch.full((cap,), -1, dtype=torch.int32, device=DEV)
    pos = torch.full((cap,), -1, dtype=torch.int32, device=DEV)
    req[:len(r)] = r.int()
    pos[:len(r)] = (torch.arange(len(r), device=DEV) - first).int()
    return req, pos


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    st = dict(case=case)
    rn = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}.get(case.get("dtype"))
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    if case["op"] == "sample":
        n, V = case["rows"], case["vocab"]
        st["logits"] = (3 * rn(n, V)).to(dt)
        st["u"] = torch.rand(n, generator=g, device=DEV)
        st["law"] = _law(case["law"], n, g)
        st["out"] = (torch.empty(n, dtype=torch.int32, device=DEV),
                     torch.empty(n, device=DEV),
                     torch.empty(n, dtype=torch.int32, device=DEV), err)
        return st
    if case["op"] == "verify":
        n, k, V = case["n"], case["k"], case["vocab"]
        rows, cu = _ragged_rows(n, k, True, g)
        st["cu"], total = cu, int(cu[-1])
        target = (3 * rn(total, V)).to(dt)
        # draft row (r, j) is the target's row with noise; slots that were not kept hold zeros
        draft = torch.zeros(n * k, V, dtype=dt, device=DEV)
        req, pos = _maps(rows, n, k)
        req, pos = req[:total].long(), pos[:total].long()
        drafted = pos < rows.long()[req] - 1
        slot = (req * k + pos)[drafted]
        draft[slot] = (target[drafted].float() + rn(int(drafted.sum()), V)).to(dt)
        law = _law(case["law"], n, g)
        u = torch.rand(n * k, generator=g, device=DEV)
        toks = torch.full((n * k,), -1, dtype=torch.int32, device=DEV)
        toks[slot] = _sample(draft[slot], u[slot], [x[req[drafted]] for x in law])[0]
        st.update(target=target, draft=draft, tokens=toks.view(n, k), law=law, seed=seed,
                  step=seed % 1000 + 1,
                  ws=torch.empty(n * (2 * k + 1) * 64, dtype=torch.uint8, device=DEV),
                  out=(torch.empty(n, k + 1, dtype=torch.int32, device=DEV),
                       torch.empty(n, dtype=torch.int32, device=DEV),
                       torch.empty(n, k, device=DEV), torch.empty(n, k, device=DEV),
                       torch.empty(n, device=DEV), err))
        return st
    n, k, hkv, d, page = (case[x] for x in ("n", "k", "kv_heads", "dim", "page"))
    rows, cu = _ragged_rows(n, k, case["ragged"], g)
    ctx = torch.full((n,), case["ctx"], dtype=torch.int32, device=DEV)
    if case["ragged"]:
        ctx = torch.randint(0, case["ctx"] + 1, (n,), generator=g, device=DEV, dtype=torch.int32)
    width = -(-(case["ctx"] + k + 1) // page)
    # pages in no order, as a pool hands them out
    table = torch.randperm(n * width, generator=g, device=DEV).int().view(n, width)
    store = torch.bfloat16 if case["cache"] == "bf16" else torch.float8_e4m3fn
    shape = (n * width, page, hkv, d)
    kc = torch.empty(shape, dtype=store, device=DEV)
    vc = torch.empty(shape, dtype=store, device=DEV)
    for c in (kc, vc):
        flat = c.view(-1)
        for i in range(0, flat.numel(), 1 << 28):
            part = flat[i:i + (1 << 28)]
            part.copy_(rn(part.numel()).to(store))
    scales = None
    if case["cache"] == "e4m3":
        scales = tuple(0.5 + torch.rand(hkv, generator=g, device=DEV) for _ in range(2))
    st.update(rows=rows, cu=cu, ctx=ctx, table=table, k=kc, v=vc, scales=scales, err=err)
    if case["op"] == "append":
        cap = n * (k + 1)
        st["req"], st["pos"] = _maps(rows, n, k)
        st["new_k"], st["new_v"] = rn(cap, hkv, d).bfloat16(), rn(cap, hkv, d).bfloat16()
        return st
    # scores with a spread of about 2: some positions weigh, most do not.  Buffers hold a full
    # step's rows; those behind the last packed row stay as they are
    st["q"] = (2 * rn(n * (k + 1), case["heads"], d)).bfloat16()
    st["scale"] = 1 / math.sqrt(d)
    st["out"] = torch.zeros_like(st["q"])
    st["lse"] = torch.zeros(n * (k + 1), case["heads"], device=DEV)
    # scratch that any call of these ranges fits in, kept as a server keeps it
    st["ws"] = torch.empty(256 << 20, dtype=torch.uint8, device=DEV)
    return st


# ---------------------------------------------------------------- plain forms

def _weights(z, law):
    """(weights in id order with 0 outside the law's support, support sizes), 64 bits."""
    t, k, p, s = [x[:, None] for x in law]
    order = torch.sort(z.float(), dim=-1, descending=True, stable=True)
    y = order.values.double() - order.values[:, :1].double()
    greedy = t == 0
    w = torch.where(greedy, (y == 0).double(), torch.exp(y / torch.where(greedy, 1, t).double()))
    rank = torch.arange(z.shape[1], device=z.device)[None]
    most = torch.where(k > 0, k, z.shape[1]).long()
    most = torch.where(greedy, 1, most)
    wk = torch.where(rank < most, w, 0)
    c = torch.cumsum(wk, -1)
    inside = (rank == 0) | (p >= 1) | (c - wk < p.double() * c[:, -1:])
    keep = inside & (rank < most) & (w >= s.double()) & torch.isfinite(y)
    size = keep.sum(-1, dtype=torch.int32)
    return torch.zeros_like(w).scatter_(1, order.indices, torch.where(keep, w, 0)), size


def _pick(w, u):
    """The smallest id whose running sum passes u of the total."""
    c = torch.cumsum(w, -1)
    at = (c <= u.double()[:, None] * c[:, -1:]).sum(-1)
    last = w.shape[1] - 1 - (w > 0).flip(-1).int().argmax(-1)
    return torch.minimum(at, last)


def _sample(z, u, law):
    w, size = _weights(z, law)
    tok = _pick(w, u)
    prob = w.gather(1, tok[:, None])[:, 0] / w.sum(-1)
    return tok.int(), prob.float(), size


def _mul_hi_lo(a, b):
    """High and low words of a 32 x 32 bit product, in 64-bit integers."""
    lo, hi = (a & 0xFFFF) * b, (a >> 16) * b
    s = (lo >> 16) + (hi & 0xFFFF)
    low = ((s & 0xFFFF) << 16) | (lo & 0xFFFF)
    return (hi >> 16) + (s >> 16), low


def _uniforms(seed, step, n, k):
    """Philox4x32-10, counter (request, position, step low, step high), key = seed."""
    c0 = torch.arange(n, device=DEV)[:, None].expand(n, k + 1)
    c1 = torch.arange(k + 1, device=DEV)[None].expand(n, k + 1)
    c2, c3 = torch.full_like(c0, step & 0xFFFFFFFF), torch.full_like(c0, step >> 32)
    key0, key1 = seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF
    for _ in range(10):
        h0, l0 = _mul_hi_lo(c0, 0xD2511F53)
        h1, l1 = _mul_hi_lo(c2, 0xCD9E8D57)
        c0, c1, c2, c3 = h1 ^ c1 ^ key0, l1, h0 ^ c3 ^ key1, l0
        key0, key1 = (key0 + 0x9E3779B9) & 0xFFFFFFFF, (key1 + 0xBB67AE85) & 0xFFFFFFFF
    return (c0 >> 8).double() / 2 ** 24, (c1 >> 8).double() / 2 ** 24


def _verify(st):
    n, k, V = (st["case"][x] for x in ("n", "k", "vocab"))
    cu = st["cu"].long()
    b = cu[1:] - cu[:-1] - 1
    u, v = _uniforms(st["seed"], st["step"], n, k)
    req = torch.repeat_interleave(torch.arange(n, device=DEV), b + 1)
    pos = torch.arange(len(req), device=DEV) - cu[req]
    p, _ = _weights(st["target"], [x[req] for x in st["law"]])
    p /= p.sum(-1, keepdim=True)
    has = pos < b[req]
    slot = req[has] * k + pos[has]
    q = torch.zeros_like(p)
    qw, _ = _weights(st["draft"][slot], [x[req[has]] for x in st["law"]])
    q[has] = qw / qw.sum(-1, keepdim=True)
    d = st["tokens"].view(-1)[slot].long()[:, None]
    pd, qd = p[has].gather(1, d)[:, 0], q[has].gather(1, d)[:, 0]
    ok = torch.where(qd > 0, u[req[has], pos[has]] < pd / qd, pd > 0)
    fine = torch.zeros(n, k + 1, dtype=torch.bool, device=DEV)
    fine[req[has], pos[has]] = ok
    L = fine.int().cumprod(-1).sum(-1)
    at = cu[:-1] + L
    w = (p[at] - q[at]).clamp(min=0)
    mass = w.sum(-1)
    rejected = L < b
    w = torch.where((mass == 0)[:, None], p[at], w)
    tok = _pick(w, v.gather(1, L[:, None])[:, 0])
    j = torch.arange(k + 1, device=DEV)[None]
    tokens = torch.nn.functional.pad(st["tokens"], (0, 1), value=-1)
    tokens = torch.where(j < L[:, None], tokens, torch.where(j == L[:, None], tok[:, None].int(),
                                                             -1))
    outp = torch.full((n, k), -1.0, device=DEV)
    outq = torch.full((n, k), -1.0, device=DEV)
    outp[req[has], pos[has]], outq[req[has], pos[has]] = pd.float(), qd.float()
    return tokens.int(), L.int(), outp, outq, torch.where(rejected, mass, -1.0).float()


def _append(st):
    case = st["case"]
    live = st["req"] >= 0
    req, pos = st["req"][live].long(), st["pos"][live].long()
    t = st["ctx"].long()[req] + pos
    page, slot = st["table"][req, t // case["page"]].long(), t % case["page"]
    new = [x[live].float() for x in (st["new_k"], st["new_v"])]
    if st["scales"]:
        new = [(x / s[None, :, None]).clamp(-448, 448) for x, s in zip(new, st["scales"])]
        st["k"].view(torch.uint8)[page, slot] = new[0].to(st["k"].dtype).view(torch.uint8)
        st["v"].view(torch.uint8)[page, slot] = new[1].to(st["v"].dtype).view(torch.uint8)
        return st["k"].float(), st["v"].float()
    st["k"][page, slot], st["v"][page, slot] = new[0].to(st["k"].dtype), new[1].to(st["v"].dtype)
    return st["k"], st["v"]


def _attend(st):
    case = st["case"]
    n, k, h, hkv, d = (case[x] for x in ("n", "k", "heads", "kv_heads", "dim"))
    table = st["table"].long()
    length = table.shape[1] * case["page"]
    kk, vv = [x.view(torch.uint8 if st["scales"] else x.dtype)[table].view(n, length, hkv, d)
              for x in (st["k"], st["v"])]
    if st["scales"]:
        kk, vv = [x.view(torch.float8_e4m3fn).float() * s[:, None]
                  for x, s in zip((kk, vv), st["scales"])]
    cu = st["cu"].long()
    rows = cu[1:] - cu[:-1]
    j = torch.arange(k + 1, device=DEV)
    live = j[None] < rows[:, None]
    index = torch.where(live, cu[:-1, None] + j[None], 0)
    q = st["q"].float()[index].view(n, k + 1, hkv, h // hkv, d)
    q = q.permute(0, 2, 1, 3, 4).reshape(n, hkv, -1, d)
    s = q @ kk.float().permute(0, 2, 3, 1).contiguous() * st["scale"]
    s = s.view(n, hkv, k + 1, h // hkv, length)
    t = st["ctx"].long()[:, None] + j[None]
    seen = torch.arange(length, device=DEV) <= t[:, None, :, None, None]
    s = torch.where(seen, s, -math.inf)
    m = s.amax(-1, keepdim=True)
    e = torch.exp(s - m)
    total = e.sum(-1, keepdim=True)
    o = (e / total).view(n, hkv, -1, length) @ vv.float().permute(0, 2, 1, 3).contiguous()
    o = o.view(n, hkv, k + 1, h // hkv, d).permute(0, 2, 1, 3, 4).reshape(n, k + 1, h, d)
    lse = (m + total.log())[..., 0].permute(0, 2, 1, 3).reshape(n, k + 1, h)
    out, out_lse = torch.zeros_like(st["out"]), torch.zeros_like(st["lse"])
    at = index[live]
    out[at], out_lse[at] = o[live].bfloat16(), lse[live]
    return out, out_lse


# ------------------------------------------------------------------------ run

def run(st):
    case = st["case"]
    if own:
        import adaptive_draft_verification_amd as sv
        if case["op"] == "sample":
            tok, prob, size, err = st["out"]
            sv.sv_sample(st["logits"], st["u"], sv.Sampling(*st["law"]), tok, prob, size, err)
            return tok, prob, size
        if case["op"] == "verify":
            toks, acc, p, q, mass, err = st["out"]
            law = sv.Sampling(*st["law"])
            sv.sv_verify_truncated(st["target"], st["draft"], st["tokens"], st["cu"], law, law,
                                   st["seed"], st["step"], toks, acc, st["ws"], p, q, mass, err)
            return toks, acc, p, q, mass
        cache = sv.PagedCache(st["k"], st["v"], *(st["scales"] or ()))
        if case["op"] == "append":
            sv.sv_cache_append(cache, st["table"], st["new_k"], st["new_v"], st["req"], st["pos"],
                               st["ctx"], st["err"])
            return (st["k"].float(), st["v"].float()) if st["scales"] else (st["k"], st["v"])
        sv.sv_cache_attend(cache, st["table"], st["q"], st["cu"], st["ctx"], case["k"],
                           st["scale"], st["out"], st["ws"], st["lse"], st["err"])
        return st["out"], st["lse"]
    if case["op"] == "sample":
        return _sample(st["logits"], st["u"], st["law"])
    return {"verify": _verify, "append": _append, "attend": _attend}[case["op"]](st)


def _attended(case):
    """Mean cached positions a request's rows see (its own rows counted), and mean rows."""
    rows = case["k"] / 2 + 1 if case["ragged"] else case["k"] + 1
    return (case["ctx"] / 2 if case["ragged"] else case["ctx"]) + rows, rows


def work(case):
    esize = {"bf16": 2, "f32": 4, "e4m3": 1}[case.get("dtype") or case["cache"]]
    if case["op"] == "sample":
        ids = case["rows"] * case["vocab"]
        return dict(bytes=ids * esize + case["rows"] * 32, flops=4 * ids)
    if case["op"] == "verify":
        ids = case["n"] * (case["k"] + 1) * case["vocab"]  # k/2 + 1 target and k/2 draft rows
        return dict(bytes=ids * esize, flops=4 * ids)
    length, rows = _attended(case)
    kv = 2 * case["kv_heads"] * case["dim"]
    if case["op"] == "append":
        # an 8-bit cache is handed back as the values it stands for: read whole, written in fp32
        cells = case["n"] * (-(-(case["ctx"] + case["k"] + 1) // case["page"])) * case["page"]
        back = cells * kv * 5 if case["cache"] == "e4m3" else 0
        return dict(bytes=int(case["n"] * rows * kv * (2 + esize)) + back,
                    flops=int(case["n"] * rows * kv))
    b = case["n"] * length * kv * esize + case["n"] * rows * case["heads"] * case["dim"] * 4
    return dict(bytes=int(b), flops=int(4 * case["n"] * rows * case["heads"] * case["dim"]
                                        * length))


# ---------------------------------------------------------------------- exact

def _exact_law(z, t, k, p, s):
    """One row's law from the definition: probabilities in id order, and its support's size."""
    z = z.double()
    if t == 0:
        one = torch.zeros_like(z)
        one[int((z == z.max()).nonzero()[0])] = 1
        return one, 1
    ids = torch.argsort(-z, stable=True)
    w = torch.exp((z[ids] - z.max()) / t)
    n = len(z) if k <= 0 else min(k, len(z))
    if p < 1:
        part = w[:n].cumsum(0)
        n = max(1, min(n, int((part < p * part[-1]).sum()) + 1))
    n = min(n, int((w >= s).sum()), int(torch.isfinite(z).sum()))
    law = torch.zeros_like(z)
    law[ids[:n]] = w[:n] / w[:n].sum()
    return law, n


def _exact_pick(w, u):
    c = w.cumsum(0)
    past = (c > u * c[-1]).nonzero()
    return int(past[0]) if len(past) else int((w > 0).nonzero()[-1])


def _exact_sample(st):
    laws = list(zip(*(x.tolist() for x in st["law"])))
    tok, prob, size = [], [], []
    for z, u, law in zip(st["logits"], st["u"].tolist(), laws):
        w, n = _exact_law(z, *law)
        tok.append(_exact_pick(w, u))
        prob.append(float(w[tok[-1]]))
        size.append(n)
    return (torch.tensor(tok, dtype=torch.int32), torch.tensor(prob, dtype=torch.float64),
            torch.tensor(size, dtype=torch.int32))


def _exact_philox(seed, step, r, j):
    c = [r, j, step & 0xFFFFFFFF, step >> 32]
    key = [seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF]
    for _ in range(10):
        a, b = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(b >> 32) ^ c[1] ^ key[0], b & 0xFFFFFFFF, (a >> 32) ^ c[3] ^ key[1], a & 0xFFFFFFFF]
        key = [(key[0] + 0x9E3779B9) & 0xFFFFFFFF, (key[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return (c[0] >> 8) / 2 ** 24, (c[1] >> 8) / 2 ** 24


def _exact_verify(st):
    n, k = st["case"]["n"], st["case"]["k"]
    cu, drafts = st["cu"].tolist(), st["tokens"].tolist()
    laws = list(zip(*(x.tolist() for x in st["law"])))
    tokens = torch.full((n, k + 1), -1, dtype=torch.int32)
    accepted = torch.zeros(n, dtype=torch.int32)
    outp = torch.full((n, k), -1.0, dtype=torch.float64)
    outq, mass = outp.clone(), torch.full((n,), -1.0, dtype=torch.float64)
    for r in range(n):
        b = cu[r + 1] - cu[r] - 1
        L, at = b, None
        for j in range(b):
            p, _ = _exact_law(st["target"][cu[r] + j], *laws[r])
            q, _ = _exact_law(st["draft"][r * k + j], *laws[r])
            pd, qd = float(p[drafts[r][j]]), float(q[drafts[r][j]])
            outp[r, j], outq[r, j] = pd, qd
            u = _exact_philox(st["seed"], st["step"], r, j)[0]
            if L == b and at is None and not (u < pd / qd if qd > 0 else pd > 0):
                L, at = j, torch.clamp(p - q, min=0)
                mass[r] = float(at.sum())
                at = at if mass[r] > 0 else p
        if at is None:
            at = _exact_law(st["target"][cu[r] + b], *laws[r])[0]
        accepted[r] = L
        tokens[r, :L] = torch.tensor(drafts[r][:L], dtype=torch.int32)
        tokens[r, L] = _exact_pick(at, _exact_philox(st["seed"], st["step"], r, L)[1])
    return tokens, accepted, outp, outq, mass


def _exact_append(st):
    case = st["case"]
    if st["scales"]:
        return None  # what is kept is the rounding to 8 bits itself
    out = []
    for cache, new in ((st["k"], st["new_k"]), (st["v"], st["new_v"])):
        full = cache.double()
        for i, (r, j) in enumerate(zip(st["req"].tolist(), st["pos"].tolist())):
            if r < 0:
                continue
            t = int(st["ctx"][r]) + j
            full[int(st["table"][r, t // case["page"]]), t % case["page"]] = new[i].double()
        out.append(full)
    return tuple(out)


def _exact_attend(st):
    case = st["case"]
    h, hkv = case["heads"], case["kv_heads"]
    cu, ctx = st["cu"].tolist(), st["ctx"].tolist()
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(st["q"].shape[:2], dtype=torch.float64, device=DEV)
    for r in range(case["n"]):
        last = ctx[r] + cu[r + 1] - cu[r]
        t = torch.arange(last, device=DEV)
        page = st["table"][r].long()[t // case["page"]]
        kv = []
        for c, cache in enumerate((st["k"], st["v"])):
            x = cache.view(torch.uint8 if st["scales"] else cache.dtype)[page, t % case["page"]]
            x = x.view(cache.dtype).double()
            kv.append(x * st["scales"][c].double()[:, None] if st["scales"] else x)
        for row in range(cu[r], cu[r + 1]):
            n = ctx[r] + row - cu[r] + 1
            q = st["q"][row].double().view(hkv, h // hkv, -1)
            s = torch.matmul(q, kv[0][:n].permute(1, 2, 0)) * st["scale"]
            lse[row] = torch.logsumexp(s, -1).view(h)
            p = torch.exp(s - torch.logsumexp(s, -1, keepdim=True))
            out[row] = torch.matmul(p, kv[1][:n].permute(1, 0, 2)).view(h, -1)
    return out, lse


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "attend" and work(case)["flops"] > 3e11:
        return None
    return {"sample": _exact_sample, "verify": _exact_verify, "append": _exact_append,
            "attend": _exact_attend}[case["op"]](st)
