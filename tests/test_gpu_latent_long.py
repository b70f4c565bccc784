"""sv_latent_attend over parts longer than the 1024 positions whose places a workgroup keeps at
a time, against the fp64 oracle; and sums that start again from larger maxima, in either type
and width, before and after those places were renewed.  Tolerances as in test_gpu_latent.py."""

import numpy as np
import pytest
import torch

import adaptive_draft_verification_amd as sv
from test_gpu_latent import Batch, values

pytestmark = pytest.mark.gpu

BF, F8 = torch.bfloat16, torch.float8_e4m3fn
HEADS, K_MAX = 32, 64  # 33 workgroups a request and part
each_form = pytest.mark.parametrize("dtype,rank", [(BF, 512), (BF, 256), (F8, 512), (F8, 256)])


@pytest.fixture(autouse=True, scope="module")
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def batch(seed, long, n, rank, page, dtype):
    """The long requests, (rows, context) each, and short ones up to n."""
    rows = [r for r, _ in long] + [1] * (n - len(long))
    ctx = [c for _, c in long] + [(7 * i) % 20 for i in range(n - len(long))]
    return Batch(seed, rows, ctx, HEADS, rank, page, dtype, k_max=K_MAX)


def part_length(b, r):
    """Positions of request r's first part, as the workspace's size tells the number of parts."""
    size = sv.sv_latent_attend_workspace_bytes(b.n, b.k_max, HEADS, b.rank, b.table.shape[1], b.page)
    each = b.n * HEADS * (b.k_max + 1) * (b.rank + 2) * 4
    assert size % each == 0
    parts, length = max(1, size // each), int(b.ctx[r] + b.cu[r + 1] - b.cu[r])
    return length if parts == 1 else max(256, (-(-length // parts) + 31) // 32 * 32)


@each_form
@pytest.mark.parametrize("page", [16, 17])
def test_long_parts(dtype, rank, page):
    b = batch(41, [(2, 2599), (1, 1536), (2, 1087)], 16, rank, page, dtype)
    assert [part_length(b, r) for r in range(3)] == [2601, 1537, 1089]
    b.device().check()


@each_form
def test_several_long_parts(dtype, rank):
    b = batch(42, [(1, 4500), (2, 2400)], 8, rank, 16, dtype)
    assert part_length(b, 0) == 2272 and part_length(b, 1) == 1216
    b.device().check()


@each_form
@pytest.mark.parametrize("at", [500, 1023, 1024, 1500, 2300])
def test_pages_missing_late_in_a_part(dtype, rank, at):
    b = batch(43, [(2, 2599), (1, 1536)], 16, rank, 16, dtype)
    assert part_length(b, 0) == 2601 and part_length(b, 1) == 1537
    b.kv[0] = float("nan")  # the page a careless kernel would read instead
    b.table[b.table == 0] = b.kv.shape[0] - 1
    b.table[0, at // 16], b.table[1, at // 32] = -1, b.kv.shape[0]
    b.device().check(want_err=sv.SV_DEV_BAD_PAGE)


@each_form
def test_sums_that_start_again(dtype, rank):
    """A key along a query makes a score far above the first tile's: in the second tile, behind
    the renewed places, in the step's own rows, and twice."""
    rises = [[(40, 3.0)], [(1600, 3.0)], [(1500, 3.0)], [(40, 2.0), (1700, 3.0)]]
    b = batch(44, [(1, 700), (2, 2100), (1, 1500), (1, 1800)], 16, rank, 16, dtype)
    k = b.kv.float()
    for r, keys in enumerate(rises):
        q0 = b.q[int(b.cu[r]), 0].float()
        for t, size in keys:
            k[int(b.table[r, t // 16]), t % 16] = size * q0
    b.kv = k.to(dtype)
    kv = values(b.kv) * (1.0 if b.kv_scale is None else b.kv_scale.item())
    for r, keys in enumerate(rises):
        assert part_length(b, r) == int(b.ctx[r] + b.cu[r + 1] - b.cu[r])
        t = np.arange(keys[-1][0] + 1)
        s = kv[b.table[r].numpy()[t // 16], t % 16] @ values(b.q[int(b.cu[r]), 0]) * b.scale
        # the kernel starts again from 2^32 on
        assert (s[-1] - s[:32].max()) / np.log(2.0) > 40
    b.device().check()


@pytest.mark.parametrize("dtype", [BF, F8])
def test_offsets_past_32_bits(dtype):
    """A cache of more than 2^32 values, the pages in use at its ends: written and attended to."""
    pages, page, rank = 120000, 64, 512
    b = Batch(45, [2, 1], [130, 200], 5, rank, page, dtype, extra=0).device()
    kv = torch.zeros(pages, page, rank + 64, dtype=dtype, device="cuda")
    table = b.table.clone()
    for i, p in enumerate(b.table.unique().tolist()):
        to = pages - 1 - i if i % 2 else i
        kv[to] = b.kv[p].cuda()
        table[b.table == p] = to
    assert int(table.max()) * page * (rank + 64) > 2 ** 32
    cache = sv.LatentCache(kv, rank, b.cache.scale)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    # the first row of either request appended anew, as the same values
    at = [(int(table[r, c // page]), c % page) for r, c in enumerate((130, 200))]
    s = 1.0 if b.kv_scale is None else b.kv_scale.item()
    rows = torch.stack([kv[p, j].float() for p, j in at])
    for p, j in at:
        kv[p, j] = 0
    sv.sv_latent_append(cache, table.cuda(), (rows * s).to(BF)[:, :rank], (rows * s).to(BF)[:, rank:],
                        i32([0, 1]), i32([0, 0]), b.ctx.cuda())
    back = torch.stack([kv[p, j].float() for p, j in at])
    # bf16 of the product (2^-8), then e4m3 (2^-4) of it: one step of e4m3 at most
    assert bool(((back - rows).abs() <= rows.abs() * (0 if dtype == BF else 2.0 ** -3)).all())
    for (p, j), row in zip(at, rows):
        kv[p, j] = row.to(dtype)
    b.cache, b.table, small = cache, table, b.table
    out, lse, err = b.attend()
    b.cache, b.table = sv.LatentCache(b.kvd, rank, b.cache.scale), small
    want, want_lse, _ = b.attend()
    assert err == 0 and torch.equal(out, want) and torch.equal(lse, want_lse)
    b.check()
