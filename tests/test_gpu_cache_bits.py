"""sv_cache_attend gives the bits on record: sha256 of out (bf16) and lse (fp32) for calls that
take each of its kernels, inputs of small integers over 32 (exact in either type).

The digests were written by the build of commit 89f51a2, before other calls came to share the
kernel's source.  They change only with what the sums are rounded to, so that a change of
the source, or of the compiler, that keeps the formula but not the results is seen."""

import hashlib
import json
import os

import pytest
import torch

import adaptive_draft_verification_amd as sv

pytestmark = pytest.mark.gpu

BF, F8 = torch.bfloat16, torch.float8_e4m3fn
GOLDEN = os.path.join(os.path.dirname(__file__), "golden", "cache_attend_bits.json")

# (requests' rows and contexts, heads, kv heads, dim, page)
CALLS = [([(2, 300), (1, 90), (8, 41)], 8, 8, 64, 16), ([(4, 777), (8, 130)], 16, 2, 64, 32),
         ([(8, 515), (7, 64)], 64, 8, 64, 17), ([(1, 1000), (2, 5)], 8, 2, 128, 16),
         ([(8, 700), (3, 257)], 32, 8, 128, 64), ([(4, 3000)], 16, 2, 128, 1),
         ([(8, 400), (5, 33)], 64, 8, 128, 16), ([(8, 900), (1, 2000)], 16, 4, 256, 64),
         ([(3, 129), (4, 64)], 4, 4, 256, 3)]


@pytest.fixture(autouse=True, scope="module")
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def digest(lib, call, dtype):
    requests, heads, kv, dim, page = CALLS[call]
    g = torch.Generator().manual_seed(call)
    draw = lambda *s: torch.randint(-64, 65, s, generator=g).float() / 32  # noqa: E731
    rows = torch.tensor([0] + [r for r, _ in requests])
    n, k_max = len(requests), int(rows.max()) - 1
    width = max(-(-(c + r) // page) for r, c in requests)
    table = torch.randperm(n * width, generator=g).int().view(n, width).cuda()
    k, v = (draw(n * width, page, kv, dim).to(dtype).cuda() for _ in range(2))
    scales = (None, None) if dtype == BF else [(1 + torch.arange(kv) / 16).cuda() for _ in range(2)]
    q = draw(int(rows.sum()), heads, dim).to(BF).cuda()
    cu = torch.cumsum(rows, 0).int().cuda()
    ctx = torch.tensor([c for _, c in requests], dtype=torch.int32, device="cuda")
    ws = torch.empty(lib.sv_cache_attend_workspace_bytes(n, k_max, heads, kv, dim, width, page) + 16,
                     dtype=torch.uint8, device="cuda")
    out, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], device="cuda")
    lib.sv_cache_attend(lib.PagedCache(k, v, *scales), table, q, cu, ctx, k_max, dim ** -0.5, out, ws,
                        lse)
    bits = out.cpu().view(torch.int16).numpy().tobytes() + lse.cpu().numpy().tobytes()
    return hashlib.sha256(bits).hexdigest()


@pytest.mark.parametrize("dtype", [BF, F8])
@pytest.mark.parametrize("call", range(len(CALLS)))
def test_cache_attend_bits(call, dtype):
    with open(GOLDEN) as f:
        want = json.load(f)
    assert digest(sv, call, dtype) == want[f"{call}-{'bf16' if dtype == BF else 'e4m3'}"]
