"""sv_sample on more rows than CUs (another launch shape than few rows get),
against the fp64 oracle and against the same rows in smaller calls.

Tokens and support sizes have to be equal, probabilities within 2^-24 of the
64-bit value and 1e-12 of both sides' own rounding, as for few rows."""

import numpy as np
import pytest
import torch

import adaptive_draft_verification_amd as sv
from test_gpu_sample import (BF, F32, ODD_SETTINGS, SETTINGS, TOP_U, check_sample, check_verify,
                             law_of, odd_rows, run_sample, verify_case)

pytestmark = pytest.mark.gpu

# every setting of the small calls, and top-k around both launch shapes' thread counts
WIDE = SETTINGS + [(1.0, k, p, 0.0) for k in (511, 512, 513, 1023, 1024, 1025) for p in (1.0, 0.9)]


@pytest.fixture(autouse=True, scope="module")
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def check_wide(z, u, settings, vocab=None):
    """Against the oracle, and against calls of 200 rows."""
    assert len(z) > 256
    tok = check_sample(z, u, settings, vocab)
    prob = run_sample(z, u, law_of(settings), vocab)[1]
    for a in range(0, len(z), 200):
        e = min(a + 200, len(z))
        t, p, _, err = run_sample(z[a:e], u[a:e], law_of(settings[a:e]), vocab)
        assert err == 0
        np.testing.assert_array_equal(t, tok[a:e])
        np.testing.assert_allclose(p, prob[a:e], rtol=2.0 ** -23, atol=1e-40)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("vocab,rows", [(1, 257), (7, 300), (8, 257), (63, 280), (511, 257),
                                        (4001, 308), (32000, 257), (70001, 257)])
def test_many_rows(dtype, vocab, rows):
    g = torch.Generator().manual_seed(vocab)
    z = (torch.randn(rows, vocab, generator=g) * 3).to(dtype).cuda()
    u = torch.rand(rows, generator=g)
    u[::11], u[5::17] = TOP_U, 0.0
    check_wide(z, u.tolist(), [WIDE[i % len(WIDE)] for i in range(rows)])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_many_rows_of_ties(dtype):
    g = torch.Generator().manual_seed(71)
    rows, V = 280, 9000
    z = torch.randint(-3, 4, (rows, V), generator=g).float() * 0.5
    z[::7] = 0.0
    z[1::7, ::2] = -0.0
    u = torch.rand(rows, generator=g).tolist()
    check_wide(z.to(dtype).cuda(), u, [WIDE[i % len(WIDE)] for i in range(rows)])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_many_odd_rows(dtype):
    """Every odd row under every setting that takes a way of its own to the border."""
    z = odd_rows(9001, 73).to(dtype)
    settings = [s for s in ODD_SETTINGS + WIDE[:16] for _ in range(len(z))]
    z = z.repeat(len(settings) // len(z), 1).cuda()
    u = torch.rand(len(z), generator=torch.Generator().manual_seed(74)).tolist()
    check_wide(z, u, settings)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_many_rows_that_start_anywhere(dtype):
    g = torch.Generator().manual_seed(75)
    rows, V = 264, 4003
    wide = torch.full((rows, 4099), float("nan"), dtype=dtype)
    wide[:, 3:3 + V] = (torch.randn(rows, V, generator=g) * 2).to(dtype)
    u = torch.rand(rows, generator=g).tolist()
    check_wide(wide.cuda()[:, 3:], u, [WIDE[i % len(WIDE)] for i in range(rows)], V)


def test_many_rows_with_faults():
    g = torch.Generator().manual_seed(77)
    rows, V = 300, 3001
    z = torch.randn(rows, V, generator=g) * 2
    settings = [WIDE[i % len(WIDE)] for i in range(rows)]
    u = torch.rand(rows, generator=g).tolist()
    want = run_sample(z.cuda(), u, law_of(settings))
    z[5, V - 1], z[270, 0], z[299] = float("nan"), float("inf"), -float("inf")
    settings[100], u[200] = (1.0, 0, -1.0, 0.0), 1.0
    got = run_sample(z.cuda(), u, law_of(settings))
    assert got[3] == sv.SV_DEV_NONFINITE | sv.SV_DEV_BAD_PARAM
    bad = [5, 100, 200, 270, 299]
    for x, y in zip(got[:3], want[:3]):
        assert (x[bad] == -1).all()
        np.testing.assert_array_equal(np.delete(x, bad), np.delete(y, bad))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_many_requests_verified(dtype):
    """More requests than CUs, rows of a fifth each of the settings a server mixes."""
    n, k, V = 280, 2, 1501
    settings = [SETTINGS[(0, 1, 3, 4, 6)[i % 5]] for i in range(n)]
    g = check_verify(verify_case(79, n, k, V, dtype, settings), V, 80, 7)
    assert (g["accepted"] >= 0).all()
