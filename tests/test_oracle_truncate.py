"""Pins of the truncated-law oracle (CPU)."""

import numpy as np
import pytest

import oracle
from oracle.truncate import sample_row, truncated_law, verify_truncated


def test_hand_derived_laws():
    z = np.log([0.5, 0.25, 0.125, 0.125])
    np.testing.assert_allclose(truncated_law(z)[0], [0.5, 0.25, 0.125, 0.125])
    np.testing.assert_allclose(truncated_law(z, k=2)[0], [2 / 3, 1 / 3, 0, 0])
    assert truncated_law(z, k=3)[1] == 3 and truncated_law(z, k=3)[0][3] == 0  # tie: lower id
    assert truncated_law(z, p=0.6)[1] == 2
    assert truncated_law(z, k=2, p=0.6)[1] == 1       # 2/3 of the first two reaches 0.6
    assert truncated_law(z, s=0.3)[1] == 2 and truncated_law(z, s=1.0)[1] == 1
    assert truncated_law(z, p=0.0)[1] == 1
    # temperature 1/2 squares the weights
    np.testing.assert_allclose(truncated_law(z, t=0.5, k=2)[0], [0.8, 0.2, 0, 0])
    law, n = truncated_law([1.0, 3.0, 3.0, -np.inf], t=0.0)
    assert n == 1 and law.tolist() == [0, 1, 0, 0]
    law, n = truncated_law([-0.0, 0.0, -np.inf], k=1)
    assert n == 1 and law.tolist() == [1, 0, 0]
    assert truncated_law([2.0, -np.inf], k=2)[1] == 1


def test_uniform_row_counts():
    z = np.zeros(1000)
    for p, n in ((0.5, 500), (0.25, 250), (0.2505, 251), (1.0, 1000)):
        assert truncated_law(z, p=p)[1] == n
    assert sample_row(z, 0.5)[0] == 500 and sample_row(z, 0.0)[0] == 0


@pytest.mark.parametrize("seed", range(5))
def test_support_by_exhaustion(seed):
    """Every prefix length tried against the definition, in exact order."""
    rng = np.random.default_rng(seed)
    z = np.round(rng.standard_normal(40) * 2, 1)
    t, k, p, s = 0.7, int(rng.integers(0, 30)), float(rng.uniform(0.3, 1)), float(
        rng.uniform(0, 0.2))
    ids = sorted(range(40), key=lambda i: (-z[i], i))
    t, p, s = (float(np.float32(x)) for x in (t, p, s))
    w = [np.exp((z[i] - z[ids[0]]) / t) for i in ids]
    n_k = k or 40
    n_p = next(n for n in range(1, n_k + 1) if sum(w[:n]) >= p * sum(w[:n_k]))
    n_m = sum(x >= s for x in w)
    law, n = truncated_law(z, t, k, p, s)
    assert n == min(n_k, n_p, n_m)
    assert set(np.nonzero(law)[0]) == set(ids[:n])
    assert abs(law.sum() - 1) < 1e-12


def test_no_truncation_is_the_plain_verify():
    rng = np.random.default_rng(3)
    n, k, V = 5, 3, 40
    cu = np.array([0, 4, 6, 7, 11, 13])
    target = rng.standard_normal((13, V)) * 2
    draft = rng.standard_normal((n * k, V)) * 2
    toks = rng.integers(0, V, (n, k))
    a = verify_truncated(target, draft, toks, cu, k, V, [(0.8, 0, 1.0, 0.0)] * n,
                         [(0.8, 0, 1.0, 0.0)] * n, 9, 4)
    b = oracle.verify(target, draft, toks, cu, k, V, oracle.STOCHASTIC, float(np.float32(0.8)),
                      9, 4)
    np.testing.assert_array_equal(a["tokens"], b["tokens"])
    np.testing.assert_array_equal(a["accepted"], b["accepted"])
    np.testing.assert_allclose(a["p_draft"], b["p_draft"], rtol=1e-6)


def test_verified_tokens_follow_the_truncated_target():
    """With drafts drawn from the truncated draft law, the first token emitted has
    the truncated target law (exact enumeration over u and the draft)."""
    rng = np.random.default_rng(6)
    V = 12
    zp, zq = rng.standard_normal(V) * 2, rng.standard_normal(V) * 2
    p, _ = truncated_law(zp, 0.9, 5, 0.95, 0.0)
    q, _ = truncated_law(zq, 0.9, 6, 1.0, 0.05)
    got = np.zeros(V)
    for d in range(V):
        if q[d] == 0:
            continue
        a = min(1.0, p[d] / q[d])
        got[d] += q[d] * a
        w, mass = oracle.residual_weights(p, q)
        got += q[d] * (1 - a) * w / w.sum()
    np.testing.assert_allclose(got, p, atol=1e-12)
