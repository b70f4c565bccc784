"""Truncated laws: sampling and verification with temperature, top-k, top-p and
min-p — oracle side (test infrastructure).

The pages name the rule only through its result (FOS blog, section "속도,
메모리, 정확도에 주는 영향", row 정확도: rejection sampling keeps the target's
law).  With the usual serving settings the target's law is its truncated
softmax: ids ordered by logit (ties to the lower id), the first k, of those
the fewest that reach p of their weight, of those the ones of at least min_p
times the largest weight; renormalised.  Readings: a temperature of 0 is the
argmax; ids of logit -inf never take part; top_k <= 0 is off.  All in fp64.
"""

import math

import numpy as np

from .philox import uniforms
from .verify import (DEV_BAD_CU_ROWS, DEV_BAD_TOKEN, DEV_NONFINITE, accept, inverse_cdf,
                     residual_weights, row_is_faulty)

DEV_BAD_PARAM = 256


def bad_settings(t, k, p, s):
    return not (t >= 0 and math.isfinite(t) and p >= 0 and 0 <= s <= 1)


def truncated_weights(z, t=1.0, k=0, p=1.0, s=0.0):
    """(weights in id order, 1 for the largest logit and 0 outside the support, ids in the
    support); settings are fp32 values."""
    z = np.asarray(z, dtype=np.float64) + 0.0  # -0 equals 0
    t, p, s = float(np.float32(t)), float(np.float32(p)), float(np.float32(s))
    law = np.zeros(len(z))
    if t == 0.0:
        law[int(np.argmax(z))] = 1.0
        return law, 1
    order = np.argsort(-z, kind="stable")
    order = order[np.isfinite(z[order])]
    w = np.exp((z[order] - z[order[0]]) / t)
    n = len(order) if k <= 0 else min(int(k), len(order))
    n_p = n
    if p < 1.0:
        c = np.cumsum(w[:n])
        n_p = min(n, int(np.searchsorted(c, p * c[-1], side="left")) + 1)
    n_m = int((w >= s).sum())
    n = max(1, min(n, n_p, n_m))
    law[order[:n]] = w[:n]
    return law, n


def truncated_law(z, t=1.0, k=0, p=1.0, s=0.0):
    """(probabilities in id order, ids in the support)."""
    w, n = truncated_weights(z, t, k, p, s)
    return w / math.fsum(w), n


def sample_row(z, u, t=1.0, k=0, p=1.0, s=0.0):
    """(token, probability, support size) of one draw: over the weights themselves, whose
    sums are exact where the weights are equal."""
    w, n = truncated_weights(z, t, k, p, s)
    tok = inverse_cdf(w, float(np.float32(u)))
    return tok, w[tok] / math.fsum(w), n


def verify_truncated(target, draft, draft_tokens, cu_rows, k_max, vocab, target_settings,
                     draft_settings, seed, step):
    """Outputs of sv_verify_truncated; settings: per request (t, k, p, s)."""
    n = len(cu_rows) - 1
    out = dict(tokens=np.full((n, k_max + 1), -1, np.int32), accepted=np.full(n, -1, np.int32),
               p_draft=np.full((n, k_max), -1.0), q_draft=np.full((n, k_max), -1.0),
               residual_mass=np.full(n, -1.0), dev_error=0)
    for r in range(n):
        lo, hi = int(cu_rows[r]), int(cu_rows[r + 1])
        b = hi - lo - 1
        if lo < 0 or b < 0 or b > k_max or hi > len(target):
            out["dev_error"] |= DEV_BAD_CU_ROWS
            continue
        fault = 0
        if bad_settings(*target_settings[r]) or (b > 0 and bad_settings(*draft_settings[r])):
            fault |= DEV_BAD_PARAM
        for j in range(b + 1):
            if row_is_faulty(target[lo + j][:vocab]):
                fault |= DEV_NONFINITE
            if j < b:
                if row_is_faulty(draft[r * k_max + j][:vocab]):
                    fault |= DEV_NONFINITE
                if not 0 <= draft_tokens[r][j] < vocab:
                    fault |= DEV_BAD_TOKEN
        if fault:
            out["dev_error"] |= fault
            continue
        L, uv = b, [uniforms(seed, r, j, step) for j in range(b + 1)]
        laws = []
        for j in range(b):
            p, _ = truncated_law(target[lo + j][:vocab], *target_settings[r])
            q, _ = truncated_law(draft[r * k_max + j][:vocab], *draft_settings[r])
            d = int(draft_tokens[r][j])
            out["p_draft"][r, j], out["q_draft"][r, j] = p[d], q[d]
            laws.append((p, q))
            if L == b and not accept(uv[j][0], p[d], q[d]):
                L = j
        if L < b:
            w, out["residual_mass"][r] = residual_weights(*laws[L])
        else:
            w, _ = truncated_weights(target[lo + b][:vocab], *target_settings[r])
        out["tokens"][r, :L] = draft_tokens[r][:L]
        out["tokens"][r, L] = inverse_cdf(w, uv[L][1])
        out["accepted"][r] = L
    return out
