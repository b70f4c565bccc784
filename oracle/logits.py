"""Histories and adjusted logits — oracle side (test infrastructure).

FOS page, section "속도, 메모리, 정확도에 주는 영향", row 정확도: the output law is the
target's; a request served with penalties, biases or a grammar has the adjusted
law as its target.  The pages do not spell the adjustments out: their form and
order (repetition, frequency and presence, bias, mask) are this library's choice, id
by id, the drafts before a row counted as said.  fp64.
"""

import numpy as np

DEV_BAD_CU_ROWS, DEV_BAD_TOKEN, DEV_BAD_PARAM, DEV_BAD_SLOT = 1, 2, 256, 512


def history_add(counts, slots, tokens, in_prompt):
    """Adds rows of ids to counts [n_slots, vocab] in place; returns the error bits."""
    err = 0
    for s, row in zip(slots, tokens):
        if not 0 <= s < len(counts):
            err |= DEV_BAD_SLOT
            continue
        for x in row:
            if 0 <= x < counts.shape[1]:
                counts[s, x] = counts[s, x] | 1 if in_prompt else counts[s, x] + 2
            elif x != -1:
                err |= DEV_BAD_TOKEN
    return err


def adjust_row(z, held, drafts, repetition=1.0, frequency=0.0, presence=0.0, bias=(), allowed=None):
    """(adjusted row, sum of the sizes of what was added up for each id).

    held [vocab]: 2 * (times emitted) + (in the prompt); drafts: those before the row;
    bias: (id, value) pairs; allowed [vocab] truth values or None."""
    z = np.asarray(z, np.float64).copy()
    size = np.abs(z)
    rho, phi, pi = (float(np.float32(v)) for v in (repetition, frequency, presence))
    said = np.asarray(held) // 2
    known = np.asarray(held) > 0
    for d in drafts:
        said[d] += 1
        known[d] = True
    with np.errstate(invalid="ignore"):
        for x in np.flatnonzero(known):
            z[x] = z[x] / rho if z[x] > 0 else z[x] * rho
            size[x] = max(size[x], abs(z[x]))
            if said[x] > 0:
                z[x] = z[x] - phi * said[x] - pi
                size[x] += abs(phi * said[x]) + abs(pi)
        for x, b in bias:
            z[x] += float(np.float32(b))
            size[x] += abs(float(np.float32(b)))
    if allowed is not None:
        z[~np.asarray(allowed, bool)] = -np.inf
    return z, size


def bits_of(allowed):
    """Truth values [vocab] as words of 32 bits, id x bit x % 32 of word x // 32."""
    allowed = np.asarray(allowed, bool)
    words = np.zeros((len(allowed) + 31) // 32, np.uint32)
    for x in np.flatnonzero(allowed):
        words[x // 32] |= np.uint32(1 << (x % 32))
    return words.view(np.int32)
