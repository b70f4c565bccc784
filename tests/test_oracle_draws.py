"""Which uniforms a draft may be drawn from (CPU)."""

import numpy as np

from oracle.truncate import sample_row
from oracle.verify import accept


def emitted(u_draw, u_test):
    """How often the first of two ids comes out, by exact counting over grids of uniforms: p =
    (1/2, 1/2), q = (3/4, 1/4); a draft of id 0 is rejected into id 1 (the residual's only id),
    a draft of id 1 is always accepted."""
    q = np.log(np.array([0.75, 0.25]))
    first = 0
    for a, b in zip(u_draw, u_test):
        d = sample_row(q, a)[0]
        first += d == 0 and accept(b, 0.5, 0.75)
    return first / len(u_draw)


def test_drafts_need_uniforms_of_their_own():
    """Independent numbers leave the target's law, 1/2; the draft's own number as the test's
    number does not: id 0 comes out wherever u < 2/3."""
    n = 48
    grid = (np.arange(n) + 0.5) / n
    a, b = np.repeat(grid, n), np.tile(grid, n)
    assert emitted(a, b) == 0.5
    assert emitted(grid, grid) == 2 / 3
