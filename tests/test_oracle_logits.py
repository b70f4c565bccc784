"""Pins of the oracle's histories and adjusted logits: rows worked out by hand."""

import numpy as np

from oracle.logits import DEV_BAD_SLOT, DEV_BAD_TOKEN, adjust_row, bits_of, history_add


def test_history_counts_by_hand():
    counts = np.zeros((2, 5), np.int32)
    assert history_add(counts, [1], [[3, 3, -1, 0]], True) == 0
    assert counts.tolist() == [[0] * 5, [1, 0, 0, 1, 0]]
    assert history_add(counts, [1, 0], [[3, 3, 4], [-1, 2, 2]], False) == 0
    assert counts.tolist() == [[0, 0, 4, 0, 0], [1, 0, 0, 5, 2]]
    # the prompt's mark stays and is set once
    assert history_add(counts, [1], [[4, 3]], True) == 0
    assert counts[1].tolist() == [1, 0, 0, 5, 3]


def test_history_errors():
    counts = np.zeros((1, 3), np.int32)
    assert history_add(counts, [0, 1, -1], [[3, 1], [0, 0], [0, 0]], False) == \
        DEV_BAD_TOKEN | DEV_BAD_SLOT
    assert counts.tolist() == [[0, 2, 0]]


def test_adjusted_row_by_hand():
    z = [2.0, -2.0, 4.0, 1.0, 0.0, -1.0]
    held = np.array([1, 1, 5, 2, 0, 0])  # prompt, prompt, prompt and twice, once, -, -
    got, _ = adjust_row(z, held, [], repetition=2.0, frequency=0.25, presence=0.5)
    assert got.tolist() == [1.0, -4.0, 2.0 - 0.5 - 0.5, 0.5 - 0.25 - 0.5, 0.0, -1.0]
    # drafts before the row count as said: id 0 once, id 5 twice
    got, _ = adjust_row(z, held, [0, 5, 5], repetition=2.0, frequency=0.25, presence=0.5)
    assert got.tolist() == [1.0 - 0.75, -4.0, 1.0, -0.25, 0.0, -2.0 - 0.5 - 0.5]
    assert held.tolist() == [1, 1, 5, 2, 0, 0]


def test_biases_and_masks_by_hand():
    got, _ = adjust_row([1.0, 2.0, 3.0], np.zeros(3, int), [], bias=[(0, 4.0), (2, -np.inf)],
                        allowed=[True, False, True])
    assert got.tolist() == [5.0, -np.inf, -np.inf]
    # a bias does not bring back what the grammar forbids
    got, _ = adjust_row([1.0, 2.0], np.zeros(2, int), [], bias=[(1, 100.0)], allowed=[True, False])
    assert got.tolist() == [1.0, -np.inf]


def test_infinities_and_nan_pass_through():
    got, _ = adjust_row([np.inf, -np.inf, np.nan], np.full(3, 2), [], repetition=1.5, frequency=1.0)
    assert got[0] == np.inf and got[1] == -np.inf and np.isnan(got[2])


def test_bits():
    assert bits_of([True] + [False] * 30 + [True, True]).tolist() == [1 - 2 ** 31, 1]
