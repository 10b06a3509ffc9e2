"""The page selection's search for the smallest kept score, modelled on the CPU
and held to a sort, with scores on both sides of its parts' ends."""
import numpy as np
import pytest

from select_model import (Picked, border_wants, kept, order_keys, scores_across_an_end, scores_below_one_far_above,
                          sorted_kept)

BINS = pytest.mark.parametrize("bins", [1024, 2048])


def test_keys_order_like_the_scores():
    x = np.array([-np.inf, -3e38, -1.0, -2.0 ** -149, -0.0, 0.0, 2.0 ** -149, 1.0, 3e38, np.inf, np.nan], np.float32)
    k = order_keys(x)
    assert (np.diff(k) >= 0).all() and (np.diff(k) == 0).tolist() == [False] * 4 + [True] + [False] * 5


# close: the scores in the last piece of their part's keys, ranked (up to 256) or counted by keys again
@BINS
@pytest.mark.parametrize("close,equal", [(3, 5), (3, 800), (200, 5), (200, 200), (400, 5), (400, 800), (3000, 30)])
def test_scores_across_a_parts_end(bins, close, equal):
    x = scores_across_an_end(997 + close + equal, bins, close, equal, close + equal)
    wants = border_wants(x, bins)
    assert len(wants) == close or (close == 3000 and len(wants) > 1000)   # (of 2048 parts the last piece holds fewer)
    for want in sorted({*wants[:4], *wants[-3:], wants[len(wants) // 2], wants[0] - 1, wants[-1] + 1}):
        assert np.array_equal(kept(x, want, bins), sorted_kept(x, want)), want
    # pieces that reach past the part's end pick or count scores of the next part
    wrong = 0
    for want in wants:
        try:
            wrong += not np.array_equal(kept(x, want, bins, cut_at_end=False), sorted_kept(x, want))
        except Picked:
            wrong += 1
    assert wrong >= len(wants) - 1                 # (all of them kept: nothing to rank)


@BINS
@pytest.mark.parametrize("n", [2000, 9000])
def test_scores_below_one_far_above(bins, n):
    met = 0
    for seed in range(20):
        x = scores_below_one_far_above(n, seed)
        wants = border_wants(x, bins)
        met += len(wants)
        for want in [*wants, 1, 2, n // 8, n // 2, n - 1]:
            assert np.array_equal(kept(x, want, bins), sorted_kept(x, want)), (seed, want)
    assert met > 0


@BINS
def test_every_number_of_kept_scores(bins):
    rng = np.random.default_rng(1)
    n = 700
    at = np.arange(n)
    rows = [rng.standard_normal(n), np.zeros(n), np.round(rng.standard_normal(n) * 2), 1.0 + at * 2.0 ** -23,
            np.where(at % 5 == 0, np.nan, at), np.where(at % 3 == 0, -np.inf, at), np.where(at < 350, 1e30, -1e30),
            np.where(at < 350, 3e38, -3e38), np.where(at % 2 == 0, 0.0, -0.0), 2.0 ** (at % 250 - 125.0),
            scores_across_an_end(n, bins, 3, 50, 2)]
    for i, row in enumerate(rows):
        x = row.astype(np.float32)
        for want in range(1, n):
            assert np.array_equal(kept(x, want, bins), sorted_kept(x, want)), (i, want)
