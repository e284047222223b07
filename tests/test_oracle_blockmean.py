"""Pins of the block-mean selection oracle: the definition as a mean over the
tile's scores by brute force, ties and neighbourhoods by hand."""
import numpy as np
import pytest

from oracle import blockmean as obm


def test_mean_score_is_the_mean_of_the_tile():
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((2, 11, 1, 3))
    sq, sk = obm.block_sums(q, 4), obm.block_sums(k, 4)
    for i in range(3):
        for j in range(3):
            tile = [float(q[a, 0] @ k[b, 0]) for a in range(4 * i, min(11, 4 * i + 4))
                    for b in range(4 * j, min(11, 4 * j + 4))]
            n = min(4, 11 - 4 * i) * min(4, 11 - 4 * j)
            s = float(sum(a * b for a, b in zip(sq[i][0], sk[j][0]))) / n
            assert s == pytest.approx(np.mean(tile), abs=1e-12)


def test_rows_by_hand():
    assert obm.keep_row([5, 5, 5, 5], 2, 2, -1) == [0, 1]
    assert obm.keep_row([5, 5, 5, 5], 2, 2, 0) == [0, 2]
    assert obm.keep_row([1, 9, 3, 9, 2], 4, 3, 0) == [1, 3, 4]
    assert obm.keep_row([1, 9, 3, 9, 2], 0, 1, 1) == [0, 1]          # the neighbourhood is never cut
    assert obm.keep_row([1, 9], 0, 7, -1) == [0, 1]
    assert obm.keep_row([-1, -float("inf"), -2], 0, 2, -1) == [0, 2]


@pytest.mark.parametrize("keep,local", [(1, -1), (2, 0), (3, 1)])
def test_float64_form_equals_the_exact_one(keep, local):
    rng = np.random.default_rng(2)
    q, k = rng.standard_normal((2, 23, 2, 5)).astype(np.float32).astype(np.float64)
    k[8:12] = k[0:4]                                                  # equal blocks: a tie
    idx, cnt = obm.select(q, k, keep, local, 4)
    want = obm.select_exact(q, k, keep, local, 4)
    for h in range(2):
        for i in range(6):
            assert list(idx[h, i, :cnt[h, i]]) == want[h][i] and (idx[h, i, cnt[h, i]:] == -1).all()
