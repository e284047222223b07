"""Pins of the rotation oracle that do not re-type its formula: the relative
property, kept lengths, a hand-made case, and differences for the gradient."""
import numpy as np
import pytest

from oracle import rope as orope


def test_scores_depend_on_position_differences_only():
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((2, 1, 1, 12))
    tabs = [orope.axis_angles(40, 2), orope.axis_angles(40, 2), orope.axis_angles(40, 1)]
    for pairing in ("adjacent", "split"):
        def score(a, b):
            ya = orope.turn(q, orope.token_angles(tabs, np.array([a]), 12), pairing)
            yb = orope.turn(k, orope.token_angles(tabs, np.array([b]), 12), pairing)
            return float((ya * yb).sum())
        base = score((3, 5, 7), (9, 2, 8))
        assert score((13, 25, 17), (19, 22, 18)) == pytest.approx(base, abs=1e-12)
        assert abs(score((3, 5, 7), (9, 3, 8)) - base) > 1e-6


def test_quarter_turn_by_hand():
    # one axis, one pair: position p turns by p; start and step make it pi/2
    ang = orope.axis_angles(2, 1, start=np.pi / 2, step=np.pi / 2)
    assert ang[:, 0] == pytest.approx([np.pi / 2, np.pi])
    x = np.array([[[1.0, 2.0, 5.0, 7.0]]])
    a = orope.token_angles([ang], np.array([[0, -1, -1]]), 4)
    assert orope.turn(x, a, "adjacent")[0, 0] == pytest.approx([-2.0, 1.0, 5.0, 7.0])
    assert orope.turn(x, a, "split")[0, 0] == pytest.approx([-5.0, 2.0, 1.0, 7.0])


def test_grid_positions_and_tail():
    pos = orope.grid_positions((2, 2, 3), (1, 0, 4), 14)
    assert pos[0].tolist() == [1, 0, 4] and pos[5].tolist() == [1, 1, 6] and pos[11].tolist() == [2, 1, 6]
    assert (pos[12:] == -1).all()


def test_norm_gives_unit_rows():
    rng = np.random.default_rng(2)
    x = rng.standard_normal((5, 3, 8)) * 10
    y = orope.norm_turn(x, np.ones(8), rng.standard_normal((5, 4)), "split", 0.0)
    assert (y * y).mean(-1) == pytest.approx(np.ones((5, 3)))


@pytest.mark.parametrize("pairing", ["adjacent", "split"])
def test_gradient_against_differences(pairing):
    rng = np.random.default_rng(3)
    x, gy = rng.standard_normal((2, 3, 2, 8))
    w = 1 + 0.3 * rng.standard_normal(8)
    ang = rng.standard_normal((3, 4))
    f = lambda x, w: float((orope.norm_turn(x, w, ang, pairing, 1e-3) * gy).sum())  # noqa: E731
    dx, dw = orope.norm_turn_back(gy, x, w, ang, pairing, 1e-3)
    e = 1e-5
    for at in [(0, 0, 0), (1, 1, 3), (2, 0, 7)]:
        d = np.zeros_like(x)
        d[at] = e
        assert (f(x + d, w) - f(x - d, w)) / (2 * e) == pytest.approx(dx[at], abs=1e-8)
    for c in (0, 5):
        d = np.zeros_like(w)
        d[c] = e
        assert (f(x, w + d) - f(x, w - d)) / (2 * e) == pytest.approx(dw[c], abs=1e-8)
