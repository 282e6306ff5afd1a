"""The float64 distillation oracle itself: its gradients against differences of its
losses, a worked row, and that a mistake in either would show."""
import numpy as np
import pytest

import distill_oracle as do


def make(seed, n=12, k=4):
    r = np.random.RandomState(seed)
    x = r.randn(n)
    ids = r.choice(n, k, replace=False)
    return r, x, ids, r.randn(k)


@pytest.mark.parametrize("seed", range(4))
@pytest.mark.parametrize("rest", [False, True])
def test_gradient_is_that_of_the_loss(seed, rest):
    r, x, ids, t = make(seed)
    tau = 0.7
    lse = np.log(np.exp(t / tau).sum()) + 0.4 if rest else None
    _, g, _, _ = do.row(x, ids, t, tau, lse)
    h = 1e-5
    for j in range(len(x)):
        up, dn = x.copy(), x.copy()
        up[j] += h
        dn[j] -= h
        diff = (do.row(up, ids, t, tau, lse)[0] - do.row(dn, ids, t, tau, lse)[0]) / (2 * h)
        # central differences: h^2 / 6 of a third derivative below 6 / tau^3, and rounding
        assert abs(diff - g[j]) <= h * h / tau**3 + 1e-10
    assert abs(g.sum()) < 1e-12
    # a gradient that forgot the list would be off by far more
    wrong = g.copy()
    wrong[ids[0]] = 0
    assert abs(wrong.sum()) > 1e-3


def test_worked_row():
    # two columns listed of three, equal scores: q = 1/3; teacher 3/4, 1/4
    x, ids, t = np.zeros(3), [2, 0], np.log([3.0, 1.0])
    loss, g, _, _ = do.row(x, ids, t, 1.0)
    p = np.array([0.75, 0.25])
    assert np.isclose(loss, (p * (np.log(p) + np.log(3))).sum())
    assert np.allclose(g, [1 / 3 - 0.25, 1 / 3, 1 / 3 - 0.75])
    # with a tenth of the mass outside
    loss, g, _, _ = do.row(x, ids, t, 1.0, np.log(4 / 0.9))
    assert np.isclose(loss, (0.9 * p * (np.log(0.9 * p) + np.log(3))).sum()
                      + 0.1 * (np.log(0.1) + np.log(3)))
    assert np.allclose(g, [1 / 3 - 0.225, 1 / 3 - 0.1, 1 / 3 - 0.675])


def test_entries_that_take_no_part():
    x = np.array([0.1, 0.4, -0.3, 0.2])
    want = do.row(x, [3, 1], [0.5, 0.1], 0.5)
    got = do.row(x, [-1, 3, 9, 3, 2, 1, 1], [5.0, 0.5, 5.0, 7.0, -np.inf, 0.1, 3.0], 0.5)
    assert np.isclose(want[0], got[0]) and np.allclose(want[1], got[1])
    assert do.row(x, [-1, 4], [1.0, 1.0], 0.5)[0] == 0
    assert do.row(np.full(4, -np.inf), [1], [1.0], 0.5)[0] == 0
