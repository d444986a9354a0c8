"""Pins of the sampling oracle (CPU): closed forms and counts worked by hand."""
import numpy as np
import pytest

from oracle import sampling as so


def test_order_is_by_logit_then_by_index():
    order, w = so.row_distribution([1.0, 3.0, 3.0, 2.0])
    assert order.tolist() == [1, 2, 3, 0]
    assert np.allclose(w, [1, 1, np.exp(-1), np.exp(-2)], rtol=1e-15)


@pytest.mark.parametrize("settings,kept", [
    (dict(top_k=2), [0, 1]), (dict(top_k=9), [0, 1, 2, 3]), (dict(top_k=-1), [0, 1, 2, 3]),
    (dict(min_p=0.5), [0, 1]), (dict(min_p=0.51), [0]), (dict(min_p=2.0), [0]), (dict(min_p=-1.0), [0, 1, 2, 3]),
    (dict(top_p=0.5), [0]), (dict(top_p=8 / 15 + 1e-9), [0, 1]), (dict(top_p=0.8), [0, 1]), (dict(top_p=0.0), [0]),
    (dict(top_k=2, top_p=0.66), [0]), (dict(top_k=2, top_p=0.67), [0, 1]), (dict(temperature=0.0), [0]),
])
def test_kept_tokens_of_halving_weights(settings, kept):
    """Weights 8, 4, 2, 1 of 15."""
    order, w = so.row_distribution(np.log([8.0, 4.0, 2.0, 1.0]) + 1e-13 * np.array([0, 1, 0, 0]), **settings)
    assert [t for t, x in zip(order.tolist(), w) if x > 0] == kept


def test_draw_takes_the_first_whose_running_weight_is_above():
    order, w = so.row_distribution([0.0, 0.0, 0.0, 0.0])
    assert [so.draw(order, w, u) for u in (0.0, 0.24999, 0.25, 0.5, 0.999999)] == [0, 0, 1, 2, 3]


def test_rows_without_a_distribution():
    inf = np.inf
    for x, s in (([np.nan, 1], {}), ([-inf, -inf], {}), ([1, 2], dict(temperature=-1.0)),
                 ([1, 2], dict(temperature=np.nan)), ([1, 2], dict(top_p=np.nan))):
        assert so.sample(x, 0.5, **s)[0] == -1
    assert so.sample([1, 2], 1.0)[0] == -1
    assert so.sample([1, inf, inf, 2], 0.6)[0] == 2 and so.sample([1, inf, inf, 2], 0.6)[1] == 0.5


def test_accept_keeps_the_target_distribution():
    """Over a fine grid of both random numbers the token after one draft is distributed as p, whatever q is."""
    p = np.array([0.5, 0.3, 0.2])
    x = np.log(p)
    q = np.array([0.2, 0.2, 0.6])
    n = 200
    grid = (np.arange(n) + 0.5) / n
    got = np.zeros(3)
    for draft in range(3):
        for u in grid:
            if so.accept(np.stack([x, x]), [0, draft], [u, 0.0], 0.5, q=[q, q])[0] == 1:
                got[draft] += q[draft] / n
                continue
            for v in grid[::10]:
                got[so.accept(np.stack([x, x]), [0, draft], [u, 0.0], v, q=[q, q])[1]] += q[draft] / n * 10 / n
    assert np.abs(got - p).max() < 0.02


def test_accept_of_certain_drafts():
    x = np.log(np.array([[0.5, 0.3, 0.2]] * 3))
    assert so.accept(x, [0, 0, 1], [0.49, 0.29, 0.9], 0.6) == (2, 1)     # both stay, then a draw from p
    assert so.accept(x, [0, 0, 1], [0.49, 0.31, 0.9], 0.72) == (1, 2)    # rest after 1: 0.5, 0, 0.2
    assert so.accept(x, [0, 7, 1], [0.0, 0.0, 0.0], 0.0) == (0, 0)       # outside the vocabulary
    assert so.accept(x[:1], [0], [0.0], 0.9) == (0, 2)
    assert so.accept(x[:0], [], [], 0.9) == (0, -1)
