"""Pins of the fp64 definitions in oracle/lm.py (CPU): closed forms and
central finite differences of every gradient."""
import numpy as np
import pytest

from oracle import lm


def rng(seed):
    return np.random.default_rng(seed)


def fd(f, x, eps=1e-6):
    """Central differences of the scalar f over every element of x."""
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        keep = x[i]
        x[i] = keep + eps
        up = f()
        x[i] = keep - eps
        down = f()
        x[i] = keep
        g[i] = (up - down) / (2 * eps)
    return g


def test_layer_norm_rows_have_mean_b_and_deviation_w():
    x = rng(0).normal(size=(5, 40)) * 3 + 7
    y, mean, rstd = lm.layer_norm_fwd(x, None, None, 0.0)
    assert np.allclose(y.mean(-1), 0) and np.allclose((y ** 2).mean(-1), 1)
    assert np.allclose(mean, x.mean(-1)) and np.allclose(1 / rstd, x.std(-1))
    y2, _, _ = lm.layer_norm_fwd(x * 10 - 3, None, None, 0.0)  # a scale and an offset of the row change nothing
    assert np.allclose(y, y2)


def test_layer_norm_of_a_constant_row_is_b():
    b = rng(1).normal(size=6)
    y, _, _ = lm.layer_norm_fwd(np.full((2, 6), 4.0), np.ones(6), b, 1e-5)
    assert np.allclose(y, b)


@pytest.mark.parametrize("D", [1, 2, 7])
def test_layer_norm_gradients_are_the_differences(D):
    r = rng(D)
    x, w, b, dy = r.normal(size=(3, D)), r.normal(size=D), r.normal(size=D), r.normal(size=(3, D))
    f = lambda: float((lm.layer_norm_fwd(x, w, b, 1e-2)[0] * dy).sum())
    _, mean, rstd = lm.layer_norm_fwd(x, w, b, 1e-2)
    dx, dw, db = lm.layer_norm_bwd(x, w, mean, rstd, dy)
    for got, arg in ((dx, x), (dw, w), (db, b)):
        assert np.allclose(got, fd(f, arg), atol=1e-7)


def test_loss_of_equal_logits_is_log_of_the_vocabulary():
    loss, lse = lm.linear_ce_fwd(np.zeros((2, 3)), rng(2).normal(size=(9, 3)), np.array([4, -1]))
    assert np.allclose(lse, np.log(9)) and np.allclose(loss, [np.log(9), 0])


def test_loss_gradients_are_the_differences():
    r = rng(3)
    x, w, dl = r.normal(size=(4, 5)), r.normal(size=(7, 5)), r.normal(size=4)
    t = np.array([0, 6, -100, 3])
    f = lambda: float((lm.linear_ce_fwd(x, w, t)[0] * dl).sum())
    dx, dw = lm.linear_ce_bwd(x, w, t, lm.linear_ce_fwd(x, w, t)[1], dl)
    assert np.allclose(dx, fd(f, x), atol=1e-7)
    assert np.allclose(dw, fd(f, w), atol=1e-7)
    assert np.all(dx[2] == 0)  # a token that is not scored
