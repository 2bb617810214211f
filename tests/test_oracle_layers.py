"""Pins of the oracle for layer norm, adapters and cross entropy: hand-worked
values and central differences of the forward functions."""
import numpy as np
import pytest

from oracle import nm_layers as L

# central differences in float64 with step h: truncation h^2/6 |f'''| and
# rounding 2^-52 |f| / h; with h = 1e-5 and |f|, |f'''| up to about 1e2 both stay
# below 1e-8, checked at 1e-6
STEP, TOL = 1e-5, 1e-6


def differences(f, a):
    """Gradient of the scalar f at array a by central differences."""
    g = np.zeros_like(a)
    for i in np.ndindex(a.shape):
        keep = a[i]
        a[i] = keep + STEP
        up = f()
        a[i] = keep - STEP
        down = f()
        a[i] = keep
        g[i] = (up - down) / (2 * STEP)
    return g


def test_layernorm_worked_row():
    # mean 2, variance 1 (eps 0): (1 - 2, 3 - 2, 1 - 2, 3 - 2)
    y, mean, rstd = L.layernorm_ref(np.array([[1.0, 3.0, 1.0, 3.0]]), eps=0.0)
    assert np.array_equal(y, [[-1.0, 1.0, -1.0, 1.0]]) and mean[0] == 2.0 and rstd[0] == 1.0
    y, _, rstd = L.layernorm_ref(np.full((1, 3), 5.0), np.full(3, 2.0), np.arange(3.0), eps=0.25)
    assert np.array_equal(y, [[0.0, 1.0, 2.0]]) and rstd[0] == 2.0


def test_layernorm_gradient_against_differences():
    rng = np.random.default_rng(0)
    x, dy = rng.normal(size=(3, 7)), rng.normal(size=(3, 7))
    w, b = rng.normal(size=7), rng.normal(size=7)
    f = lambda: float((L.layernorm_ref(x, w, b)[0] * dy).sum())
    _, mean, rstd = L.layernorm_ref(x, w, b)
    dx, dw, db = L.layernorm_bwd_ref(dy, x, mean, rstd, w)
    for got, a in ((dx, x), (dw, w), (db, b)):
        assert np.abs(got - differences(f, a)).max() < TOL


def test_adapter_worked_values():
    w = np.array([[1.0, 2.0]])
    x = np.array([[3.0, 4.0], [3.0, 4.0], [3.0, 4.0]])
    A = np.array([[[1.0, 1.0]], [[0.0, 2.0]]])
    B = np.array([[[10.0]], [[1.0]]])
    y, xa = L.adapter_ref(w, x, [0, 1, -1], A, B, np.array([0.5, 3.0]))
    assert np.array_equal(xa[:, 0], [7.0, 8.0, 0.0])
    assert np.array_equal(y[:, 0], [11 + 0.5 * 70, 11 + 3 * 8, 11.0])


def test_adapter_gradient_against_differences():
    rng = np.random.default_rng(1)
    T, R, K, r, n = 5, 4, 6, 3, 3
    w, x, g = rng.normal(size=(R, K)), rng.normal(size=(T, K)), rng.normal(size=(T, R))
    A, B, s = rng.normal(size=(n, r, K)), rng.normal(size=(n, R, r)), rng.normal(size=n)
    ids = [0, 2, -1, 2, 7]
    f = lambda: float((L.adapter_ref(w, x, ids, A, B, s)[0] * g).sum())
    _, xa = L.adapter_ref(w, x, ids, A, B, s)
    dx, dA, dB = L.adapter_bwd_ref(w, g, x, xa, ids, A, B, s)
    for got, a in ((dx, x), (dA, A), (dB, B)):
        assert np.abs(got - differences(f, a)).max() < TOL
    assert not dA[1].any() and not dB[1].any()     # no token uses adapter 1


def test_xent_worked_values():
    # logits (0, ln 3): probabilities 1/4, 3/4
    x, w = np.array([[1.0], [1.0]]), np.array([[0.0], [np.log(3.0)]])
    loss, lse = L.xent_ref(x, w, [0, -100])
    assert np.allclose(loss, [np.log(4.0), 0.0]) and np.allclose(lse, np.log(4.0))
    dx, dw = L.xent_bwd_ref(x, w, [0, -100], np.array([2.0, 2.0]))
    assert np.allclose(dw[:, 0], [2 * (0.25 - 1), 2 * 0.75])
    assert np.allclose(dx[:, 0], [2 * 0.75 * np.log(3.0), 0.0])


def test_xent_gradient_against_differences():
    rng = np.random.default_rng(2)
    x, w, g = rng.normal(size=(5, 4)), rng.normal(size=(9, 4)), rng.normal(size=5)
    labels = [3, 0, -100, 8, 9]
    f = lambda: float((L.xent_ref(x, w, labels)[0] * g).sum())
    dx, dw = L.xent_bwd_ref(x, w, labels, g)
    for got, a in ((dx, x), (dw, w)):
        assert np.abs(got - differences(f, a)).max() < TOL
