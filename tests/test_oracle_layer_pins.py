"""Pins of oracle/layer.py (CPU): hand-worked values, and every gradient
against central differences of the forward function."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import gau, layer


def differences(f, x, h=1e-5):
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        a, b = x.copy(), x.copy()
        a[i] += h
        b[i] -= h
        g[i] = (f(a) - f(b)) / (2 * h)
    return g


def close(a, b):
    # central differences with step 1e-5 of functions of size ~10: truncation
    # ~1e-10 f''', rounding ~1e-15 * 10 / 1e-5 = 1e-9
    np.testing.assert_allclose(a, b, rtol=1e-6, atol=1e-7)


def test_layer_norm_by_hand():
    y, xhat, mean, rstd = layer.layer_norm([[1.0, 3.0]], [2.0, 5.0], [0.5, -1.0], 3.0)
    # mean 2, variance 1, rstd 1 / sqrt(4)
    assert mean[0] == 2.0 and rstd[0] == 0.5
    np.testing.assert_allclose(y, [[2.0 * -0.5 + 0.5, 5.0 * 0.5 - 1.0]])


@pytest.mark.parametrize("residual", [False, True])
def test_layer_norm_gradients_are_differences(residual):
    r = np.random.default_rng(3)
    h, dy = r.normal(size=(3, 5)), r.normal(size=(3, 5))
    w, b = r.normal(size=5), r.normal(size=5)
    dh = r.normal(size=(3, 5)) if residual else None

    def total(hh, ww, bb):
        t = (layer.layer_norm(hh, ww, bb, 1e-2)[0] * dy).sum()
        return t + ((hh * dh).sum() if residual else 0.0)
    dx, dw, db = layer.layer_norm_backward(dy, h, w, 1e-2, dh)
    close(dx, differences(lambda a: total(a, w, b), h))
    close(dw, differences(lambda a: total(h, a, b), w))
    close(db, differences(lambda a: total(h, w, a), b))


def test_projection_gradients_are_differences():
    r = np.random.default_rng(4)
    M, d, e, s = 3, 4, 2, 3
    X, Wt = r.normal(size=(M, d)), r.normal(size=(2 * e + s, d))
    up = [r.normal(size=(M, k)) for k in (e, e, s)]

    def total(x, w):
        return sum((o * g).sum() for o, g in zip(gau.gau_project(x, w, e, s), up))
    dX, dWt, _ = layer.gau_project_backward(X, Wt, *up)
    close(dX, differences(lambda a: total(a, Wt), X))
    close(dWt, differences(lambda a: total(X, a), Wt))
    Y, Wo, dOut = r.normal(size=(M, e)), r.normal(size=(d, e)), r.normal(size=(M, d))
    dY, dWo = layer.gau_output_backward(Y, Wo, dOut)
    close(dY, differences(lambda a: (gau.gau_output(a, Wo) * dOut).sum(), Y))
    close(dWo, differences(lambda a: (gau.gau_output(Y, a) * dOut).sum(), Wo))


def test_vocab_loss_by_hand():
    # logits ln 1, ln 2, ln 5: probabilities 1/8, 2/8, 5/8
    W = np.log([[1.0], [2.0], [5.0]])
    loss, lse = layer.vocab_loss([[1.0], [1.0], [1.0]], W, [2, -100, 0])
    np.testing.assert_allclose(loss, [-np.log(5 / 8), 0.0, -np.log(1 / 8)])
    np.testing.assert_allclose(lse, [np.log(8), 0.0, np.log(8)])
    dX, dW = layer.vocab_loss_backward([[1.0], [7.0], [1.0]], W, [2, 3, 1], [2.0, 1e30, 0.0])
    np.testing.assert_allclose(dW[:, 0], 2 * np.array([1 / 8, 2 / 8, 5 / 8 - 1]))
    assert dX[1, 0] == 0.0 and dX[2, 0] == 0.0


def test_vocab_gradients_are_differences():
    r = np.random.default_rng(5)
    X, W = r.normal(size=(4, 3)), r.normal(size=(6, 3))
    target, g = np.array([5, -1, 0, 2]), r.normal(size=4)
    dX, dW = layer.vocab_loss_backward(X, W, target, g)
    close(dX, differences(lambda a: (layer.vocab_loss(a, W, target)[0] * g).sum(), X))
    close(dW, differences(lambda a: (layer.vocab_loss(X, a, target)[0] * g).sum(), W))
