"""fp64 CPU oracle of the training operators around the attention core: layer
norm, the GAU projections' gradients and the vocabulary's softmax cross entropy.

TEST INFRASTRUCTURE ONLY (as the rest of ``oracle/``).  Plain numpy in 64 bits,
each gradient written out from its formula; the tests also check the formulas
against central differences of the forward functions here.
"""
from __future__ import annotations

import numpy as np


def f64(a):
    return np.asarray(a, dtype=np.float64)


def layer_norm(h, weight, bias, eps):
    """(y, xhat, mean, rstd) of rows h [M, d]."""
    h = f64(h)
    mean = h.mean(1)
    c = h - mean[:, None]
    rstd = 1.0 / np.sqrt((c * c).mean(1) + eps)
    xhat = c * rstd[:, None]
    return xhat * f64(weight) + f64(bias), xhat, mean, rstd


def layer_norm_backward(dy, h, weight, eps, dh=None):
    """(dx, dweight, dbias) of sum(y * dy) + sum(h * dh)."""
    dy = f64(dy)
    _, xhat, _, rstd = layer_norm(h, weight, np.zeros(np.shape(h)[1]), eps)
    t = dy * f64(weight)
    dx = rstd[:, None] * (t - t.mean(1, keepdims=True)
                          - xhat * (t * xhat).mean(1, keepdims=True))
    if dh is not None:
        dx = dx + f64(dh)
    return dx, (dy * xhat).sum(0), dy.sum(0)


def gau_project_backward(X, Wt, dU, dV, dZ):
    """(dX, dWt, dpre) for [U|V|Z] = silu(X Wt^T)."""
    X, Wt = f64(X), f64(Wt)
    pre = X @ Wt.T
    sig = 1.0 / (1.0 + np.exp(-pre))
    dpre = np.concatenate([f64(dU), f64(dV), f64(dZ)], 1) * sig * (1.0 + pre * (1.0 - sig))
    return dpre @ Wt, dpre.T @ X, dpre


def gau_output_backward(Y, Wo_t, dOut):
    """(dY, dWo_t) for Out = Y Wo_t^T."""
    dOut = f64(dOut)
    return dOut @ f64(Wo_t), dOut.T @ f64(Y)


def vocab_loss(X, W, target):
    """(loss, lse) per row; rows whose target is outside 0 .. V - 1 get 0, and
    their X is not looked at."""
    X, W, target = f64(X), f64(W), np.asarray(target)
    loss, lse = np.zeros(len(target)), np.zeros(len(target))
    rows = np.flatnonzero((target >= 0) & (target < len(W)))
    z = X[rows] @ W.T
    if len(rows):
        top = z.max(1)
        lse[rows] = top + np.log(np.exp(z - top[:, None]).sum(1))
        loss[rows] = lse[rows] - z[np.arange(len(rows)), target[rows]]
    return loss, lse


def vocab_loss_backward(X, W, target, dloss):
    """(dX, dW) of sum(loss * dloss) over the rows that have a target."""
    X, W, target = f64(X), f64(W), np.asarray(target)
    rows = np.flatnonzero((target >= 0) & (target < len(W)))
    dX, dW = np.zeros_like(X), np.zeros_like(W)
    if len(rows):
        z = X[rows] @ W.T
        p = np.exp(z - z.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
        p[np.arange(len(rows)), target[rows]] -= 1.0
        p *= f64(dloss)[rows, None]
        dX[rows] = p @ W
        dW = p.T @ X[rows]
    return dX, dW
