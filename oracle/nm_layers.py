"""CPU oracle for the operators beside an N:M projection: layer norm, low-rank
adapters and softmax cross entropy, with their gradients.

TEST INFRASTRUCTURE ONLY.  Like nm_oracle, this module exists to check the GPU
library and shares no code with the HIP path.  Everything is computed from the
definitions in float64 on plain arrays (inputs already widened from their
storage type); the gradients are pinned against central differences of the
forward functions and against hand-worked values by tests/test_oracle_layers.py.
"""
from __future__ import annotations

import numpy as np


def layernorm_ref(x, weight=None, bias=None, eps=1e-5):
    """(y, mean, rstd) of each row of x [T, H]."""
    mean = x.mean(axis=1)
    rstd = 1.0 / np.sqrt(((x - mean[:, None]) ** 2).mean(axis=1) + eps)
    y = (x - mean[:, None]) * rstd[:, None]
    if weight is not None:
        y = y * weight
    if bias is not None:
        y = y + bias
    return y, mean, rstd


def layernorm_bwd_ref(dy, x, mean, rstd, weight=None):
    """(dx, dw, db) from dy = dL/dy and the forward pass's statistics."""
    xh = (x - mean[:, None]) * rstd[:, None]
    p = dy if weight is None else dy * weight
    dx = rstd[:, None] * (p - p.mean(axis=1)[:, None] - xh * (p * xh).mean(axis=1)[:, None])
    return dx, (dy * xh).sum(axis=0), dy.sum(axis=0)


def adapter_ref(w, x, adapter, A, B, scale):
    """(Y, xa): y_t = W x_t + s B (A x_t) with the token's own adapter, W [R, K] dense
    (the decompressed weight), x [T, K], adapter [T] (an id outside [0, n): none),
    A [n, r, K], B [n, R, r]; xa_t = A x_t, zeros without an adapter."""
    y = x @ w.T
    xa = np.zeros((x.shape[0], A.shape[1]))
    for t, a in enumerate(adapter):
        if 0 <= a < A.shape[0]:
            xa[t] = A[a] @ x[t]
            y[t] += scale[a] * (B[a] @ xa[t])
    return y, xa


def adapter_bwd_ref(w, g, x, xa, adapter, A, B, scale):
    """(dX, dA, dB) from g = dL/dY [T, R] and xa of the forward pass."""
    dx = g @ w
    dA, dB = np.zeros_like(A), np.zeros_like(B)
    for t, a in enumerate(adapter):
        if 0 <= a < A.shape[0]:
            u = scale[a] * (g[t] @ B[a])
            dx[t] += u @ A[a]
            dA[a] += np.outer(u, x[t])
            dB[a] += scale[a] * np.outer(g[t], xa[t])
    return dx, dA, dB


def xent_ref(x, w, labels):
    """(loss, lse) per token of logits x w^T, x [T, H], w [V, H]; a label outside
    [0, V) carries no loss."""
    logits = x @ w.T
    top = logits.max(axis=1)
    lse = top + np.log(np.exp(logits - top[:, None]).sum(axis=1))
    loss = np.zeros(x.shape[0])
    for t, v in enumerate(labels):
        if 0 <= v < w.shape[0]:
            loss[t] = lse[t] - logits[t, v]
    return loss, lse


def xent_bwd_ref(x, w, labels, dloss):
    """(dx, dw) from dloss = dL/dloss [T]: d = dloss (softmax - onehot), zeros for a
    token without loss; dx = d w, dw = d^T x."""
    logits = x @ w.T
    e = np.exp(logits - logits.max(axis=1)[:, None])
    d = e / e.sum(axis=1)[:, None]
    for t, v in enumerate(labels):
        if 0 <= v < w.shape[0]:
            d[t, v] -= 1.0
            d[t] *= dloss[t]
        else:
            d[t] = 0.0
    return d @ w, d.T @ x
