"""CPU oracle for products grouped by expert, microscaled 4-bit floats and the
global norm of gradients.

TEST INFRASTRUCTURE ONLY.  Like nm_oracle, this module exists to check the GPU
library and shares no code with the HIP path.  Everything is computed from the
definitions in float64 on plain arrays; tests/test_oracle_experts.py pins it by
hand-worked values, by searching all sixteen representable values, and against
central differences.
"""
from __future__ import annotations

import numpy as np

from . import nm_oracle as O
from . import nm_train as N

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def rows_of(offsets, T):
    """[(lo, hi)] of each expert: its offsets clamped into [0, T], one by one, hi >= lo."""
    out = []
    for a, b in zip(offsets[:-1], offsets[1:]):
        lo = min(max(int(a), 0), T)
        out.append((lo, min(max(int(b), lo), T)))
    return out


def group_ref(values, idx, K, n, m, act_bits, offsets, dtype):
    """(Y, size, owned): Y[t] = W_e act[t], the sum of the magnitudes it is made of, and the rows
    that belong to an expert.  values, idx: E packed weights (bits, words)."""
    x = O.half_bits_to_f64(act_bits, dtype)
    y = np.zeros((x.shape[0], values.shape[1]))
    size, owned = np.zeros_like(y), np.zeros(x.shape[0], dtype=bool)
    for e, (lo, hi) in enumerate(rows_of(offsets, x.shape[0])):
        if lo < hi:
            w = O.half_bits_to_f64(O.decompress(values[e], idx[e], K, n, m), dtype)
            y[lo:hi], size[lo:hi], owned[lo:hi] = x[lo:hi] @ w.T, np.abs(x[lo:hi]) @ np.abs(w).T, True
    return y, size, owned


def group_dx_ref(values, idx, K, n, m, g_bits, offsets, dtype):
    """(dX, size, owned): dX[t] = W_e^T G[t]."""
    g = O.half_bits_to_f64(g_bits, dtype)
    dx = np.zeros((g.shape[0], K))
    size, owned = np.zeros_like(dx), np.zeros(g.shape[0], dtype=bool)
    for e, (lo, hi) in enumerate(rows_of(offsets, g.shape[0])):
        if lo < hi:
            w = O.half_bits_to_f64(O.decompress(values[e], idx[e], K, n, m), dtype)
            dx[lo:hi], size[lo:hi], owned[lo:hi] = g[lo:hi] @ w, np.abs(g[lo:hi]) @ np.abs(w), True
    return dx, size, owned


def group_dw_ref(idx, K, n, m, g_bits, act_bits, offsets, dtype):
    """(dW, size): dW[e, r, s] = sum over e's rows of G[t, r] act[t, k(r, s)]."""
    g, x = O.half_bits_to_f64(g_bits, dtype), O.half_bits_to_f64(act_bits, dtype)
    dw = np.zeros((idx.shape[0], idx.shape[1], K // m * n))
    size = np.zeros_like(dw)
    for e, (lo, hi) in enumerate(rows_of(offsets, g.shape[0])):
        col = N.stored_columns(idx[e], K, n, m)
        dw[e] = np.take_along_axis(g[lo:hi].T @ x[lo:hi], col, 1)
        size[e] = np.take_along_axis(np.abs(g[lo:hi]).T @ np.abs(x[lo:hi]), col, 1)
    return dw, size


def mx_quantize_ref(x):
    """(codes [T, K] of 4 bits, bytes [T, K / 32]) of x [T, K] (float64 holding the stored values)."""
    b = x.reshape(x.shape[0], -1, 32)
    finite = np.isfinite(b).all(axis=2)
    top = np.where(finite, np.abs(np.where(np.isfinite(b), b, 0.0)).max(axis=2), 0.0)
    _, e = np.frexp(top)                      # top = m 2^e, m in [.5, 1): floor(log2 top) = e - 1
    byte = np.where(top > 0, np.maximum(e - 1 - 2 + 127, 0), 0)
    byte = np.where(finite, byte, 255)
    a = np.abs(np.where(finite[:, :, None], b, 0.0)) / 2.0 ** (byte[:, :, None].astype(np.float64) - 127)
    near = np.abs(np.minimum(a, 6.0)[..., None] - E2M1)
    # ties go to the even mantissa bit: an even code
    code = np.argmin(near + 1e-9 * (np.arange(8) % 2) * (near == near.min(axis=3, keepdims=True)), axis=3)
    code = code + 8 * (np.signbit(b) & finite[:, :, None])
    return code.reshape(x.shape).astype(np.uint8), byte.astype(np.uint8)


def mx_values_ref(code, byte):
    """The values [T, K] of codes and exponent bytes."""
    mag = np.where(code >= 8, -1.0, 1.0) * E2M1[code & 7]
    scale = np.where(byte == 255, np.nan, 2.0 ** (byte.astype(np.float64) - 127))
    with np.errstate(invalid="ignore"):
        return (mag.reshape(code.shape[0], -1, 32) * scale[:, :, None]).reshape(code.shape)


def mx_pack_ref(code, byte):
    """q [T, K / 2] and scale [ceil(K / 256), T, 8] of the stored format."""
    panels = np.pad(byte, ((0, 0), (0, -byte.shape[1] % 8))).reshape(code.shape[0], -1, 8)
    return code[:, 0::2] | (code[:, 1::2] << 4), np.ascontiguousarray(panels.transpose(1, 0, 2))


def grad_clip_ref(grads, max_norm, eps):
    """(norm, scaled gradients) of a list of float64 arrays."""
    norm = np.sqrt(sum((g.astype(np.longdouble) ** 2).sum() for g in grads)) if grads else np.longdouble(0)
    ratio = np.longdouble(max_norm) / (norm + eps) if norm + eps != 0 else np.longdouble(1)
    coef = ratio if np.isnan(ratio) else min(np.longdouble(1), ratio)
    with np.errstate(invalid="ignore"):
        return float(norm), [(g * coef).astype(np.float64) for g in grads]
