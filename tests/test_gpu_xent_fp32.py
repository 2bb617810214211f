"""Cross entropy's fp32 gradients on MI355X (nm_xent_bwd with fp32 dx or dw) against
the float64 oracle.

Bounds, with u = 2^-23: d = g (p - onehot) is off by |g| p (e + e_lse + (|l - lse| +
4) u) + 2 u |g| as in test_gpu_xent (e = H u sum |x w|).  It enters the products in
two 16-bit parts: each rounds to within 2^-8 (bf16) or 2^-11 (fp16) of what it takes,
so the two are within 2^-16 or 2^-22 of d; fp16 parts also end at 2^-38 of the
largest |g|.  The sums of 2 V or 2 T products add their own u a term.
"""
import ctypes

import numpy as np
import pytest

import structured_sparse_gemm_nm_amd as nm
from oracle import nm_layers as L
from gpu_util import log, to_dev, torch_dtype
from test_gpu_xent import U, f64, host, inputs, within

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

PARTS = {"bf16": 2.0 ** -16, "f16": 2.0 ** -22}


def bounds(X, W, labels, g, dt):
    """(dx, dw) bounds of fp32 outputs."""
    (T, H), V = X.shape, W.shape[0]
    _, lse = L.xent_ref(X, W, labels)
    e = H * U * (np.abs(X) @ np.abs(W).T)
    el = e.max(axis=1) + 64 * U + 2 * U * np.abs(lse)
    keep = (labels >= 0) & (labels < V)
    l = X @ W.T
    p = np.exp(l - lse[:, None])
    d = p.copy()
    d[np.arange(T)[keep], labels[keep]] -= 1
    ag = np.where(keep, np.abs(g), 0)[:, None]
    d *= ag
    ed = ag * p * (e + el[:, None] + (np.abs(l - lse[:, None]) + 4) * U) + ag * 2 * U
    ed += PARTS[dt] * (np.abs(d) + ed) + (2.0 ** -38 * ag.max() if dt == "f16" else 0)
    mag = np.abs(d) + ed
    return (ed @ np.abs(W) + (2 * V + 64) * U * (mag @ np.abs(W)) + 1e-30,
            ed.T @ np.abs(X) + (2 * T + 64) * U * (mag.T @ np.abs(X)) + 1e-30)


# the few-token kernel with one fragment and several, the products with W transposed,
# ragged sizes
@pytest.mark.parametrize("T,V,H", [(1, 300, 64), (7, 1000, 200), (16, 129, 72), (65, 513, 40), (128, 600, 64),
                                   (200, 1000, 96), (257, 513, 136), (300, 3001, 64)])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_fp32_gradients_keep_their_bits(T, V, H, dt):
    log(f"xent fp32 gradients T={T} V={V} H={H} {dt}")
    x, w, labels, g = inputs(T, V, H, dt)
    labels[0] = V // 2
    X, W = to_dev(x, dt), to_dev(w, dt)
    lab, gd = torch.from_numpy(labels).cuda(), torch.from_numpy(g).cuda()
    _, lse = nm.nm_xent(X, W, lab)
    dx, dw = nm.nm_xent_bwd(X, W, lab, lse, gd)
    torch.cuda.synchronize()
    g = g.astype(np.float64)
    rx, rw = L.xent_bwd_ref(f64(x, dt), f64(w, dt), labels, g)
    bx, bw = bounds(f64(x, dt), f64(w, dt), labels, g, dt)
    within(host(dx), rx, bx)
    within(host(dw), rw, bw)


def call(X, W, lab, lse, gd, dxt, dwt):
    """nm_xent_bwd with a type of its own for each output, in a workspace full of NaN."""
    (T, H), V = X.shape, W.shape[0]
    lib, b, code = nm.lib(), ctypes.c_size_t(), nm.NM_BF16 if X.dtype == torch.bfloat16 else nm.NM_F16
    assert lib.nm_xent_bwd_workspace_size(T, V, H, code, 1, 1, ctypes.byref(b)) == 0
    ws = torch.full((b.value,), 0xFF, dtype=torch.uint8, device="cuda")
    out = [torch.empty((n, H), dtype=t, device="cuda") for n, t in ((T, dxt), (V, dwt))]
    codes = [nm.NM_F32 if t == torch.float32 else code for t in (dxt, dwt)]
    st = lib.nm_xent_bwd(X.data_ptr(), T, H, H, W.data_ptr(), V, H, code, lab.data_ptr(), lse.data_ptr(),
                         gd.data_ptr(), out[0].data_ptr(), H, codes[0], out[1].data_ptr(), H, codes[1],
                         ws.data_ptr(), b.value, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert st == 0
    return out


@pytest.mark.parametrize("T", [9, 100, 300])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_each_output_has_its_own_type(T, dt):
    # an output does not depend on the type, or the absence, of the other
    log(f"xent output types T={T} {dt}")
    x, w, labels, g = inputs(T, 700, 72, dt)
    X, W = to_dev(x, dt), to_dev(w, dt)
    lab, gd = torch.from_numpy(labels).cuda(), torch.from_numpy(g).cuda()
    _, lse = nm.nm_xent(X, W, lab)
    f, h = torch.float32, torch_dtype(dt)
    ff, hh, fh, hf = (call(X, W, lab, lse, gd, *t) for t in ((f, f), (h, h), (f, h), (h, f)))
    assert torch.equal(fh[0], ff[0]) and torch.equal(hf[0], hh[0])
    assert torch.equal(hf[1], ff[1]) and torch.equal(fh[1], hh[1])
    assert torch.equal(nm.nm_xent_bwd(X, W, lab, lse, gd, need_dw=False)[0], ff[0])
    assert torch.equal(nm.nm_xent_bwd(X, W, lab, lse, gd, need_dx=False)[1], ff[1])


@pytest.mark.parametrize("T", [40, 200])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_dloss_of_many_magnitudes(T, dt):
    # dloss from 1 down to 2^-44: dx keeps its relative bound whatever a token's share
    # (dloss multiplies it last); fp16 dw adds 2^-39 of the largest dloss an element,
    # bf16 dw nothing
    log(f"xent dloss magnitudes T={T} {dt}")
    V, H = 500, 64
    x, w, labels, _ = inputs(T, V, H, dt)
    labels[:] = np.arange(T) * 3 % V                # words that only one or two tokens name
    g = (2.0 ** -(44.0 * np.arange(T) / (T - 1))).astype(np.float32)
    X, W = to_dev(x, dt), to_dev(w, dt)
    lab, gd = torch.from_numpy(labels).cuda(), torch.from_numpy(g).cuda()
    _, lse = nm.nm_xent(X, W, lab)
    dx, dw = nm.nm_xent_bwd(X, W, lab, lse, gd)
    torch.cuda.synchronize()
    g = g.astype(np.float64)
    rx, rw = L.xent_bwd_ref(f64(x, dt), f64(w, dt), labels, g)
    # a token at a time: q's own steps of 2^-38 (fp16) are of its g
    bx = np.concatenate([bounds(f64(x, dt)[t:t + 1], f64(w, dt), labels[t:t + 1], g[t:t + 1], dt)[0] for t in range(T)])
    _, bw = bounds(f64(x, dt), f64(w, dt), labels, g, dt)
    within(host(dx), rx, bx)
    within(host(dw), rw, bw)
