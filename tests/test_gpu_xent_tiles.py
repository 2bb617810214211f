"""Cross entropy's larger tiles and longer walks on MI355X: the pipelined 256 x 256
product over several steps with a ragged last one, and few tokens whose vocabulary
takes several pieces, the last one with fewer shares.  References in float64 on the
device, a slice of the vocabulary at a time.

Bounds, with u = 2^-23: a logit is off by e = H u sum |x w| at most, lse by max e +
64 u + 2 u |lse|; p = exp(l - lse) by p (e + e_lse + (|l - lse| + 4) u); d enters the
products in parts within 2^-16 (bf16) or 2^-22 (fp16) of it, fp16 ones in steps of
2^-38 of the largest |g|; the sums of 2 V or 2 T products add u a term.
"""
import numpy as np
import pytest

import structured_sparse_gemm_nm_amd as nm
from gpu_util import log, torch_dtype

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = 2.0 ** -23
PARTS = {"bf16": 2.0 ** -16, "f16": 2.0 ** -22}
ROUND = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"bf16": 1e-38, "f16": 2.0 ** -24}


def inputs(T, V, H, dt, sigma=2.0):
    gen = torch.Generator(device="cuda").manual_seed(T + V + H)
    x = torch.randn((T, H), generator=gen, device="cuda").to(torch_dtype(dt))
    w = (sigma * H ** -0.5 * torch.randn((V, H), generator=gen, device="cuda")).to(torch_dtype(dt))
    labels = torch.randint(0, V, (T,), generator=gen, device="cuda")
    labels[T // 3::5] = V - 1 - torch.arange(labels[T // 3::5].numel(), device="cuda")   # the last words
    labels[1::7] = -100
    g = (torch.rand(T, generator=gen, device="cuda") + 0.5) / T
    return x, w, labels.to(torch.int32), g


def reference(x, w, labels, g, dt, slices=1 << 16):
    """[(loss, bound), (lse, bound), (dx, bound), (dw, bound)]."""
    T, V = x.shape[0], w.shape[0]
    X, H = x.double(), x.shape[1]
    parts = range(0, V, slices)
    at = lambda v0: w[v0:v0 + slices].double()
    lse = torch.logsumexp(torch.stack([torch.logsumexp(X @ at(v0).t(), 1) for v0 in parts]), 0)
    e_max = torch.stack([(X.abs() @ at(v0).abs().t()).amax(1) for v0 in parts]).amax(0) * H * U
    el = e_max + 64 * U + 2 * U * lse.abs()
    keep = labels >= 0
    safe = labels.clamp(min=0).long()
    zero = torch.zeros((), dtype=torch.float64, device="cuda")
    loss = torch.where(keep, lse - (X * w[safe].double()).sum(1), zero)
    gk = torch.where(keep, g.double(), zero)[:, None]
    dx, bx = torch.zeros_like(X), torch.zeros_like(X)
    dw, bw = [], []
    for v0 in parts:
        W = at(v0)
        l = X @ W.t()
        p = (l - lse[:, None]).exp()
        e = H * U * (X.abs() @ W.abs().t())
        ed = gk.abs() * p * (e + el[:, None] + ((l - lse[:, None]).abs() + 4) * U) + 2 * U * gk.abs()
        here = keep & (safe >= v0) & (safe < v0 + W.shape[0])
        p[here, safe[here] - v0] -= 1
        d = p * gk
        ed += PARTS[dt] * (d.abs() + ed) + (2.0 ** -38 * gk.abs().max() if dt == "f16" else 0)
        mag = d.abs() + ed
        dx += d @ W
        bx += ed @ W.abs() + (2 * V + 64) * U * (mag @ W.abs())
        dw.append(d.t() @ X)
        bw.append(ed.t() @ X.abs() + (2 * T + 64) * U * (mag.t() @ X.abs()))
    return [(loss, 2 * el + U * lse.abs()), (lse, el), (dx, bx), (torch.cat(dw), torch.cat(bw))]


def check(T, V, H, dt):
    x, w, labels, g = inputs(T, V, H, dt)
    loss, lse = nm.nm_xent(x, w, labels)
    full = nm.nm_xent_bwd(x, w, labels, lse, g)
    half = nm.nm_xent_bwd(x, w, labels, lse, g, out_dtype=torch_dtype(dt))
    torch.cuda.synchronize()
    ref = reference(x, w, labels, g, dt)
    for got, (r, b) in zip((loss, lse, *full), ref):
        assert ((got.double() - r).abs() <= b + 1e-30).all(), ((got.double() - r).abs() / (b + 1e-30)).max()
    # 16-bit outputs: one rounding of the operand and one of the result, in norm (and
    # fp16's smallest step an entry)
    for got, (r, _) in zip(half, ref[2:]):
        assert (got.double() - r).norm() <= 2 * ROUND[dt] * r.norm() + TINY[dt] * r.numel() ** 0.5
    assert all(torch.equal(a, b) for a, b in zip(full, nm.nm_xent_bwd(x, w, labels, lse, g)))


# 256 x 256 logit tiles: one step, a ragged second one, whole steps, a last step of one
# 16-byte chunk; token and word counts inside a tile
@pytest.mark.parametrize("T,V,H", [(300, 16500, 64), (300, 16500, 72), (257, 16641, 256), (600, 11000, 200),
                                   (300, 16500, 392), (1025, 7000, 584)])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_pipelined_tiles(T, V, H, dt):
    log(f"xent pipelined T={T} V={V} H={H} {dt}")
    check(T, V, H, dt)


# few tokens past 2^26 logits: two pieces, the last a few words or a few shares long
@pytest.mark.parametrize("T,V,H", [(100, 600001, 8), (70, 524300, 16), (16, 1048700, 8), (3, 1600000, 16)])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_few_tokens_several_pieces(T, V, H, dt):
    log(f"xent few tokens, pieces T={T} V={V} H={H} {dt}")
    check(T, V, H, dt)
