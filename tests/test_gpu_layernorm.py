"""Layer norm on MI355X (nm_layernorm, nm_layernorm_bwd) against the float64 oracle.

Bounds, with u = 2^-24: a row's sums are taken by threads of at most 16 (long
rows: 17 for the widths here) terms, six shuffles and at most 16 waves, so a sum
of n terms is off by at most 40 u sum |terms|; with the few roundings of each
element's own chain every quantity below stays within C = 64 u of the sum of the
magnitudes it is made of, plus one rounding of the output.
"""
import numpy as np
import pytest

import structured_sparse_gemm_nm_amd as nm
from oracle import nm_layers as L
from gpu_util import log

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

C = 64 * 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
# half an ulp relative to the value, and the smallest spacing
ROUND = {"bf16": (2.0 ** -8, 1e-38), "f16": (2.0 ** -11, 2.0 ** -24), "f32": (2.0 ** -24, 1e-38)}


def f64(t):
    return t.detach().double().cpu().numpy()


def rounding(ref, dt):
    rel, tiny = ROUND[dt]
    return np.abs(ref) * rel + tiny


def within(got, ref, bound):
    assert got.shape == ref.shape
    assert np.isfinite(got).all()
    worst = (np.abs(got - ref) / bound).max() if ref.size else 0.0
    assert worst <= 1.0, f"{worst:.2f} times the bound"


def case(T, H, dt, seed=0, pad=0):
    g = torch.Generator().manual_seed(seed * 1000003 + T * 131 + H)
    mk = lambda *s: torch.randn(*s, generator=g)
    x = mk(T, H + pad) + 3 * mk(T, 1)
    return tuple(t.to(DT[dt]).cuda() for t in (x, mk(T, H + pad), 1 + 0.5 * mk(H), mk(H)))


def check_forward(x, w, b, dt, eps=1e-5, **kw):
    y, mean, rstd = nm.nm_layernorm(x, w, b, eps=eps, stats=True, **kw)
    torch.cuda.synchronize()
    X, W, B = f64(x), 1.0 if w is None else f64(w), 0.0 if b is None else f64(b)
    ry, rm, rr = L.layernorm_ref(X, W, B, np.float32(eps).astype(np.float64))
    size = np.abs(X).mean(axis=1)
    xh = (X - rm[:, None]) * rr[:, None]
    within(f64(mean), rm, C * size + 1e-30)
    within(f64(rstd), rr, rr * (C + C * C * (size * rr) ** 2))
    within(f64(y), ry, C * (np.abs(W) * ((size * rr)[:, None] + 2 * np.abs(xh)) + np.abs(B)) + rounding(ry, dt) + 1e-30)
    return y, mean, rstd


def check_backward(dy, x, w, dt, out_dtype=None, **kw):
    X, G, W = f64(x), f64(dy), 1.0 if w is None else f64(w)
    _, rm, rr = L.layernorm_ref(X, W, 0.0, 1e-5)
    mean, rstd = (torch.from_numpy(a.astype(np.float32)).cuda() for a in (rm, rr))
    rm, rr = f64(mean), f64(rstd)      # both sides take the statistics as stored
    dx, dw, db = nm.nm_layernorm_bwd(dy, x, mean, rstd, w, out_dtype=out_dtype, **kw)
    torch.cuda.synchronize()
    rx, rw, rb = L.layernorm_bwd_ref(G, X, rm, rr, W)
    xh = np.abs((X - rm[:, None]) * rr[:, None])
    p = np.abs(G * W)
    bx = rr[:, None] * (p + p.mean(1)[:, None] + xh * (p * xh).mean(1)[:, None])
    within(f64(dx), rx, C * bx + rounding(rx, dt) + 1e-30)
    if dw is not None:
        # a column's sum: T terms in some order of at most T + 64 additions
        c = (X.shape[0] + 64) * 2.0 ** -24
        od = dt if out_dtype is not None else "f32"
        within(f64(dw), rw, c * (np.abs(G) * xh).sum(0) + rounding(rw, od) + 1e-30)
        within(f64(db), rb, c * np.abs(G).sum(0) + rounding(rb, od) + 1e-30)
    return dx, dw, db


# widths at and past each group's limit, odd ones, one feature, and rows walked in loops
WIDTHS = [1, 3, 8, 64, 511, 512, 513, 1024, 1025, 2048, 2056, 4096, 4097, 8192, 8200, 16384, 16391, 20000]


@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("dt", list(DT))
def test_widths(H, dt):
    log(f"layernorm H={H} {dt}")
    x, dy, w, b = case(5, H, dt)
    check_forward(x, w, b, dt)
    if H > 1:
        check_backward(dy, x, w, dt)


@pytest.mark.parametrize("T", [1, 2, 4, 7, 511, 513, 2049, 5000])
@pytest.mark.parametrize("H", [96, 1100])
def test_token_counts(T, H):
    log(f"layernorm T={T} H={H}")
    x, dy, w, b = case(T, H, "bf16")
    check_forward(x, w, b, "bf16")
    check_backward(dy, x, w, "bf16")


@pytest.mark.parametrize("dt", list(DT))
def test_no_weights_and_rounded_gradients(dt):
    log(f"layernorm without weights {dt}")
    x, dy, w, b = case(33, 200, dt)
    check_forward(x, None, None, dt)
    check_forward(x, w, None, dt)
    check_forward(x, None, b, dt, eps=0.5)
    check_backward(dy, x, None, dt)
    check_backward(dy, x, w, dt, out_dtype=DT[dt])
    dx, dw, db = check_backward(dy, x, w, dt, affine=False)
    assert dw is None and db is None


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("H,off", [(515, 1), (2048, 3), (16390, 5)])
def test_unaligned_views(dt, H, off):
    # columns off .. off + H of a wider buffer whose other columns are NaN: rows
    # start at element alignment only and nothing outside them is used or written
    log(f"layernorm view H={H} off={off} {dt}")
    T = 6
    x, dy, w, b = case(T, H, dt)
    hold = lambda: torch.full((T, H + off + 4), float("nan"), dtype=DT[dt], device="cuda")
    X, G, O = hold(), hold(), hold()
    X[:, off:off + H] = x
    G[:, off:off + H] = dy
    check_forward(X[:, off:off + H], w, b, dt, out=O[:, off:off + H])
    check_backward(G[:, off:off + H], X[:, off:off + H], w, dt, out=O[:, off:off + H])
    O = O.float()
    assert O[:, :off].isnan().all() and O[:, off + H:].isnan().all()


def test_large_offset_keeps_the_variance():
    # a mean 4096 times the deviation: the variance about the mean, not from moments
    log("layernorm large offset")
    g = torch.Generator().manual_seed(5)
    x = (4096 + torch.randn(4, 3000, generator=g)).cuda()
    check_forward(x, None, None, "f32")


def test_constant_and_extreme_rows():
    # a constant row has no deviation (y = bias); Inf or NaN stay in their own row
    log("layernorm extreme rows")
    x = torch.randn(4, 700, device="cuda")
    x[1] = 3.0
    x[2, 5] = float("inf")
    b = torch.randn(700, device="cuda")
    y, mean, rstd = nm.nm_layernorm(x, None, b, stats=True)
    torch.cuda.synchronize()
    assert torch.equal(y[1], b)
    assert y[2].isnan().all()
    check_forward(x[[0, 3]].contiguous(), None, b, "f32")
    assert torch.equal(y[[0, 3]], nm.nm_layernorm(x[[0, 3]].contiguous(), None, b))
    # the same for gradients: the row's dx and the column sums, no other row's dx
    dy = torch.randn(4, 700, device="cuda")
    dx, dw, _ = nm.nm_layernorm_bwd(dy, x, mean, rstd)
    keep = [0, 1, 3]
    ref, _, _ = nm.nm_layernorm_bwd(dy[keep].contiguous(), x[keep].contiguous(), mean[keep], rstd[keep])
    assert torch.equal(dx[keep], ref) and dx[2].isnan().all() and dw.isnan().all()


def test_gradient_against_differences():
    # dL of L = sum(y dy) along a direction v, by central differences of the
    # float32 forward: the difference of two sums of 200 products of size ~1 holds
    # C * 200 * 2 / (2 * step) of rounding and step^2 |L'''| / 6 of truncation
    log("layernorm differences")
    g = torch.Generator().manual_seed(3)
    x, dy, v = (torch.randn(2, 100, generator=g).cuda() for _ in range(3))
    w = torch.randn(100, generator=g).cuda()
    _, mean, rstd = nm.nm_layernorm(x, w, stats=True)
    dx, _, _ = nm.nm_layernorm_bwd(dy, x, mean, rstd, w)
    h = 0.02
    val = lambda t: (nm.nm_layernorm(t, w).double() * dy.double()).sum().item()
    num = (val(x + h * v) - val(x - h * v)) / (2 * h)
    ref = (dx.double() * v.double()).sum().item()
    # h exactly representable steps are not needed: x + h v is rounded (2^-24 |x|
    # an element, times |dx|), inside the first term
    assert abs(num - ref) <= C * 400 / h + h * h * 200


def test_empty_and_repeatable():
    log("layernorm empty")
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    assert nm.nm_layernorm(x).shape == (0, 64)
    e = torch.empty(0, device="cuda")
    dx, dw, db = nm.nm_layernorm_bwd(x, x, e, e)
    assert dx.shape == (0, 64) and not dw.any() and not db.any()
    x, dy, w, b = case(3000, 320, "bf16")
    y, mean, rstd = nm.nm_layernorm(x, w, b, stats=True)
    first = nm.nm_layernorm_bwd(dy, x, mean, rstd, w)
    again = nm.nm_layernorm_bwd(dy, x, mean, rstd, w)
    assert all(torch.equal(p, q) for p, q in zip(first, again))


def test_another_stream():
    log("layernorm stream")
    x, dy, w, b = case(64, 512, "f16")
    ref = nm.nm_layernorm(x, w, b)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        y = nm.nm_layernorm(x, w, b)
    s.synchronize()
    assert torch.equal(y, ref)


def test_binding_refusals():
    x = torch.zeros((4, 16), device="cuda")
    st = torch.zeros(4, device="cuda")
    with pytest.raises(TypeError):
        nm.nm_layernorm(x.double())
    with pytest.raises(ValueError):
        nm.nm_layernorm(x.t())
    with pytest.raises(ValueError):
        nm.nm_layernorm(x, torch.zeros(15, device="cuda"))
    with pytest.raises(ValueError):
        nm.nm_layernorm(x, torch.zeros(16, dtype=torch.float16, device="cuda"))
    with pytest.raises(ValueError):
        nm.nm_layernorm(torch.zeros(4, 16))
    with pytest.raises(ValueError):
        nm.nm_layernorm_bwd(x[:3], x, st, st)
    with pytest.raises(ValueError):
        nm.nm_layernorm_bwd(x, x, st[:3], st)
    with pytest.raises(TypeError):
        nm.nm_layernorm_bwd(x, x, st, st, out_dtype=torch.float16)
    with pytest.raises(nm.NMError):
        nm.nm_layernorm(x, eps=-1.0)
    with pytest.raises(nm.NMError):
        nm.nm_layernorm(x, out=x)          # in place: the output overlaps the input
