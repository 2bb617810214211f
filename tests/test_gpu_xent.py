"""Softmax cross entropy over a vocabulary on MI355X (nm_xent, nm_xent_bwd)
against the float64 oracle.

Bounds, with u = 2^-23: a logit is a sum of H exact products, off by
e = H u sum |x w|.  The sum of exponentials adds 64 u relative (the hardware
exponential's few ulps and |l - max| u of its argument, whose weighted mean is
at most log V, and the additions), so lse is off by at most max e + 64 u +
2 u |lse|.  d = g (p - onehot) is off by |g| p (e + e_lse + (|l - lse| + 4) u) and
one rounding to 16 bits; the products add their sums' errors, and a 16-bit
output one rounding more.
"""
import ctypes

import numpy as np
import pytest

import nm_inputs
import structured_sparse_gemm_nm_amd as nm
from oracle import nm_layers as L
from oracle import nm_oracle as O
from gpu_util import log, to_dev, torch_dtype

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = 2.0 ** -23
HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}          # relative rounding
TINY = {"bf16": 1e-38, "f16": 2.0 ** -24}              # smallest spacing


def inputs(T, V, H, dt, sigma=2.0, seed=0):
    x = nm_inputs.normal_half((T, H), 1.0, dt, 95, 1, seed + T + V)
    w = nm_inputs.normal_half((V, H), sigma * H ** -0.5, dt, 95, 0, seed + V + H)
    rng = np.random.default_rng([96, seed, T, V])
    labels = rng.integers(0, V, size=T).astype(np.int32)
    labels[rng.random(T) < 0.15] = -100
    return x, w, labels, (rng.random(T).astype(np.float32) + 0.5) / T


def f64(bits, dt):
    return O.half_bits_to_f64(bits.reshape(-1), dt).reshape(bits.shape)


def host(t):
    return t.double().cpu().numpy()


def within(got, ref, bound):
    assert got.shape == ref.shape and np.isfinite(got).all()
    worst = (np.abs(got - ref) / bound).max()
    assert worst <= 1.0, f"{worst:.2f} times the bound"


def bounds(X, W, labels, g, dt):
    """(loss, lse, dx, dw) bounds, the last two before an output's rounding."""
    V, H = W.shape
    T = X.shape[0]
    _, lse = L.xent_ref(X, W, labels)
    e = H * U * (np.abs(X) @ np.abs(W).T)
    el = e.max(axis=1) + 64 * U + 2 * U * np.abs(lse)
    keep = (labels >= 0) & (labels < V)
    at = np.where(keep, labels, 0)
    eloss = np.where(keep, el + e[np.arange(T), at] + U * np.abs(lse), 0) + 1e-30
    l = X @ W.T
    p = np.exp(l - lse[:, None])
    d = p.copy()
    d[np.arange(T)[keep], labels[keep]] -= 1
    ag = np.where(keep, np.abs(g), 0)[:, None]
    d *= ag
    ed = ag * p * (e + el[:, None] + (np.abs(l - lse[:, None]) + 4) * U) + ag * 2 * U
    ed += HALF[dt] * (np.abs(d) + ed) + (2.0 ** -38 * ag.max() if dt == "f16" else 0)
    mag = np.abs(d) + ed
    return (eloss, el, ed @ np.abs(W) + V * U * (mag @ np.abs(W)) + 1e-30,
            ed.T @ np.abs(X) + (T + 64) * U * (mag.T @ np.abs(X)) + 1e-30)


def check(T, V, H, dt, **kw):
    x, w, labels, g = inputs(T, V, H, dt, **kw)
    X, W = f64(x, dt), f64(w, dt)
    dx_, dw_, = to_dev(x, dt), to_dev(w, dt)
    lab, gd = torch.from_numpy(labels).cuda(), torch.from_numpy(g).cuda()
    loss, lse = nm.nm_xent(dx_, dw_, lab)
    torch.cuda.synchronize()
    rloss, rlse = L.xent_ref(X, W, labels)
    bl, be, bx, bw = bounds(X, W, labels, g.astype(np.float64), dt)
    within(host(loss), rloss, bl)
    within(host(lse), rlse, be)
    rx, rw = L.xent_bwd_ref(X, W, labels, g.astype(np.float64))
    # the backward pass takes the lse that the forward pass stored
    a, b = nm.nm_xent_bwd(dx_, dw_, lab, lse, gd)
    torch.cuda.synchronize()
    within(host(a), rx, bx)
    within(host(b), rw, bw)
    ah, bh = nm.nm_xent_bwd(dx_, dw_, lab, lse, gd, out_dtype=torch_dtype(dt))
    torch.cuda.synchronize()
    within(host(ah), rx, bx + HALF[dt] * np.abs(rx) + TINY[dt])
    within(host(bh), rw, bw + HALF[dt] * np.abs(rw) + TINY[dt])
    only_x, none = nm.nm_xent_bwd(dx_, dw_, lab, lse, gd, need_dw=False)
    none2, only_w = nm.nm_xent_bwd(dx_, dw_, lab, lse, gd, need_dx=False)
    assert none is None and none2 is None and torch.equal(only_x, a) and torch.equal(only_w, b)


# one token, the narrow tiles' edges, whole and ragged large tiles; vocabularies
# of one word, around a tile, odd; H below, at and past a 64-wide step
@pytest.mark.parametrize("T,V,H", [(1, 1, 8), (1, 300, 64), (7, 1000, 200), (16, 129, 72), (17, 128, 128),
                                   (64, 257, 1040), (65, 5, 40), (200, 1000, 96), (257, 513, 264), (300, 3001, 64),
                                   (520, 700, 512)])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_against_oracle(T, V, H, dt):
    log(f"xent T={T} V={V} H={H} {dt}")
    check(T, V, H, dt)


@pytest.mark.parametrize("sigma", [0.0, 30.0])
def test_flat_and_peaked_distributions(sigma):
    # all logits zero (loss log V), and logits of hundreds (one word takes all)
    log(f"xent sigma={sigma}")
    check(100, 777, 64, "bf16", sigma=sigma)
    check(100, 777, 64, "f16", sigma=sigma)


def test_several_pieces():
    # 4096 tokens cut 40001 words into three pieces; the reference in float64 on the device
    log("xent pieces")
    T, V, H = 4096, 40001, 64
    x, w, labels, g = inputs(T, V, H, "bf16")
    X, W, lab, gd = to_dev(x, "bf16"), to_dev(w, "bf16"), torch.from_numpy(labels).cuda(), torch.from_numpy(g).cuda()
    loss, lse = nm.nm_xent(X, W, lab)
    dx, dw = nm.nm_xent_bwd(X, W, lab, lse, gd)
    torch.cuda.synchronize()
    l = X.double() @ W.double().t()
    ref = torch.logsumexp(l, 1)
    # the logits' bound: H u sum |x w| <= 64 u 64 max|x w|, below 1e-4 here
    assert (lse.double() - ref).abs().max() < 1e-4
    p = (l - ref[:, None]).exp_()
    keep = lab >= 0
    p[torch.arange(T, device="cuda")[keep], lab[keep].long()] -= 1
    p *= (gd.double() * keep)[:, None]
    # 2^-8 of sum |d w| by the rounding of d, 2^-12 more for everything above
    c = 2.0 ** -8 + 2.0 ** -12
    for got, r, b in ((dx, p @ W.double(), p.abs() @ W.double().abs()),
                      (dw, p.t() @ X.double(), p.abs().t() @ X.double().abs())):
        assert ((got.double() - r).abs() <= c * b + 1e-12).all()


@pytest.mark.parametrize("T", [5, 40, 300])
def test_all_ignored(T):
    # no label counts, whatever the number that marks it: zero loss and gradients
    log(f"xent ignored T={T}")
    x, w, labels, g = inputs(T, 500, 64, "bf16")
    labels[:] = -100
    labels[1::3] = 500
    labels[2::3] = np.iinfo(np.int32).min
    X, W, lab, gd = to_dev(x, "bf16"), to_dev(w, "bf16"), torch.from_numpy(labels).cuda(), torch.from_numpy(g).cuda()
    loss, lse = nm.nm_xent(X, W, lab)
    dx, dw = nm.nm_xent_bwd(X, W, lab, lse, gd)
    torch.cuda.synchronize()
    assert not loss.any() and lse.isfinite().all() and not dx.any() and not dw.any()


def test_non_finite_stays_in_its_token():
    # an ignored token of Inf and NaN reaches no gradient; a counted one only its own
    # loss and dx (and dw, which sums over tokens)
    log("xent non-finite")
    T, V, H = 300, 600, 72
    x, w, labels, g = inputs(T, V, H, "bf16")
    labels[:] = np.arange(T) % V
    labels[[3, 200]] = -100
    X, W, lab, gd = to_dev(x, "bf16"), to_dev(w, "bf16"), torch.from_numpy(labels).cuda(), torch.from_numpy(g).cuda()
    loss, lse = nm.nm_xent(X, W, lab)
    dx, dw = nm.nm_xent_bwd(X, W, lab, lse, gd)
    X2 = X.clone()
    X2[3], X2[200, 5] = float("nan"), float("inf")
    loss2, lse2 = nm.nm_xent(X2, W, lab)
    dx2, dw2 = nm.nm_xent_bwd(X2, W, lab, lse2, gd)
    torch.cuda.synchronize()
    assert torch.equal(loss2, loss) and torch.equal(dx2, dx) and torch.equal(dw2, dw)
    X2 = X.clone()
    X2[10, 0] = float("nan")
    loss3, lse3 = nm.nm_xent(X2, W, lab)
    dx3, _ = nm.nm_xent_bwd(X2, W, lab, lse3, gd)
    torch.cuda.synchronize()
    rest = torch.arange(T, device="cuda") != 10
    assert loss3[10].isnan() and dx3[10].isnan().all()
    assert torch.equal(loss3[rest], loss[rest]) and torch.equal(dx3[rest], dx[rest])


def test_words_that_no_token_can_take():
    # logits of -inf (a word's row holds -inf against positive activations): probability
    # 0; their tiles hold no finite logit at all
    log("xent -inf words")
    T, V, H = 70, 1000, 64
    x, w, labels, g = inputs(T, V, H, "bf16")
    X, W = to_dev(x, "bf16").abs(), to_dev(w, "bf16")
    W2 = W.clone()
    W2[256:768] = float("-inf")
    labels = np.where(labels >= 0, labels % 256, labels).astype(np.int32)
    lab = torch.from_numpy(labels).cuda()
    kept = torch.cat([W[:256], W[768:]]).contiguous()
    loss, lse = nm.nm_xent(X, W2, lab)
    ref, rlse = L.xent_ref(host(X), host(kept), labels)
    torch.cuda.synchronize()
    assert np.abs(host(lse) - rlse).max() < 1e-4 and np.abs(host(loss) - ref).max() < 1e-4


@pytest.mark.parametrize("scale", [2.0 ** -30, 2.0 ** 30])
def test_f16_gradients_of_any_size(scale):
    # dloss far outside fp16's range: d is scaled by a power of two for the
    # products, so scaling dloss by one scales the gradients exactly
    log(f"xent f16 scale={scale}")
    x, w, labels, g = inputs(130, 400, 64, "f16")
    X, W, lab, gd = to_dev(x, "f16"), to_dev(w, "f16"), torch.from_numpy(labels).cuda(), torch.from_numpy(g).cuda()
    _, lse = nm.nm_xent(X, W, lab)
    a, b = nm.nm_xent_bwd(X, W, lab, lse, gd)
    a2, b2 = nm.nm_xent_bwd(X, W, lab, lse, gd * scale)
    zx, zw = nm.nm_xent_bwd(X, W, lab, lse, gd * 0)
    torch.cuda.synchronize()
    assert torch.equal(a2, a * scale) and torch.equal(b2, b * scale) and not zx.any() and not zw.any()


@pytest.mark.parametrize("which", ["one", "all"])
def test_nan_in_dloss_is_not_lost(which):
    # a NaN upstream gradient of a counted token reaches its dx and every entry of dW,
    # also where it is the only kind of gradient there is
    log(f"xent nan dloss {which}")
    T, V, H = 40, 300, 64
    x, w, labels, g = inputs(T, V, H, "bf16")
    labels[:2] = 5, -100
    if which == "one":
        g[0] = np.nan
    else:
        g[:] = np.nan
    X, W = to_dev(x, "bf16"), to_dev(w, "bf16")
    lab, gd = torch.from_numpy(labels).cuda(), torch.from_numpy(g).cuda()
    _, lse = nm.nm_xent(X, W, lab)
    dx, dw = nm.nm_xent_bwd(X, W, lab, lse, gd)
    torch.cuda.synchronize()
    bad = torch.from_numpy(np.isnan(g) & (labels >= 0)).cuda()
    assert dw.isnan().all() and dx[bad].isnan().all()
    assert dx[~bad].isfinite().all() and not dx[1].any()


def test_ignored_token_has_no_gradient_whatever_the_head_holds():
    # an Inf or NaN in a word's row: the counted tokens' gradients are lost, an ignored
    # token's stays zero
    log("xent ignored token, bad word")
    for T in (40, 200):
        V, H = 300, 64
        x, w, labels, g = inputs(T, V, H, "bf16")
        labels[3] = -100
        X, W = to_dev(x, "bf16"), to_dev(w, "bf16")
        W[7, 5], W[290, 9] = float("nan"), float("inf")
        lab, gd = torch.from_numpy(labels).cuda(), torch.from_numpy(g).cuda()
        loss, lse = nm.nm_xent(X, W, lab)
        dx, _ = nm.nm_xent_bwd(X, W, lab, lse, gd)
        torch.cuda.synchronize()
        assert not dx[lab < 0].any() and not loss[lab < 0].any()


def test_gradient_against_differences():
    # L = sum g loss along a random direction of x, by central differences with
    # steps exact in fp16: 2 sum |g| (bound on loss) / 2h of rounding, and h^2 / 6 of
    # a third derivative, at most sum |g| (2 max |v . w|)^3 for a direction v
    log("xent differences")
    T, V, H, dt = 20, 90, 32, "f16"
    x, w, labels, g = inputs(T, V, H, dt)
    h = 2.0 ** -5
    x = nm_inputs.to_half_bits(np.round(f64(x, dt) / h).astype(np.float32) * np.float32(h), dt)
    X, W = f64(x, dt), f64(w, dt)
    v = np.random.default_rng(0).choice([-1.0, 1.0], size=(T, H)) * (np.random.default_rng(1).random((T, H)) < 0.1)
    lab, gd, Wd = torch.from_numpy(labels).cuda(), torch.from_numpy(g).cuda(), to_dev(w, dt)
    val = lambda a: (host(nm.nm_xent(torch.from_numpy(a).half().cuda(), Wd, lab)[0]) * g).sum()
    num = (val(X + h * v) - val(X - h * v)) / (2 * h)
    _, lse = nm.nm_xent(to_dev(x, dt), Wd, lab)
    dx, _ = nm.nm_xent_bwd(to_dev(x, dt), Wd, lab, lse, gd)
    bl, _, bx, _ = bounds(X, W, labels, g.astype(np.float64), dt)
    tol = (g * bl).sum() * 2 / h + h * h / 6 * (g * (2 * np.abs(v @ W.T).max(1)) ** 3).sum() + (bx * np.abs(v)).sum()
    assert abs(num - (host(dx) * v).sum()) <= tol


def test_views_streams_and_workspace_contents():
    # operands inside wider NaN buffers, another stream, and a workspace full of NaN
    log("xent views")
    T, V, H, dt = 90, 333, 72, "bf16"
    x, w, labels, g = inputs(T, V, H, dt)
    X, W, lab, gd = to_dev(x, dt), to_dev(w, dt), torch.from_numpy(labels).cuda(), torch.from_numpy(g).cuda()
    loss, lse = nm.nm_xent(X, W, lab)
    dx, dw = nm.nm_xent_bwd(X, W, lab, lse, gd)
    Xw = torch.full((T, H + 16), float("nan"), dtype=torch.bfloat16, device="cuda")
    Ww = torch.full((V, H + 24), float("nan"), dtype=torch.bfloat16, device="cuda")
    Xw[:, 8:H + 8], Ww[:, 16:H + 16] = X, W
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        loss2, lse2 = nm.nm_xent(Xw[:, 8:H + 8], Ww[:, 16:H + 16], lab)
        dx2, dw2 = nm.nm_xent_bwd(Xw[:, 8:H + 8], Ww[:, 16:H + 16], lab, lse2, gd)
    s.synchronize()
    assert torch.equal(loss2, loss) and torch.equal(lse2, lse) and torch.equal(dx2, dx) and torch.equal(dw2, dw)
    lib, b = nm.lib(), ctypes.c_size_t()
    assert lib.nm_xent_bwd_workspace_size(T, V, H, nm.NM_BF16, 1, 1, ctypes.byref(b)) == 0
    ws = torch.full((b.value,), 0xFF, dtype=torch.uint8, device="cuda")
    dx3, dw3 = torch.full_like(dx, float("nan")), torch.full((V, H + 4), float("nan"), device="cuda")
    st = lib.nm_xent_bwd(X.data_ptr(), T, H, H, W.data_ptr(), V, H, nm.NM_BF16, lab.data_ptr(), lse.data_ptr(),
                         gd.data_ptr(), dx3.data_ptr(), H, nm.NM_F32, dw3.data_ptr(), H + 4, nm.NM_F32, ws.data_ptr(),
                         b.value, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert st == 0 and torch.equal(dx3, dx) and torch.equal(dw3[:, :H], dw) and dw3[:, H:].isnan().all()


def test_empty():
    log("xent empty")
    w = torch.randn(50, 64, device="cuda").bfloat16()
    x, lab, e = w[:0], torch.empty(0, dtype=torch.int32, device="cuda"), torch.empty(0, device="cuda")
    loss, lse = nm.nm_xent(x, w, lab)
    assert loss.shape == (0,) and lse.shape == (0,)
    for od in (None, torch.bfloat16):
        dx, dw = nm.nm_xent_bwd(x, w, lab, lse, e, out_dtype=od)
        torch.cuda.synchronize()
        assert dx.shape == (0, 64) and dw.shape == (50, 64) and not dw.any()


def test_binding_refusals():
    w = torch.zeros((50, 64), dtype=torch.bfloat16, device="cuda")
    x, lab = w[:4], torch.zeros(4, dtype=torch.int32, device="cuda")
    f = torch.zeros(4, device="cuda")
    with pytest.raises(TypeError):
        nm.nm_xent(x.float(), w.float(), lab)
    with pytest.raises(ValueError):
        nm.nm_xent(x, w.half(), lab)
    with pytest.raises(ValueError):
        nm.nm_xent(x, w[:, :56], lab)
    with pytest.raises(ValueError):
        nm.nm_xent(x, w, lab.long())
    with pytest.raises(ValueError):
        nm.nm_xent(x, w, lab[:3])
    with pytest.raises(ValueError):
        nm.nm_xent(x, w, lab, ignore_index=3)
    with pytest.raises(ValueError):
        nm.nm_xent_bwd(x, w, lab, f[:3], f)
    with pytest.raises(ValueError):
        nm.nm_xent_bwd(x, w, lab, f, f.double())
    with pytest.raises(TypeError):
        nm.nm_xent_bwd(x, w, lab, f, f, out_dtype=torch.float16)
    with pytest.raises(nm.NMError):
        nm.nm_xent(w[:4, :60].contiguous(), w[:, :60].contiguous(), lab)      # H % 8
