"""Low-rank adapters beside an N:M projection on MI355X (nm_adapter_spmm,
nm_adapter_spmm_bwd) against the float64 oracle.

Bounds, with u = 2^-23 (sums of exact products in any order, round toward zero
allowed): an fp32 sum of n terms is off by n u sum |terms|.  xa carries its own
sum's error into the second product; there it is split into two bf16 parts
(2^-16 of each term), and the sum over the rank adds r u.  Half outputs add one
rounding (assert_close's terms).
"""
import numpy as np
import pytest

import nm_inputs
import structured_sparse_gemm_nm_amd as nm
from oracle import nm_layers as L
from oracle import nm_oracle as O
from gpu_util import assert_close, log, to_dev, torch_dtype

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = 2.0 ** -23
SPLIT = 2.0 ** -16


def half(shape, sigma, dt, *seed):
    return nm_inputs.normal_half(shape, sigma, dt, 90, *seed)


def f64(bits, dt):
    return O.half_bits_to_f64(bits.reshape(-1), dt).reshape(bits.shape)


class Case:
    def __init__(self, R, K, T, r, na, dt, n=2, m=4, ids=None, seed=0):
        self.R, self.K, self.T, self.r, self.na, self.dt, self.n, self.m = R, K, T, r, na, dt, n, m
        self.vals, self.idx = O.prune_pack(half((R, K), 0.05, dt, 0, seed), n, m)
        self.w = O.half_bits_to_f64(O.decompress(self.vals, self.idx, K, n, m), dt)
        self.act, self.g = half((T, K), 1.0, dt, 1, seed), half((T, R), 1.0, dt, 4, seed)
        self.A = half((na * r, K), K ** -0.5, dt, 5, seed).reshape(na, r, K)
        self.B = half((na * R, r), 0.3, dt, 6, seed).reshape(na, R, r)
        rng = np.random.default_rng([91, seed, T, na])
        self.scale = (0.5 + rng.random(na)).astype(np.float32)
        if ids is None:     # runs of one adapter, some without
            ids = np.repeat(rng.integers(-1, na, size=T), rng.integers(1, 24, size=T))[:T]
        self.ids = np.asarray(ids, dtype=np.int32)

    def dev(self):
        d = lambda x: to_dev(x.reshape(-1, x.shape[-1]), self.dt).view(x.shape)
        return dict(values=to_dev(self.vals, self.dt), idx=torch.from_numpy(self.idx.view(np.int32)).cuda(),
                    act=d(self.act), adapter=torch.from_numpy(self.ids).cuda(), A=d(self.A), B=d(self.B),
                    scale=torch.from_numpy(self.scale).cuda()), d(self.g)

    def wide(self):
        return (f64(self.act, self.dt), f64(self.g, self.dt), f64(self.A, self.dt), f64(self.B, self.dt),
                self.scale.astype(np.float64))

    def forward(self, out_dtype=None, **kw):
        d, _ = self.dev()
        y, xa = nm.nm_adapter_spmm(**d, K=self.K, n=self.n, m=self.m, out_dtype=out_dtype, **kw)
        torch.cuda.synchronize()
        return y, xa

    def check_forward(self, half_out=True):
        x, _, A, B, s = self.wide()
        ref, rxa = L.adapter_ref(self.w, x, self.ids, A, B, s)
        mag, mxa = L.adapter_ref(np.abs(self.w), np.abs(x), self.ids, np.abs(A), np.abs(B), s)
        terms = mag - np.abs(x) @ np.abs(self.w).T      # sum |s B (A x)| with magnitudes inside
        bound = self.K * U * mag + (SPLIT + (self.K + self.r + 8) * U) * terms + 1e-30
        y, xa = self.forward()
        err = np.abs(xa.double().cpu().numpy() - rxa)
        assert (err <= self.K * U * mxa + 1e-30).all()
        assert_close(y, ref.T, bound.T)
        if half_out:
            yh, _ = self.forward(torch_dtype(self.dt))
            assert_close(yh, ref.T, bound.T, out_half=self.dt)

    def check_backward(self, half_out=True, need_dx=True):
        x, g, A, B, s = self.wide()
        _, xa = L.adapter_ref(self.w, x, self.ids, A, B, s)
        xa = xa.astype(np.float32)
        dx, dA, dB = L.adapter_bwd_ref(self.w, g, x, xa.astype(np.float64), self.ids, A, B, s)
        ab = np.abs
        mx, mA, mB = L.adapter_bwd_ref(ab(self.w), ab(g), ab(x), ab(xa).astype(np.float64), self.ids, ab(A), ab(B), s)
        base = ab(g) @ ab(self.w)
        c = SPLIT + (self.R + self.r + 8) * U
        bx = self.R * U * mx + c * (mx - base) + 1e-30
        bA = (c + self.T * U) * mA + 1e-30
        bB = (SPLIT + (self.T + 8) * U) * mB + 1e-30
        d, G = self.dev()
        X = torch.from_numpy(xa).cuda()
        got = nm.nm_adapter_spmm_bwd(G=G, xa=X, **d, K=self.K, n=self.n, m=self.m, need_dx=need_dx)
        torch.cuda.synchronize()
        if need_dx:
            assert_close(got[0], dx.T, bx.T)
        else:
            assert got[0] is None
        for t, ref, b in ((got[1], dA, bA), (got[2], dB, bB)):
            assert (np.abs(t.double().cpu().numpy() - ref) <= b).all()
        if half_out and need_dx:
            gh = nm.nm_adapter_spmm_bwd(G=G, xa=X, **d, K=self.K, n=self.n, m=self.m, out_dtype=torch_dtype(self.dt))
            torch.cuda.synchronize()
            assert_close(gh[0], dx.T, bx.T, out_half=self.dt)
            assert torch.equal(gh[1], got[1]) and torch.equal(gh[2], got[2])


# (R, K, T, rank, adapters): one token, a few, a fragment's edge, prefill tiles;
# odd R and rank, K that is no multiple of the 64-wide step, one adapter and many
FORWARD = [(64, 64, 1, 1, 1), (301, 208, 3, 5, 4), (256, 1040, 16, 16, 24), (1000, 512, 17, 33, 3),
           (264, 384, 130, 8, 2), (520, 256, 333, 64, 5), (300, 128, 200, 100, 2), (4096, 256, 5, 24, 6),
           (256, 4224, 7, 16, 3)]


@pytest.mark.parametrize("R,K,T,r,na", FORWARD)
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_forward(R, K, T, r, na, dt):
    log(f"adapter R={R} K={K} T={T} r={r} n={na} {dt}")
    Case(R, K, T, r, na, dt).check_forward()


@pytest.mark.parametrize("n,m", nm.PATTERNS)
@pytest.mark.parametrize("T", [4, 40, 150])
def test_patterns(n, m, T):
    log(f"adapter {n}:{m} T={T}")
    c = Case(320, 512, T, 12, 3, "bf16", n, m)
    c.check_forward()
    c.check_backward()


# the shared product in shares of K: one tile and several, a last step of 32,
# more steps than waves, 16 tokens of a K past the few-token family; and shapes
# of as few tokens whose K is too short to share out
@pytest.mark.parametrize("R,K,T,n,m", [(33, 2080, 17, 2, 4), (32, 64, 20, 2, 4), (250, 96, 40, 2, 4),
                                       (5, 8224, 16, 2, 4), (300, 4160, 33, 2, 4), (100, 1056, 65, 1, 4),
                                       (301, 8192, 64, 1, 4), (48, 4128, 9, 1, 4), (250, 2112, 129, 1, 8),
                                       (37, 6208, 16, 1, 8), (64, 128, 31, 1, 8)])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_product_in_shares(R, K, T, n, m, dt):
    log(f"adapter shares R={R} K={K} T={T} {n}:{m} {dt}")
    c = Case(R, K, T, 7, 3, dt, n, m)
    c.check_forward()
    # activations inside a wider buffer of NaN: nothing past K is used
    d, _ = c.dev()
    X = torch.full((T, K + 64), float("nan"), dtype=torch_dtype(dt), device="cuda")
    X[:, :K] = d["act"]
    y, _ = nm.nm_adapter_spmm(**d, K=K, n=n, m=m)
    y2, _ = nm.nm_adapter_spmm(**dict(d, act=X[:, :K]), K=K, n=n, m=m)
    torch.cuda.synchronize()
    assert torch.equal(y, y2)

# 1:8 with K an odd multiple of 32: rows of values on 8 bytes, a last step of 4 values
@pytest.mark.parametrize("R,K,T", [(33, 1056, 17), (531, 2848, 261), (100, 4128, 9), (32, 1120, 64)])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_product_in_shares_of_short_rows(R, K, T, dt):
    log(f"adapter shares R={R} K={K} T={T} 1:8 {dt}")
    Case(R, K, T, 12, 3, dt, 1, 8).check_forward()


@pytest.mark.parametrize("R,K,T,r,na", [(64, 64, 1, 1, 1), (304, 224, 3, 5, 4), (136, 1056, 50, 17, 3),
                                        (520, 256, 333, 64, 5), (72, 96, 200, 100, 2), (256, 512, 129, 32, 1)])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_backward(R, K, T, r, na, dt):
    log(f"adapter backward R={R} K={K} T={T} r={r} n={na} {dt}")
    c = Case(R, K, T, r, na, dt)
    c.check_backward()
    c.check_backward(need_dx=False)


@pytest.mark.parametrize("T", [16, 100, 160])
def test_tokens_in_any_order(T):
    # every token its own draw, ids far outside the range among them
    log(f"adapter mixed order T={T}")
    rng = np.random.default_rng(T)
    ids = rng.integers(-2, 9, size=T).astype(np.int32)
    ids[::7] = np.iinfo(np.int32).max
    ids[1::11] = np.iinfo(np.int32).min
    c = Case(264, 320, T, 20, 7, "bf16", ids=ids)
    c.check_forward()
    c.check_backward()


@pytest.mark.parametrize("ids", [-1, 3])
def test_all_or_none(ids):
    # no token with an adapter: the shared projection alone, and zero gradients
    log(f"adapter all {ids}")
    c = Case(264, 320, 140, 9, 4, "f16", ids=np.full(140, ids))
    c.check_forward()
    c.check_backward()
    if ids < 0:
        d, _ = c.dev()
        y, xa = c.forward()
        assert torch.equal(y, nm.nm_spmm(d["values"], d["idx"], d["act"], c.K)) and not xa.any()


def test_small_and_large_values_in_f16():
    # gradients near fp16's smallest numbers and shrunk activations past its largest
    log("adapter f16 range")
    c = Case(264, 320, 33, 8, 2, "f16")
    c.g = nm_inputs.to_half_bits(1e-6 * np.random.default_rng(0).normal(size=(33, 264)).astype(np.float32), "f16")
    c.A = nm_inputs.to_half_bits(300 * np.random.default_rng(1).normal(size=c.A.shape).astype(np.float32), "f16")
    c.act = nm_inputs.to_half_bits(50 * np.random.default_rng(2).normal(size=c.act.shape).astype(np.float32), "f16")
    assert np.abs(L.adapter_ref(c.w, *[c.wide()[0], c.ids, *c.wide()[2:]])[1]).max() > 65504
    c.check_forward(half_out=False)
    c.check_backward(half_out=False)


def test_non_finite_stays_with_its_token_and_adapter():
    log("adapter non-finite")
    rng = np.random.default_rng(4)
    c = Case(264, 320, 140, 12, 3, "bf16", ids=rng.integers(0, 3, size=140))
    d, G = c.dev()
    y, xa = nm.nm_adapter_spmm(**d, K=c.K)
    dx, dA, dB = nm.nm_adapter_spmm_bwd(G=G, xa=xa, **d, K=c.K)
    d["act"][5] = float("inf")
    d["B"][1] = float("nan")
    d["A"][1, 0, 0] = float("nan")
    G[6] = float("nan")
    y2, xa2 = nm.nm_adapter_spmm(**d, K=c.K)
    dx2, dA2, dB2 = nm.nm_adapter_spmm_bwd(G=G, xa=xa2, **d, K=c.K)
    torch.cuda.synchronize()
    clean = torch.from_numpy(c.ids != 1).cuda()
    clean[5] = False
    assert torch.equal(y2[clean], y[clean]) and torch.equal(xa2[clean], xa[clean])
    assert not y2[~clean].isfinite().any()
    clean[5], clean[6] = bool(c.ids[5] != 1), False      # dX does not read act
    assert torch.equal(dx2[clean], dx[clean])
    for a in range(3):
        if a != 1 and a not in (c.ids[5], c.ids[6]):
            assert torch.equal(dA2[a], dA[a]) and torch.equal(dB2[a], dB[a])


def test_exact_on_integers():
    # integers small enough that every partial sum is exact, xa (below 2^16) in two bf16 parts too
    log("adapter integers")
    for dt in ("bf16", "f16"):
        c = Case(136, 96, 75, 6, 3, dt)
        w = nm_inputs.integer_half((136, 96), -3, 3, dt, 92, 0)
        c.vals, c.idx = O.prune_pack(w, 2, 4)
        c.w = O.half_bits_to_f64(O.decompress(c.vals, c.idx, 96, 2, 4), dt)
        c.act, c.g = nm_inputs.integer_half((75, 96), -3, 3, dt, 92, 1), nm_inputs.integer_half((75, 136), -3, 3, dt, 92, 4)
        c.A = nm_inputs.integer_half((18, 96), -3, 3, dt, 92, 5).reshape(3, 6, 96)
        c.B = nm_inputs.integer_half((3 * 136, 6), -3, 3, dt, 92, 6).reshape(3, 136, 6)
        c.scale = np.array([1.0, 2.0, 0.5], dtype=np.float32)
        x, g, A, B, s = c.wide()
        ref, rxa = L.adapter_ref(c.w, x, c.ids, A, B, s)
        y, xa = c.forward()
        assert np.array_equal(xa.double().cpu().numpy(), rxa) and np.array_equal(y.double().cpu().numpy(), ref)
        d, G = c.dev()
        got = nm.nm_adapter_spmm_bwd(G=G, xa=xa, **d, K=c.K)
        for t, q in zip(got, L.adapter_bwd_ref(c.w, g, x, rxa, c.ids, A, B, s)):
            assert np.array_equal(t.double().cpu().numpy(), q)


def test_gradient_against_differences():
    # L = sum(Y G) along random directions of act (fp16 steps of 2^-4 on values below
    # 4: exact), A and B; the map is bilinear, so a central difference along one of
    # them has no truncation and only both forwards' bounds / (2 h) of rounding
    log("adapter differences")
    c = Case(136, 96, 40, 6, 3, "f16", seed=3)
    rng = np.random.default_rng(9)
    d, G = c.dev()
    q = lambda a, step: torch.from_numpy(np.round(a / step) * step).to(torch.float16).cuda()
    h = 2.0 ** -4
    d["act"] = q(rng.uniform(-2, 2, (40, 96)), h)
    d["A"] = q(rng.uniform(-2, 2, (3, 6, 96)), h)
    d["B"] = q(rng.uniform(-2, 2, (3, 136, 6)), h)
    _, xa = nm.nm_adapter_spmm(**d, K=c.K)
    dx, dA, dB = nm.nm_adapter_spmm_bwd(G=G, xa=xa, **d, K=c.K)
    mag = L.adapter_ref(np.abs(c.w), np.abs(d["act"].double().cpu().numpy()) + h, c.ids,
                        np.abs(d["A"].double().cpu().numpy()) + h, np.abs(d["B"].double().cpu().numpy()) + h,
                        c.scale.astype(np.float64))[0]
    tol = (2 * SPLIT + 512 * U) * (mag * np.abs(c.wide()[1])).sum() / h
    for name, grad in (("act", dx), ("A", dA), ("B", dB)):
        v = torch.from_numpy(rng.choice([-1.0, 1.0], d[name].shape)).to(torch.float16).cuda()
        keep = d[name]
        vals = []
        for sign in (1, -1):
            d[name] = keep + sign * h * v
            vals.append((nm.nm_adapter_spmm(**d, K=c.K)[0].double() * G.double()).sum().item())
        d[name] = keep
        num = (vals[0] - vals[1]) / (2 * h)
        assert abs(num - (grad.double() * v.double()).sum().item()) <= tol


def test_views_streams_and_empty():
    log("adapter views")
    c = Case(264, 320, 50, 9, 3, "bf16")
    d, G = c.dev()
    y, xa = nm.nm_adapter_spmm(**d, K=c.K)
    ref = nm.nm_adapter_spmm_bwd(G=G, xa=xa, **d, K=c.K)
    # rows inside wider NaN buffers, on another stream
    X = torch.full((50, 320 + 24), float("nan"), dtype=torch.bfloat16, device="cuda")
    X[:, 8:328] = d["act"]
    Gw = torch.full((50, 264 + 16), float("nan"), dtype=torch.bfloat16, device="cuda")
    Gw[:, :264] = G
    Y = torch.full((50, 264 + 3), float("nan"), device="cuda")
    e = dict(d, act=X[:, 8:328])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        y2, xa2 = nm.nm_adapter_spmm(**e, K=c.K, out=Y[:, :264])
        got = nm.nm_adapter_spmm_bwd(G=Gw[:, :264], xa=xa2, **e, K=c.K)
    s.synchronize()
    assert torch.equal(y2, y) and torch.equal(xa2, xa) and Y[:, 264:].isnan().all()
    assert all(torch.equal(p, q) for p, q in zip(got, ref))
    # no tokens, and no adapters
    e = dict(d, act=d["act"][:0], adapter=d["adapter"][:0])
    y0, xa0 = nm.nm_adapter_spmm(**e, K=c.K)
    assert y0.shape == (0, 264) and xa0.shape == (0, 9)
    dx0, dA0, dB0 = nm.nm_adapter_spmm_bwd(G=G[:0], xa=xa0, **e, K=c.K)
    assert dx0.shape == (0, 320) and not dA0.any() and not dB0.any()
    e = dict(d, A=d["A"][:0], B=d["B"][:0], scale=d["scale"][:0])
    y1, xa1 = nm.nm_adapter_spmm(**e, K=c.K)
    assert torch.equal(y1, nm.nm_spmm(d["values"], d["idx"], d["act"], c.K)) and not xa1.any()


def test_no_rows():
    # R == 0: nothing to write but xa; gradients through no rows are zeros
    log("adapter R=0")
    c = Case(64, 320, 40, 9, 3, "bf16")
    d, G = c.dev()
    e = dict(d, values=d["values"][:0], idx=d["idx"][:0], B=d["B"][:, :0].contiguous())
    y, xa = nm.nm_adapter_spmm(**e, K=c.K)
    _, ref = nm.nm_adapter_spmm(**d, K=c.K)
    dx, dA, dB = nm.nm_adapter_spmm_bwd(G=G[:, :0], xa=xa, **e, K=c.K)
    torch.cuda.synchronize()
    assert y.shape == (40, 0) and torch.equal(xa, ref)
    assert not dx.any() and not dA.any() and dB.shape == (3, 0, 9)


def test_binding_refusals():
    c = Case(264, 320, 10, 9, 3, "bf16")
    d, G = c.dev()
    bad = [dict(adapter=d["adapter"].long()), dict(adapter=d["adapter"][:9]), dict(A=d["A"][:, :, :304]),
           dict(A=d["A"].float()), dict(B=d["B"].transpose(1, 2)), dict(B=d["B"][:2]), dict(scale=d["scale"].double()),
           dict(act=d["act"][:, :304]), dict(act=d["act"].half()), dict(adapter=d["adapter"].cpu())]
    for change in bad:
        with pytest.raises(ValueError):
            nm.nm_adapter_spmm(**dict(d, **change), K=c.K)
    with pytest.raises(TypeError):
        nm.nm_adapter_spmm(**d, K=c.K, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        nm.nm_adapter_spmm(**d, K=c.K, xa=torch.empty(10, 8, device="cuda"))
    y, xa = nm.nm_adapter_spmm(**d, K=c.K)
    with pytest.raises(ValueError):
        nm.nm_adapter_spmm_bwd(G=G[:, :256], xa=xa, **d, K=c.K)
    with pytest.raises(nm.NMError):          # R % 8
        c2 = Case(260, 320, 10, 9, 3, "bf16")
        d2, G2 = c2.dev()
        nm.nm_adapter_spmm_bwd(G=G2, xa=xa, **d2, K=c.K)
