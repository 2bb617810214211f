"""Microscaled 4-bit floats on MI355X (nm_mx_quantize, nm_mx_dequantize, nm_mx_gemm)
against the float64 oracle: codes and exponents equal, products within the bound of
an fp32 sum (products of two 4-bit values in their scales are exact; K of them summed
in any order with unit 2^-23 are off by at most K 2^-23 of the sum of their
magnitudes) plus half a step of the output's type.
"""
import numpy as np
import pytest

import structured_sparse_gemm_nm_amd as nm
from oracle import nm_experts as E
from gpu_util import log

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
ROUND = {"bf16": (2.0 ** -8, 1e-38), "f16": (2.0 ** -11, 2.0 ** -24), "f32": (2.0 ** -24, 1e-38)}


def f64(t):
    return t.detach().double().cpu().numpy()


def data(T, K, dt, seed=0):
    g = torch.Generator().manual_seed(seed * 1000003 + T * 131 + K)
    x = torch.randn(T, K, generator=g) * 2.0 ** torch.randint(-6, 6, (T, 1), generator=g)
    return x.to(DT[dt])


def check_quantize(x):
    q, s = nm.nm_mx_quantize(x.cuda() if not x.is_cuda else x)
    torch.cuda.synchronize()
    code, byte = E.mx_quantize_ref(f64(x))
    rq, rs = E.mx_pack_ref(code, byte)
    assert (s.cpu().numpy() == rs).all() and (q.cpu().numpy() == rq).all()
    return q, s, code, byte


@pytest.mark.parametrize("T,K", [(1, 32), (1, 4096), (3, 64), (5, 288), (7, 256), (33, 544), (300, 1056)])
@pytest.mark.parametrize("dt", list(DT))
def test_quantize_and_back(T, K, dt):
    log(f"mx quantise {T}x{K} {dt}")
    x = data(T, K, dt)
    q, s, code, byte = check_quantize(x)
    ref = E.mx_values_ref(code, byte)
    for out in DT:
        y = nm.nm_mx_dequantize(q, s, DT[out])
        torch.cuda.synchronize()
        want = torch.from_numpy(ref).to(DT[out])
        assert torch.equal(y.cpu(), want)
    assert nm.nm_mx_dequantize(q, s).dtype == torch.float32


def test_quantize_ties_and_every_exponent():
    """Each tie and its neighbours in every scale fp32 has, subnormal blocks and the largest among them."""
    log("mx ties in every exponent")
    points = np.array([0.0, 0.25, 0.5, 0.75, 1.0, 1.25, 1.5, 1.75, 2.0, 2.5, 3.0, 3.5, 4.0, 5.0, 6.0, 7.0])
    rows = []
    for e in range(-151, 126):
        p = (points * 2.0 ** e).astype(np.float32)
        up, down = np.nextafter(p, np.float32(np.inf)), np.nextafter(p, np.float32(-np.inf))
        for v in (p, up, down):
            rows.append(np.concatenate([v, -v]))
    x = np.stack(rows)
    x[~np.isfinite(x)] = 1.0
    check_quantize(torch.from_numpy(x))
    # blocks whose largest value is each of fp32's powers of two and just below, beside small ones
    top = np.zeros((277, 32), dtype=np.float32)
    top[:, 5] = 2.0 ** np.arange(-149.0, 128.0)
    top[:, 6] = -np.nextafter(top[:, 5], np.float32(0))
    top[:, 7:] = (top[:, 5:6] * np.linspace(0, 0.3, 25)).astype(np.float32)
    check_quantize(torch.from_numpy(top))
    check_quantize(torch.full((2, 32), torch.finfo(torch.float32).max))


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_quantize_every_half(dt):
    """Every finite 16-bit value, alone in its block and beside one sixteen times as large."""
    log(f"mx every {dt}")
    v = torch.arange(-32768, 32768, dtype=torch.int32).to(torch.int16).view(DT[dt])
    v = v[torch.isfinite(v.float())]
    x = torch.zeros(v.numel(), 64, dtype=DT[dt])
    x[:, 3] = v
    big = (v.float() * 16).to(DT[dt])
    x[:, 40], x[:, 41] = v, torch.where(torch.isfinite(big.float()), big, v)
    check_quantize(x)


@pytest.mark.parametrize("dt", list(DT))
def test_quantize_nonfinite_and_zeros(dt):
    log(f"mx nonfinite {dt}")
    x = data(6, 320, dt)
    x[0, 5], x[1, 40], x[2, 319] = float("inf"), float("nan"), float("-inf")
    x[3, 64:96] = 0.0
    x[4, 32:64] = -0.0
    q, s, code, byte = check_quantize(x)
    y = nm.nm_mx_dequantize(q, s)
    torch.cuda.synchronize()
    got = f64(y)
    assert np.isnan(got[0, :32]).all() and np.isnan(got[1, 32:64]).all() and np.isnan(got[2, 288:]).all()
    assert np.isnan(got).sum() == 96 and not got[3, 64:96].any()


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("off", [1, 3, 8])
def test_quantize_strides(dt, off):
    log(f"mx strided {dt} {off}")
    base = data(9, 200 + off, dt).cuda()
    check_quantize(base[:, off: off + 160])
    check_quantize(base[::2, off: off + 96])


def test_dequantize_every_byte():
    """Every code in every exponent, NaN's among them."""
    log("mx every exponent byte")
    code = np.tile(np.arange(16, dtype=np.uint8), (256, 2))
    byte = np.arange(256, dtype=np.uint8)[:, None]
    q, s = E.mx_pack_ref(code, byte)
    for out in DT:
        y = nm.nm_mx_dequantize(torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda(), DT[out])
        torch.cuda.synchronize()
        want = torch.from_numpy(E.mx_values_ref(code, byte)).float().to(DT[out])
        got = y.cpu()
        assert torch.equal(torch.isnan(got.float()), torch.isnan(want.float()))
        ok = ~torch.isnan(want.float())
        assert torch.equal(got[ok], want[ok])


def operands(rows, K, seed, E_=None):
    x = data((E_ or 1) * rows, K, "f32", seed)
    code, byte = E.mx_quantize_ref(f64(x))
    v = E.mx_values_ref(code, byte)
    if E_ is None:
        return v, *(torch.from_numpy(a).cuda() for a in E.mx_pack_ref(code, byte))
    p = [E.mx_pack_ref(code[e * rows: (e + 1) * rows], byte[e * rows: (e + 1) * rows]) for e in range(E_)]
    return v.reshape(E_, rows, K), *(torch.from_numpy(np.stack([a[i] for a in p])).cuda() for i in range(2))


def within(got, ref, size, K, out):
    assert got.shape == ref.shape and np.isfinite(got).all()
    rel, tiny = ROUND[out]
    bound = K * 2.0 ** -23 * size + np.abs(ref) * rel + tiny + 1e-30
    worst = (np.abs(got - ref) / bound).max() if ref.size else 0.0
    assert worst <= 1.0, f"{worst:.2f} times the bound"


def check_gemm(T, R, K, out, seed=0, ldpad=0):
    w, wq, ws = operands(R, K, seed + 1)
    x, xq, xs = operands(T, K, seed + 2)
    whole = torch.full((T + 2, R + ldpad), 77.0, dtype=DT[out], device="cuda")
    nm.nm_mx_gemm(wq, ws, xq, xs, out_dtype=DT[out], out=whole[:T, :R])
    torch.cuda.synchronize()
    ref, size = x @ w.T, np.abs(x) @ np.abs(w).T
    if out == "f16":
        ref = np.clip(ref, -60000, 60000)
    within(np.clip(f64(whole[:T, :R]), -60000 if out == "f16" else -np.inf, 60000 if out == "f16" else np.inf), ref, size, K, out)
    assert (f64(whole[T:]) == 77.0).all() and (f64(whole[:, R:]) == 77.0).all()


@pytest.mark.parametrize("T,R,K", [(1, 1, 32), (1, 100, 256), (3, 17, 96), (16, 64, 1024), (17, 129, 160), (40, 250, 288),
                                   (65, 96, 4096), (130, 300, 512), (257, 260, 544), (300, 513, 1056), (520, 770, 768)])
@pytest.mark.parametrize("out", list(DT))
def test_gemm(T, R, K, out):
    log(f"mx gemm {T}x{R}x{K} {out}")
    check_gemm(T, R, K, out)


@pytest.mark.parametrize("ldpad", [1, 2, 4, 8])
@pytest.mark.parametrize("T", [5, 300])
def test_gemm_output_strides(T, ldpad):
    log(f"mx gemm strided output {T} {ldpad}")
    for out in DT:
        check_gemm(T, 268, 288, out, ldpad=ldpad)


@pytest.mark.parametrize("lengths", [[0, 1, 0, 1], [3, 0, 17, 1], [70, 2, 0, 200], [300, 129, 0, 513]])
@pytest.mark.parametrize("R,K", [(100, 96), (257, 512), (264, 1056)])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_gemm_of_experts(lengths, R, K, out):
    log(f"mx gemm experts {lengths} {R}x{K} {out}")
    before, behind = 4, 7
    T = before + sum(lengths) + behind
    off = np.cumsum([before, *lengths]).astype(np.int32)
    w, wq, ws = operands(R, K, 3, len(lengths))
    x, xq, xs = operands(T, K, 4)
    xs[:, :before] = 255                      # rows of no expert: NaN
    xs[:, T - behind:] = 255
    whole = torch.full((T + 2, R), 77.0, dtype=DT[out], device="cuda")
    nm.nm_mx_gemm(wq, ws, xq, xs, torch.from_numpy(off).cuda(), out_dtype=DT[out], out=whole[:T])
    torch.cuda.synchronize()
    got = f64(whole)
    assert (got[:before] == 77.0).all() and (got[T - behind:] == 77.0).all()
    for e, (lo, hi) in enumerate(zip(off[:-1], off[1:])):
        within(got[lo:hi], x[lo:hi] @ w[e].T, np.abs(x[lo:hi]) @ np.abs(w[e]).T, K, out)


@pytest.mark.parametrize("T", [5, 300])
def test_gemm_of_a_nan_block(T):
    """A NaN exponent makes the row (of x) or the column (of w) NaN, and nothing else; bytes behind
    the last block of a panel are not looked at."""
    log(f"mx gemm NaN {T}")
    w, wq, ws = operands(264, 288, 1)
    x, xq, xs = operands(T, 288, 2)
    clean = nm.nm_mx_gemm(wq, ws, xq, xs)
    ws[1, :, 1:], xs[1, :, 1:] = 255, 255
    again = nm.nm_mx_gemm(wq, ws, xq, xs)
    xs[0, 2, 3], ws[1, 7, 0] = 255, 255
    y = nm.nm_mx_gemm(wq, ws, xq, xs)
    torch.cuda.synchronize()
    assert torch.equal(clean, again)
    nan = torch.zeros(T, 264, dtype=torch.bool)
    nan[2], nan[:, 7] = True, True
    assert torch.equal(torch.isnan(y).cpu(), nan) and torch.equal(y.cpu()[~nan], clean.cpu()[~nan])


def test_gemm_far_exponents():
    """Scales whose product leaves fp32's range either way."""
    log("mx gemm far exponents")
    code = np.full((1, 64), 7, dtype=np.uint8)
    for a, b, want in [(254, 254, np.inf), (0, 0, 0.0), (254, 0, 64 * 36.0), (200, 54, 64 * 36.0)]:
        wq, ws = (torch.from_numpy(v).cuda() for v in E.mx_pack_ref(code, np.full((1, 2), a, dtype=np.uint8)))
        xq, xs = (torch.from_numpy(v).cuda() for v in E.mx_pack_ref(code, np.full((1, 2), b, dtype=np.uint8)))
        y = nm.nm_mx_gemm(wq, ws, xq, xs)
        torch.cuda.synchronize()
        assert float(y) == want, (a, b, float(y))


def test_empty_stacks_streams_and_graphs():
    log("mx empty, stacked, on a side stream, captured")
    for dt in DT:
        q, s = nm.nm_mx_quantize(torch.empty((0, 64), dtype=DT[dt], device="cuda"))
        assert q.shape == (0, 32) and s.shape == (1, 0, 8) and nm.nm_mx_dequantize(q, s).shape == (0, 64)
    w = torch.stack([data(40, 288, "f32", i) for i in range(3)]).cuda()
    wq, ws = nm.nm_mx_quantize(w)
    back = nm.nm_mx_dequantize(wq, ws)
    for e in range(3):
        q, s = nm.nm_mx_quantize(w[e])
        assert torch.equal(q, wq[e]) and torch.equal(s, ws[e]) and torch.equal(nm.nm_mx_dequantize(q, s), back[e])
    x = data(90, 288, "bf16", 9).cuda()
    off = torch.tensor([0, 30, 30, 90], dtype=torch.int32, device="cuda")

    def serve():
        return nm.nm_mx_gemm(wq, ws, *nm.nm_mx_quantize(x), off, out_dtype=torch.bfloat16)
    first = serve()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = serve()
    torch.cuda.synchronize()
    assert torch.equal(first, second)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = serve()
    for i in range(4):
        x.copy_(data(90, 288, "bf16", 20 + i))
        off.copy_(torch.tensor([0, 20 * i, 20 * i + 5, 90], dtype=torch.int32))
        graph.replay()
        want = serve()
        torch.cuda.synchronize()
        assert torch.equal(held, want)


@pytest.mark.parametrize("T,R,K", [(3, 70, 9248), (40, 100, 8224), (300, 300, 11264)])
def test_gemm_long(T, R, K):
    log(f"mx gemm long {T}x{R}x{K}")
    check_gemm(T, R, K, "f32")


@pytest.mark.parametrize("E_,T", [(70, 90), (300, 500), (300, 30000)])
def test_gemm_of_many_experts(E_, T):
    """More experts than a wave looks at in one go; enough for a table of tiles; many rows."""
    log(f"mx gemm experts={E_} T={T}")
    R, K = 40, 64
    lengths = np.bincount(np.random.default_rng(E_).integers(0, E_, T), minlength=E_)
    lengths[3] = 0
    T = int(lengths.sum())
    off = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    w, wq, ws = operands(R, K, 3, E_)
    x, xq, xs = operands(T, K, 4)
    y = nm.nm_mx_gemm(wq, ws, xq, xs, torch.from_numpy(off).cuda())
    torch.cuda.synchronize()
    ids = np.repeat(np.arange(E_), lengths)
    ref = np.einsum("tk,trk->tr", x, w[ids]) if T < 1000 else np.concatenate(
        [x[off[e]: off[e + 1]] @ w[e].T for e in range(E_)])
    size = np.concatenate([np.abs(x[off[e]: off[e + 1]]) @ np.abs(w[e]).T for e in range(E_)])
    within(f64(y), ref, size, K, "f32")


@pytest.mark.parametrize("T", [12, 300])
@pytest.mark.parametrize("offsets", [[-5, 700, 3, 90], [400, 100, 300, 0], [0, 5, 2 ** 31 - 1, -2 ** 31], [0, 300, 0, 300]])
def test_broken_offsets_stay_inside(offsets, T):
    """Clamped (the rule is run over every small list by test_host_offsets); nothing around Y changes."""
    log(f"mx broken offsets {offsets} T={T}")
    w, wq, ws = operands(136, 160, 3, 3)
    x, xq, xs = operands(T, 160, 4)
    whole = torch.full((T + 600, 144), 77.0, device="cuda")
    nm.nm_mx_gemm(wq, ws, xq, xs, torch.tensor(offsets, dtype=torch.int32, device="cuda"), out=whole[300: 300 + T, :136])
    torch.cuda.synchronize()
    got = whole.cpu().numpy()
    assert (got[:300] == 77.0).all() and (got[300 + T:] == 77.0).all() and (got[:, 136:] == 77.0).all()
