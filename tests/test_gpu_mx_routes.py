"""The largest tiles of the 4-bit product against the float64 oracle: one weight and experts, one
and several steps of K, whole and part ones, every output type, rows of outputs on any element.
Bounds as in test_gpu_mx: K exact products in any order with unit 2^-23, and half a step of the
output's type.  Which tiles a call takes is held against the rule, written down here once more."""
import numpy as np
import pytest

import structured_sparse_gemm_nm_amd as nm
from oracle import nm_experts as E
from gpu_util import log
from test_gpu_mx import DT, f64, within

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def route(weights, R, T):
    """`weights`: those that can have rows (1 without offsets)."""
    rows = T // weights
    if rows <= 64:
        return "few"
    return "large" if weights * -(-rows // 256) * -(-R // 256) >= 256 else "middle"


def operand(rows, K, seed):
    """(values in float64, q, scale) of rows x K numbers in scales from 2^-6 to 2^1."""
    g = np.random.default_rng(seed * 1000003 + rows * 131 + K)
    x = (g.standard_normal((rows, K), dtype=np.float32) * 2.0 ** g.integers(-4, 2, (rows, 1))).astype(np.float64)
    code, byte = E.mx_quantize_ref(x)
    return E.mx_values_ref(code, byte), *(torch.from_numpy(a).cuda() for a in E.mx_pack_ref(code, byte))


@pytest.mark.parametrize("K", [32, 256, 288, 544, 1056])
def test_large_tiles(K):
    log(f"mx large tiles K={K}")
    T, R = 4090, 4100
    assert route(1, R, T) == "large"
    w, wq, ws = operand(R, K, 1)
    x, xq, xs = operand(T, K, 2)
    ref, size = x @ w.T, np.abs(x) @ np.abs(w).T
    for out, ldpad in [("f32", 0), ("f32", 1), ("bf16", 4), ("bf16", 3), ("f16", 0), ("f16", 12)]:
        whole = torch.full((T + 2, R + ldpad), 77.0, dtype=DT[out], device="cuda")
        nm.nm_mx_gemm(wq, ws, xq, xs, out_dtype=DT[out], out=whole[:T, :R])
        torch.cuda.synchronize()
        within(f64(whole[:T, :R]), ref, size, K, out)
        assert (whole[T:].float() == 77.0).all() and (whole[:, R:].float() == 77.0).all()


@pytest.mark.parametrize("E_,R,K,mean", [(64, 1030, 288, 100), (64, 1030, 544, 100), (300, 200, 96, 70)])
def test_large_tiles_of_experts(E_, R, K, mean):
    """Some experts without rows, one with several tiles; more of them than a workgroup looks through."""
    log(f"mx large tiles of {E_} experts R={R} K={K}")
    lengths = np.bincount(np.random.default_rng(E_).integers(0, E_, E_ * mean), minlength=E_)
    lengths[3], lengths[E_ // 2], lengths[-1] = 0, 700, 257
    before, behind = 3, 5
    off = np.cumsum([before, *lengths]).astype(np.int32)
    T = int(off[-1]) + behind
    assert route(E_, R, T) == ("large" if -(-R // 256) * E_ >= 256 else "middle") == "large"
    w = [operand(R, K, 10 + e) for e in range(E_)]
    wq, ws = (torch.stack([p[i] for p in w]) for i in (1, 2))
    x, xq, xs = operand(T, K, 2)
    xs[:, :before], xs[:, T - behind:] = 255, 255              # rows of no expert: NaN
    for out, ldpad in [("bf16", 2), ("f16", 8), ("f32", 5)]:
        whole = torch.full((T + 2, R + ldpad), 77.0, dtype=DT[out], device="cuda")
        nm.nm_mx_gemm(wq, ws, xq, xs, torch.from_numpy(off).cuda(), out_dtype=DT[out], out=whole[:T, :R])
        torch.cuda.synchronize()
        got = f64(whole)
        assert (got[:before] == 77.0).all() and (got[T - behind:] == 77.0).all() and (got[:, R:] == 77.0).all()
        for e, (lo, hi) in enumerate(zip(off[:-1], off[1:])):
            if lo < hi:
                within(got[lo:hi, :R], x[lo:hi] @ w[e][0].T, np.abs(x[lo:hi]) @ np.abs(w[e][0]).T, K, out)


@pytest.mark.parametrize("T", [300, 4090])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_nan_blocks(T, out):
    """A NaN exponent in each of several steps, the part one among them, makes its row or column NaN
    and nothing else; bytes behind the last block are not looked at."""
    R, K = 4100, 544
    log(f"mx NaN blocks T={T} {out}")
    assert route(1, R, T) == {300: "middle", 4090: "large"}[T]
    _, wq, ws = operand(R, K, 1)
    _, xq, xs = operand(T, K, 2)
    clean = nm.nm_mx_gemm(wq, ws, xq, xs, out_dtype=DT[out])
    ws[2, :, 1:], xs[2, :, 1:] = 255, 255
    again = nm.nm_mx_gemm(wq, ws, xq, xs, out_dtype=DT[out])
    xs[0, 2, 3], xs[1, 270, 7], xs[2, 131, 0] = 255, 255, 255
    ws[0, 7, 0], ws[1, 300, 2], ws[2, 4099, 0] = 255, 255, 255
    y = nm.nm_mx_gemm(wq, ws, xq, xs, out_dtype=DT[out])
    torch.cuda.synchronize()
    assert torch.isfinite(clean).all() and torch.equal(clean, again)
    nan = torch.zeros(T, R, dtype=torch.bool, device="cuda")
    nan[[2, 270, 131]] = True
    nan[:, [7, 300, 4099]] = True
    assert torch.equal(torch.isnan(y), nan) and torch.equal(y[~nan], clean[~nan])


def test_large_tiles_on_another_stream_and_captured():
    log("mx large tiles, side stream, graph")
    T, R, K = 4090, 4100, 544
    _, wq, ws = operand(R, K, 1)
    _, xq, xs = operand(T, K, 2)
    first = nm.nm_mx_gemm(wq, ws, xq, xs, out_dtype=torch.bfloat16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = nm.nm_mx_gemm(wq, ws, xq, xs, out_dtype=torch.bfloat16)
    third = nm.nm_mx_gemm(wq, ws, xq, xs, out_dtype=torch.bfloat16)
    torch.cuda.synchronize()
    assert torch.equal(first, second) and torch.equal(first, third)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = nm.nm_mx_gemm(wq, ws, xq, xs, out_dtype=torch.bfloat16)
    for i in range(3):
        xq.copy_(xq.roll(i + 1, 0))
        graph.replay()
        want = nm.nm_mx_gemm(wq, ws, xq, xs, out_dtype=torch.bfloat16)
        torch.cuda.synchronize()
        assert torch.equal(held, want)
