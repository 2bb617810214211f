"""Stacks of 4-bit matrices on MI355X whose scales do not begin on 16 bytes (odd rows, an odd
number of panels of 256 columns): quantised and back, and multiplied, as a whole and one matrix
at a time.  Codes and values are equal to the oracle's; a product of one matrix of a stack is
the same call on other addresses, so it is equal to that of a copy of its own."""
import numpy as np
import pytest

import structured_sparse_gemm_nm_amd as nm
from oracle import nm_experts as E
from gpu_util import log

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def stack(n, R, K, dt, seed=0):
    g = torch.Generator().manual_seed(seed * 1000003 + R * 131 + K)
    x = torch.randn(n, R, K, generator=g) * 2.0 ** torch.randint(-6, 6, (n, R, 1), generator=g)
    return x.to(DT[dt]).cuda()


def check(x):
    """q, scale of the stack x, held against the oracle's of each matrix."""
    q, s = nm.nm_mx_quantize(x)
    back = {dt: nm.nm_mx_dequantize(q, s, DT[dt]) for dt in DT}
    torch.cuda.synchronize()
    for e in range(x.shape[0]):
        code, byte = E.mx_quantize_ref(x[e].double().cpu().numpy())
        rq, rs = E.mx_pack_ref(code, byte)
        assert (q[e].cpu().numpy() == rq).all() and (s[e].cpu().numpy() == rs).all()
        values = torch.from_numpy(E.mx_values_ref(code, byte))
        for dt in DT:
            assert torch.equal(back[dt][e].cpu(), values.to(DT[dt]))
    return q, s, back


@pytest.mark.parametrize("n,R,K", [(3, 101, 256), (3, 101, 64), (4, 7, 544), (3, 1, 32), (1, 5, 96), (2, 33, 288)])
@pytest.mark.parametrize("dt", list(DT))
def test_stack_and_each_of_its_matrices(n, R, K, dt):
    log(f"mx stack {n} x {R} x {K} {dt}")
    x = stack(n, R, K, dt)
    q, s, back = check(x)
    for e in range(n):                       # views of the stack: their scales begin on 8 bytes
        assert torch.equal(nm.nm_mx_dequantize(q[e], s[e]), back["f32"][e])
        one, scale = nm.nm_mx_quantize(x[e])
        assert torch.equal(one, q[e]) and torch.equal(scale, s[e])
    torch.cuda.synchronize()


def test_stack_strides():
    """Matrices and rows further apart, at any element, one behind all of them, none at all."""
    log("mx stack strides")
    for dt in DT:
        base = stack(6, 22, 200, dt, 1)
        for x in (base[::2], base[:, ::2, 8:168], base[1:4, 3:14, 3:35], base[0].expand(3, 22, 200)[:, :, :192],
                  base[:, 0::22, :64], base.permute(1, 0, 2)[:, :, :96]):
            x = x[:, :, : x.shape[2] // 32 * 32]
            check(x)
    assert nm.nm_mx_quantize(base[:0, :, :64])[0].shape == (0, 22, 32)
    assert nm.nm_mx_dequantize(*nm.nm_mx_quantize(base[:, :0, :64])).shape == (6, 0, 64)
    torch.cuda.synchronize()


def test_more_matrices_than_a_grid_takes():
    log("mx stack of 65539")
    x = stack(65539, 1, 32, "bf16")
    q, s = nm.nm_mx_quantize(x)
    back = nm.nm_mx_dequantize(q, s, torch.bfloat16)
    flat_q, flat_s = nm.nm_mx_quantize(x.view(-1, 32))       # the same rows as one matrix of one panel
    torch.cuda.synchronize()
    assert torch.equal(q.view(-1, 16), flat_q) and torch.equal(s.view(-1, 8), flat_s.view(-1, 8))
    assert torch.equal(back.view(-1, 32), nm.nm_mx_dequantize(flat_q, flat_s, torch.bfloat16))


@pytest.mark.parametrize("K", [64, 256, 544])
@pytest.mark.parametrize("T", [5, 40, 301])
def test_products_of_a_stacks_matrices(T, K):
    """Few rows and tiles: one weight of a stack, one matrix of a stack of activations, and the
    stack itself under experts, all with scales on 8 bytes."""
    log(f"mx stack products T={T} K={K}")
    R = 101
    wq, ws = nm.nm_mx_quantize(stack(3, R, K, "f32", 2))
    xq, xs = nm.nm_mx_quantize(stack(2, T, K, "f32", 3))
    assert ws[1].data_ptr() % 16 == 8
    x1, xs1 = xq[1].clone(), xs[1].clone()
    want = [nm.nm_mx_gemm(wq[e].clone(), ws[e].clone(), x1, xs1) for e in range(3)]
    for e in range(3):
        assert torch.equal(nm.nm_mx_gemm(wq[e], ws[e], xq[1], xs[1]), want[e])
    code, byte = (E.mx_quantize_ref(stack(2, T, K, "f32", 3)[1].double().cpu().numpy()))
    x = E.mx_values_ref(code, byte)
    w = E.mx_values_ref(*E.mx_quantize_ref(stack(3, R, K, "f32", 2)[1].double().cpu().numpy()))
    got = want[1].double().cpu().numpy()
    # K exact products in any order with unit 2^-23, and the output's rounding
    assert (np.abs(got - x @ w.T) <= K * 2.0 ** -23 * (np.abs(x) @ np.abs(w).T) + np.abs(x @ w.T) * 2.0 ** -24 + 1e-30).all()
    ends = [0, T // 3, T // 3, T]
    y = nm.nm_mx_gemm(wq, ws, xq[1], xs[1], torch.tensor(ends, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    for e in range(3):
        lo, hi = ends[e], ends[e + 1]
        size = np.abs(x[lo:hi]) @ np.abs(E.mx_values_ref(*E.mx_quantize_ref(stack(3, R, K, "f32", 2)[e].double().cpu().numpy()))).T
        diff = (y[lo:hi] - want[e][lo:hi]).double().cpu().numpy()
        assert (np.abs(diff) <= 2 * (K * 2.0 ** -23 + 2.0 ** -24) * size + 2e-30).all()
