"""What the adapters keep between their two products: xa and u (fp32) enter the matrix
cores in three bf16 parts, which hold all 24 bits, and an fp16 A or B in two.

Whole numbers chosen so that every product and every partial sum, in any order and
split into parts, is a whole number below 2^24: the results are exact, and a part
that went missing, or one rounded away, changes them.  Each case asserts that on the
host, and that two parts would not have held its xa or u.
"""
import numpy as np
import pytest

import nm_inputs
import structured_sparse_gemm_nm_amd as nm
from oracle import nm_layers as L
from oracle import nm_oracle as O
from gpu_util import log, torch_dtype
from test_gpu_adapter import Case, f64

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

LIMIT = 2 ** 24     # of twice a result: one adapter's scale is 0.5


def whole(shape, low, most, dt, *seed):
    return nm_inputs.integer_half(shape, low, most, dt, 97, *seed)


def in_parts(v, n):
    """v as n bf16 parts hold it."""
    kept, rest = np.zeros_like(v), v.copy()
    for _ in range(n):
        part = nm_inputs.to_half_bits(rest.astype(np.float32), "bf16")
        part = O.half_bits_to_f64(part.reshape(-1), "bf16").reshape(v.shape)
        kept, rest = kept + part, rest - part
    return kept


def make(R, K, T, r, dt, n=2, m=4, na=3):
    """Tokens of three adapters in turn, every fourth without one; weights of 0 and +-1."""
    c = Case(R, K, T, r, na, dt, n, m, ids=np.arange(T) % (na + 1) - 1)
    w = whole((R, K), -1, 1, dt, 0, R + T)
    c.vals, c.idx = O.prune_pack(w, n, m)
    c.w = O.half_bits_to_f64(O.decompress(c.vals, c.idx, K, n, m), dt)
    c.scale = np.array([1.0, 2.0, 0.5], dtype=np.float32)
    return c


def ends_only(bits):
    """Two tokens of each adapter, one from either end; the others' rows are zeros."""
    bits = bits.copy()
    bits[4:-4] = 0
    return bits


def needs_three(v):
    assert np.array_equal(in_parts(v, 3), v) and (in_parts(v, 2) != v).mean() > 0.25


# the kernel a forward pass takes: 2:4 prefill, the product in shares, what nm_spmm
# chooses (with 16 and 64 columns a wave), and the few-token kernel (fp32 throughout)
FORWARD = [(256, 128, 130, 2, 4), (48, 1056, 40, 2, 4), (40, 1024, 33, 1, 8), (136, 96, 50, 2, 4), (3456, 96, 300, 2, 4),
           (64, 128, 15, 2, 4)]


@pytest.mark.parametrize("R,K,T,n,m", FORWARD)
@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("r", [1, 6, 8])
def test_forward_keeps_24_bits(R, K, T, n, m, dt, r):
    log(f"adapter 24 bits R={R} K={K} T={T} r={r} {n}:{m} {dt}")
    c = make(R, K, T, r, dt, n, m)
    c.act = whole((T, K), 0, 255, dt, 1, T)
    c.act[:, 96:] = 0                                   # xa sums 96 products: about 1.5e6
    c.A = whole((3 * r, K), 0, 255, dt, 2, r).reshape(3, r, K)
    c.B = whole((3 * R, r), -1, 1, dt, 4, r).reshape(3, R, r)
    c.B[:, :, 2:] = 0
    c.B[1, :, 1:] = 0                                   # the adapter whose scale is 2
    x, _, A, B, s = c.wide()
    y, xa = L.adapter_ref(c.w, x, c.ids, A, B, s)
    assert (L.adapter_ref(np.abs(c.w), x, c.ids, A, np.abs(B), s)[0] * 2).max() < LIMIT
    needs_three(xa[c.ids >= 0])
    got, gxa = c.forward()
    assert np.array_equal(gxa.double().cpu().numpy(), xa) and np.array_equal(got.double().cpu().numpy(), y)


@pytest.mark.parametrize("T", [7, 40, 200])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("r", [1, 6, 24, 40])
def test_backward_keeps_24_bits(T, dt, r):
    # u = s B^T g of 20 bits into dX = W^T g + A^T u and dA = sum u x^T; xa of 20 bits,
    # given, into dB = s sum g xa^T
    log(f"adapter 24 bits backward T={T} r={r} {dt}")
    R, K = 136, 96
    c = make(R, K, T, r, dt)
    c.g = whole((T, R), 0, 255, dt, 1, T)
    c.g[:, 64:] = 0
    c.B = whole((3 * R, r), 0, 255, dt, 3, r).reshape(3, R, r)
    c.A = whole((3 * r, K), -1, 1, dt, 4, r).reshape(3, r, K)
    c.A[:, 2:] = 0
    c.act = ends_only(whole((T, K), -1, 1, dt, 5, T))
    xa = np.random.default_rng(r).integers(-2 ** 19, 2 ** 19, size=(T, r)).astype(np.float64) * 2 + 1
    xa[c.ids < 0] = 0
    x, g, A, B, s = c.wide()
    d, G = c.dev()
    ab = np.abs
    ref = L.adapter_bwd_ref(c.w, g, x, xa, c.ids, A, B, s)
    mag = L.adapter_bwd_ref(ab(c.w), g, ab(x), ab(xa), c.ids, ab(A), B, s)
    assert (mag[0] * 2).max() < LIMIT and (mag[1] * 2).max() < LIMIT
    needs_three(xa[c.ids >= 0])
    needs_three(np.stack([s[a] * (g[t] @ B[a]) for t, a in enumerate(c.ids) if a >= 0]))
    X = torch.from_numpy(xa.astype(np.float32)).cuda()
    got = nm.nm_adapter_spmm_bwd(G=G, xa=X, **d, K=K)
    torch.cuda.synchronize()
    for t, q in zip(got[:2], ref[:2]):
        assert np.array_equal(t.double().cpu().numpy(), q)
    # dB, from small gradients of its own
    g = f64(ends_only(whole((T, R), -1, 1, dt, 6, T)), dt)
    ref = L.adapter_bwd_ref(c.w, g, x, xa, c.ids, A, B, s)[2]
    assert (L.adapter_bwd_ref(ab(c.w), ab(g), ab(x), ab(xa), c.ids, ab(A), B, s)[2] * 2).max() < LIMIT
    dB = nm.nm_adapter_spmm_bwd(G=torch.from_numpy(g).to(torch_dtype(dt)).cuda(), xa=X, **d, K=K)[2]
    assert np.array_equal(dB.double().cpu().numpy(), ref)


def test_f16_weights_of_11_bits():
    # A and B of 11 bits, which one bf16 part does not hold
    log("adapter 11 bits")
    for T in (33, 200):
        c = make(256, 128, T, 8, "f16")
        c.act, c.g = whole((T, 128), -1, 1, "f16", 1, T), whole((T, 256), -1, 1, "f16", 2, T)
        c.act[:, 16:], c.g[:, 16:] = 0, 0
        c.A = whole((24, 128), -15, 15, "f16", 3).reshape(3, 8, 128)
        c.B = whole((3 * 256, 8), -2047, 2047, "f16", 4).reshape(3, 256, 8)
        x, g, A, B, s = c.wide()
        y, xa = L.adapter_ref(c.w, x, c.ids, A, B, s)
        assert (in_parts(B, 1) != B).mean() > 0.5
        assert (2 * L.adapter_ref(np.abs(c.w), np.abs(x), c.ids, np.abs(A), np.abs(B), s)[0]).max() < LIMIT
        got, gxa = c.forward()
        assert np.array_equal(got.double().cpu().numpy(), y)
        # the backward pass's A, and its x and g, take the same two parts
        c.A, c.B = whole((24, 128), -2047, 2047, "f16", 5).reshape(3, 8, 128), whole((3 * 256, 8), -15, 15, "f16", 6).reshape(3, 256, 8)
        c.act = whole((T, 128), -2047, 2047, "f16", 7, T)
        c.act[np.random.default_rng(T).random(c.act.shape) > 8 / T] = 0
        x, g, A, B, s = c.wide()
        d, G = c.dev()
        xa = np.ones((T, 8))
        ab = np.abs
        ref = L.adapter_bwd_ref(c.w, g, x, xa, c.ids, A, B, s)
        mag = L.adapter_bwd_ref(ab(c.w), ab(g), ab(x), xa, c.ids, ab(A), ab(B), s)
        assert max((2 * q).max() for q in mag) < LIMIT
        out = nm.nm_adapter_spmm_bwd(G=G, xa=torch.ones(T, 8, device="cuda"), **d, K=128)
        torch.cuda.synchronize()
        for t, q in zip(out, ref):
            assert np.array_equal(t.double().cpu().numpy(), q)
