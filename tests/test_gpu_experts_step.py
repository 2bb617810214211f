"""The grouped products, the clipping and the 4-bit floats as they are used together: a
layer of experts trained with its pattern held, its gradients clipped, and served in
four bits, against the same step in float64.
"""
import numpy as np
import pytest

import structured_sparse_gemm_nm_amd as nm
from oracle import nm_experts as E
from oracle import nm_oracle as O
from gpu_util import bits_of, log

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def route(T, E_, seed):
    """(order, offsets): tokens ordered by the expert each one is sent to, two a token."""
    g = torch.Generator().manual_seed(seed)
    ids = torch.rand(T, E_, generator=g).topk(2, dim=1).indices.reshape(-1)
    order = torch.argsort(ids, stable=True)
    offsets = torch.zeros(E_ + 1, dtype=torch.int32)
    offsets[1:] = torch.bincount(ids, minlength=E_).cumsum(0)
    return (order // 2).cuda(), offsets.cuda()


def dense(values, idx, K, n, m):
    v, i = bits_of(values), idx.cpu().numpy().view(np.uint32)
    return torch.stack([torch.from_numpy(O.half_bits_to_f64(O.decompress(v[e], i[e], K, n, m), "bf16"))
                        for e in range(v.shape[0])])


class Layer:
    """Two grouped products with a ReLU between, on packed weights."""

    def __init__(self, E_, H, F, pat, seed):
        g = torch.Generator().manual_seed(seed)
        self.n, self.m = pat
        self.H, self.F = H, F
        self.up = self.pack(torch.randn(E_, F, H, generator=g) * H ** -0.5)
        self.down = self.pack(torch.randn(E_, H, F, generator=g) * F ** -0.5)

    def pack(self, w):
        E_, R, K = w.shape
        v, i = nm.nm_compress(w.to(BF).cuda().view(E_ * R, K), self.n, self.m)
        return v.view(E_, R, -1), i.view(E_, R, -1)

    def step(self, x, order, offsets, target):
        """(loss's gradient outputs): y, dx, and the two packed gradients."""
        xs = x[order].contiguous()
        h = nm.nm_group_spmm(*self.up, xs, offsets, self.H, self.n, self.m, out_dtype=BF)
        a = torch.relu(h)
        y = nm.nm_group_spmm(*self.down, a, offsets, self.F, self.n, self.m, out_dtype=BF)
        gy = (y - target).contiguous()                  # of 0.5 |y - target|^2
        ga = nm.nm_group_spmm_dx(*self.down, gy, offsets, self.F, self.n, self.m, out_dtype=BF)
        gh = (ga * (h > 0)).contiguous()
        d_down = nm.nm_group_spmm_dw(self.down[1], gy, a, offsets, self.F, self.n, self.m, out_dtype=BF)
        d_up = nm.nm_group_spmm_dw(self.up[1], gh, xs, offsets, self.H, self.n, self.m, out_dtype=BF)
        dx = nm.nm_group_spmm_dx(*self.up, gh, offsets, self.H, self.n, self.m)
        return y, dx, d_up, d_down


@pytest.mark.parametrize("T,E_,H,F,pat", [(3, 8, 64, 96, (2, 4)), (40, 4, 96, 160, (1, 4)), (300, 5, 160, 256, (1, 8)),
                                          (700, 3, 256, 320, (2, 4))])
def test_training_step(T, E_, H, F, pat):
    log(f"experts step T={T} E={E_} {H}x{F} {pat}")
    g = torch.Generator().manual_seed(T)
    layer = Layer(E_, H, F, pat, 7)
    x = torch.randn(T, H, generator=g).to(BF).cuda()
    target = torch.randn(2 * T, H, generator=g).to(BF).cuda()
    order, offsets = route(T, E_, 5)
    y, dx, d_up, d_down = layer.step(x, order, offsets, target)
    before = [layer.up[0].clone(), layer.down[0].clone()]
    norm, clipped = nm.nm_grad_clip([d_up, d_down, dx], 1.0, out=[torch.empty_like(t) for t in (d_up, d_down, dx)])
    torch.cuda.synchronize()
    # the same step in float64, each stored intermediate rounded to bf16 as the step rounds it
    wu, wd = dense(*layer.up, H, *pat), dense(*layer.down, F, *pat)
    off = offsets.tolist()
    xs = x[order].double().cpu()
    rnd = lambda t: t.to(BF).double()
    per = lambda rows, w: torch.cat([rows[off[e]: off[e + 1]] @ w[e].t() for e in range(E_)])
    back = lambda rows, w: torch.cat([rows[off[e]: off[e + 1]] @ w[e] for e in range(E_)])
    h = per(xs, wu)
    # the layer's own h decides the ReLU: a value near zero may round to either side
    hs = nm.nm_group_spmm(*layer.up, x[order].contiguous(), offsets, H, *pat, out_dtype=BF).double().cpu()
    u = 2.0 ** -8
    assert (hs - h).abs().max() <= u * h.abs().max() * 1.05
    a = torch.relu(hs)
    ry = per(a, wd)
    assert (y.double().cpu() - ry).abs().max() <= u * ry.abs().max() * 1.05
    gy = rnd(y.double().cpu() - target.double().cpu())
    ga = back(gy, wd)
    gh = rnd(ga) * (hs > 0)
    rdx = back(gh, wu)
    # gh was rounded on both sides, by at most one step apart where their sums straddle a midpoint
    assert (dx.double().cpu() - rdx).abs().max() <= 4 * u * rdx.abs().max()
    for got, rows, cols, (v, i), K in ((d_down, gy, a, layer.down, F), (d_up, gh, xs, layer.up, H)):
        full = torch.stack([rows[off[e]: off[e + 1]].t() @ cols[off[e]: off[e + 1]] for e in range(E_)])
        from oracle.nm_train import stored_columns
        words = i.cpu().numpy().view(np.uint32)
        ref = torch.stack([torch.gather(full[e], 1, torch.from_numpy(stored_columns(words[e], K, *pat)).long())
                           for e in range(E_)])
        assert got.shape == v.shape and (got.double().cpu() - ref).abs().max() <= 4 * u * ref.abs().max() + 1e-30
    want = torch.sqrt(sum((t.double() ** 2).sum() for t in (d_up, d_down, dx)))
    assert abs(float(norm) - float(want)) <= 2.0 ** -23 * float(want)
    total = torch.sqrt(sum((t.double() ** 2).sum() for t in clipped))
    assert float(total) <= 1.0 + 2.0 ** -8
    # the update stays in the packed layout and takes effect in the next product
    layer.up[0].sub_(0.1 * clipped[0])
    layer.down[0].sub_(0.1 * clipped[1])
    assert not torch.equal(before[0], layer.up[0])
    y2 = layer.step(x, order, offsets, target)[0]
    torch.cuda.synchronize()
    loss = lambda t: float((t.double() - target.double()).square().sum())
    assert np.isfinite(loss(y2)) and loss(y2) != loss(y)


def test_step_in_a_graph():
    """The whole step and the clipping captured once, replayed with other tokens and other routes."""
    log("experts step in a graph")
    T, E_, H, F = 120, 4, 96, 160
    layer = Layer(E_, H, F, (2, 4), 3)
    x, target = torch.zeros(T, H, dtype=BF, device="cuda"), torch.zeros(2 * T, H, dtype=BF, device="cuda")
    order, offsets = route(T, E_, 0)
    grads = [torch.empty_like(layer.up[0]), torch.empty_like(layer.down[0])]
    held = nm.nm_grad_list(grads)

    def step():
        y, dx, d_up, d_down = layer.step(x, order, offsets, target)
        grads[0].copy_(d_up)
        grads[1].copy_(d_down)
        norm, _ = nm.nm_grad_clip(held, 0.5)
        return y, dx, norm
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = step()
    for i in range(4):
        g = torch.Generator().manual_seed(i)
        x.copy_(torch.randn(T, H, generator=g))
        target.copy_(torch.randn(2 * T, H, generator=g))
        o, f = route(T, E_, 10 + i)
        order.copy_(o)
        offsets.copy_(f)
        graph.replay()
        mine = [t.clone() for t in (*kept, *grads)]
        want = step()
        torch.cuda.synchronize()
        for a, b in zip(mine, (*want, *grads)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("T", [1, 9, 200])
def test_served_in_four_bits(T):
    """The trained experts' weights in four bits: quantised once, each call's tokens as they come."""
    log(f"experts served T={T}")
    E_, H, F = 4, 160, 288
    layer = Layer(E_, H, F, (2, 4), 11)
    wu = torch.stack([nm.nm_decompress(layer.up[0][e], layer.up[1][e], H) for e in range(E_)])
    wq, ws = nm.nm_mx_quantize(wu)
    order, offsets = route(T, E_, T)
    x = torch.randn(T, H, generator=torch.Generator().manual_seed(T)).to(BF).cuda()[order].contiguous()
    xq, xs = nm.nm_mx_quantize(x)
    y = nm.nm_mx_gemm(wq, ws, xq, xs, offsets)
    torch.cuda.synchronize()
    w64 = nm.nm_mx_dequantize(wq, ws).double().cpu()
    x64 = nm.nm_mx_dequantize(xq, xs).double().cpu()
    off = offsets.tolist()
    for e in range(E_):
        rows = x64[off[e]: off[e + 1]]
        ref, size = rows @ w64[e].t(), rows.abs() @ w64[e].abs().t()
        err = (y[off[e]: off[e + 1]].double().cpu() - ref).abs()
        assert (err <= H * 2.0 ** -23 * size + 1e-30).all()
    # four bits hold a value to a quarter of its block's largest at worst: the product follows the weights
    plain = torch.cat([x[off[e]: off[e + 1]].double().cpu() @ wu[e].double().cpu().t() for e in range(E_)])
    assert float((y.double().cpu() - plain).norm() / plain.norm()) < 0.3


@pytest.mark.parametrize("pat", [(2, 4), (1, 4), (1, 8)])
@pytest.mark.parametrize("T,seed", [(12, 1), (400, 2)])
def test_gradients_against_differences(pat, T, seed):
    """sum G Y is linear in act and in the stored weights, so a central difference of products is the
    directional derivative: values, directions and steps are short binary fractions, exact in fp16."""
    log(f"group differences {pat} T={T}")
    E_, R, K = 3, 48, 96
    g = torch.Generator().manual_seed(seed)
    w = (torch.randint(-64, 65, (E_, R, K), generator=g) / 64).to(torch.float16).cuda()
    v, i = nm.nm_compress(w.view(E_ * R, K), *pat)
    v, i = v.view(E_, R, -1), i.view(E_, R, -1)
    act = (torch.randint(-32, 33, (T, K), generator=g) / 32).to(torch.float16).cuda()
    G = (torch.randint(-32, 33, (T, R), generator=g) / 32).to(torch.float16).cuda()
    da = torch.randint(-1, 2, (T, K), generator=g).to(torch.float16).cuda()
    dv = torch.randint(-1, 2, v.shape, generator=g).to(torch.float16).cuda()
    off = torch.tensor([0, T // 3, T // 3, T], dtype=torch.int32, device="cuda")
    f = lambda vv, aa: (G.double() * nm.nm_group_spmm(vv, i, aa, off, K, *pat).double()).sum()
    dx = nm.nm_group_spmm_dx(v, i, G, off, K, *pat).double()
    dw = nm.nm_group_spmm_dw(i, G, act, off, K, *pat).double()
    h = 0.25
    # every product here is a multiple of 2^-13 below 2^11 in a sum below 2^24 steps: exact in fp32
    assert float(f(v, act + h * da) - f(v, act - h * da)) / (2 * h) == pytest.approx(float((dx * da).sum()), abs=1e-9)
    assert float(f(v + h * dv, act) - f(v - h * dv, act)) / (2 * h) == pytest.approx(float((dw * dv).sum()), abs=1e-9)
