"""Global norm of gradients and clipping on MI355X (nm_grad_norm, nm_grad_clip)
against the oracle in extended precision.

Bounds: squares are summed in 64 bits, where n <= 2^28 terms in any order are off by
at most 2^28 2^-53 of their sum; the norm is then rounded once to fp32 (2^-24).  The
factor and its product with an element are rounded to fp32 (2^-24 each), then to the
output's type.
"""
import numpy as np
import pytest

import structured_sparse_gemm_nm_amd as nm
from oracle import nm_experts as E
from gpu_util import log

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
# half a step, and half the smallest spacing
ROUND = {torch.bfloat16: (2.0 ** -8, 2.0 ** -134), torch.float16: (2.0 ** -11, 2.0 ** -25),
         torch.float32: (2.0 ** -24, 2.0 ** -150)}
SUM = 2.0 ** -25


def f64(t):
    return t.detach().double().cpu().numpy()


def grads(shapes, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed + 17)
    return [(torch.randn(s, generator=g) * scale).to(DT[dt]).cuda() for s, dt in shapes]


def check(gs, max_norm, eps=1e-6, in_place=False):
    ref_norm, ref = E.grad_clip_ref([f64(g) for g in gs], max_norm, eps)
    n = nm.nm_grad_norm(gs)
    before = [g.clone() for g in gs]
    norm, out = nm.nm_grad_clip(gs, max_norm, eps, out=None if in_place else [torch.empty_like(g) for g in gs])
    torch.cuda.synchronize()
    assert n.shape == () and torch.equal(n, norm)
    if ref_norm > 3.41e38:                 # past fp32's largest value, 3.403e38: it rounds to Inf
        assert float(norm) == float("inf")
    else:
        assert abs(float(norm) - ref_norm) <= (2.0 ** -24 + SUM) * ref_norm + 2.0 ** -150
    for o, r, g, b in zip(out, ref, gs, before):
        assert o.dtype == g.dtype and o.shape == g.shape
        rel, tiny = ROUND[g.dtype]
        bound = np.abs(r) * (rel + 3 * 2.0 ** -24 + SUM) * 1.001 + tiny + 2.0 ** -149
        assert (np.abs(f64(o) - r) <= bound).all()
        assert in_place or torch.equal(g, b)
        assert not in_place or o is g
    return norm, out


MIXED = [((64, 33), "f32"), ((1,), "bf16"), ((0,), "f16"), ((7, 5, 3), "f16"), ((16385,), "bf16"), ((8192,), "f32"),
         ((8193,), "f32"), ((16384,), "f16"), ((100001,), "bf16"), ((3,), "f32")]


@pytest.mark.parametrize("max_norm", [0.0, 0.3, 50.0, 1e9, float("inf")])
@pytest.mark.parametrize("in_place", [False, True])
def test_mixed_tensors(max_norm, in_place):
    log(f"grad mixed {max_norm} {in_place}")
    check(grads(MIXED), max_norm, in_place=in_place)


@pytest.mark.parametrize("n", [1, 2, 7, 8, 255, 4095, 4096, 4097, 8191, 16383, 16384, 16385, 32769, 300000])
@pytest.mark.parametrize("dt", list(DT))
def test_sizes(n, dt):
    log(f"grad {n} {dt}")
    check(grads([((n,), dt)], n), 0.5)


def test_no_tensors_and_empty_ones():
    log("grad empty lists")
    norm, out = nm.nm_grad_clip([], 1.0)
    assert float(norm) == 0.0 and out == [] and float(nm.nm_grad_norm([])) == 0.0
    check(grads([((0,), "f32"), ((0, 5), "bf16")]), 1.0)
    check([torch.zeros(1000, device="cuda")], 0.0, eps=0.0)        # 0 / 0: the factor is 1


@pytest.mark.parametrize("count", [132, 133, 180, 181, 400, 2000])
def test_many_tensors(count):
    """More tensors than one launch takes, of odd sizes."""
    log(f"grad {count} tensors")
    rng = np.random.default_rng(count)
    shapes = [((int(k),), ["f32", "bf16", "f16"][i % 3]) for i, k in enumerate(rng.integers(0, 3000, count))]
    check(grads(shapes, count), 1.0)
    check(grads(shapes, count), 1.0, in_place=True)


@pytest.mark.parametrize("off", [1, 2, 3, 5])
@pytest.mark.parametrize("dt", list(DT))
def test_unaligned_views(off, dt):
    """Views at any element, and outputs at another: nothing around them changes."""
    log(f"grad views {off} {dt}")
    base = torch.randn(70000).to(DT[dt]).cuda()
    gs = [base[off: off + 20001], base[30000 + off: 30000 + off + 7], base[40000 - off: 40000 + 9000]]
    _, ref = E.grad_clip_ref([f64(g) for g in gs], 0.5, 1e-6)
    whole = torch.full((40000,), 77.0, dtype=DT[dt], device="cuda")
    outs = [whole[3: 3 + 20001], whole[20004: 20011], whole[20011: 20011 + gs[2].numel()]]
    norm, _ = nm.nm_grad_clip(gs, 0.5, out=outs)
    torch.cuda.synchronize()
    rel, tiny = ROUND[DT[dt]]
    for o, r in zip(outs, ref):
        assert (np.abs(f64(o) - r) <= np.abs(r) * (rel + 2.0 ** -22) * 1.001 + tiny + 2.0 ** -149).all()
    assert (f64(whole[:3]) == 77).all() and (f64(whole[20011 + gs[2].numel():]) == 77).all()


@pytest.mark.parametrize("scale", [1e-38, 1e-25, 1e20, 1e37])
def test_far_magnitudes(scale):
    """Squares that fp32 does not hold."""
    log(f"grad scale {scale}")
    check(grads([((3000,), "f32"), ((50, 7), "bf16")], scale=scale), scale)


def test_norm_past_fp32():
    log("grad norm past fp32")
    g = torch.full((1 << 20,), 3e38, device="cuda")
    norm, out = nm.nm_grad_clip([g], 1.0, out=[torch.empty_like(g)])
    torch.cuda.synchronize()
    assert float(norm) == float("inf") and abs(float(out[0][5]) - 2.0 ** -10) < 1e-9   # the factor is taken in 64 bits


def test_nonfinite():
    log("grad nonfinite")
    gs = grads(MIXED)
    gs[4][77] = float("inf")
    norm, out = nm.nm_grad_clip(gs, 1.0, out=[torch.empty_like(g) for g in gs])
    torch.cuda.synchronize()
    assert float(norm) == float("inf") and torch.isnan(out[4][77]) and int(sum(torch.isnan(o).sum() for o in out)) == 1
    assert not out[0].any() and not out[5].any()
    gs[0][3, 3] = float("nan")
    norm, out = nm.nm_grad_clip(gs, 1.0)
    torch.cuda.synchronize()
    assert torch.isnan(norm) and all(torch.isnan(o).all() for o in out)


@pytest.mark.parametrize("in_place", [False, True])
def test_no_limit_scales_nothing(in_place):
    """max_norm Inf is no limit, of an infinite norm too; a NaN still reaches everything."""
    log(f"grad no limit {in_place}")
    gs = grads(MIXED)
    gs[4][77] = -float("inf")
    before = [g.clone() for g in gs]
    norm, out = nm.nm_grad_clip(gs, float("inf"), out=None if in_place else [torch.empty_like(g) for g in gs])
    torch.cuda.synchronize()
    assert float(norm) == float("inf") and all(torch.equal(o, b) for o, b in zip(out, before))
    gs[0][3, 3] = float("nan")
    norm, out = nm.nm_grad_clip(gs, float("inf"))
    torch.cuda.synchronize()
    assert torch.isnan(norm) and all(torch.isnan(o).all() for o in out)


def test_nothing_to_clip_leaves_the_bits():
    log("grad untouched")
    gs = grads(MIXED)
    gs[0].view(torch.int32)[0, :2] = torch.tensor([1, -2 ** 31], dtype=torch.int32).cuda()      # subnormal, -0
    before = [g.clone() for g in gs]
    nm.nm_grad_clip(gs, 1e9)
    _, out = nm.nm_grad_clip(gs, 1e9, out=[torch.empty_like(g) for g in gs])
    torch.cuda.synchronize()
    for b, g, o in zip(before, gs, out):
        same = b.view(torch.int32 if b.dtype == torch.float32 else torch.int16)
        assert torch.equal(same, g.view(same.dtype)) and torch.equal(same, o.view(same.dtype))


def test_one_tensor_twice():
    log("grad one tensor twice")
    g = grads([((500,), "f32")])[0]
    norm = nm.nm_grad_norm([g, g])                    # read only: counted twice
    torch.cuda.synchronize()
    assert abs(float(norm) - 2 ** 0.5 * np.linalg.norm(f64(g))) < 1e-5
    with pytest.raises(nm.NMError):
        nm.nm_grad_clip([g, g], 1.0)
    with pytest.raises(nm.NMError):
        nm.nm_grad_clip([g[:300], g[200:]], 1.0)
    nm.nm_grad_clip([g, g], 1.0, out=[torch.empty_like(g), torch.empty_like(g)])
    torch.cuda.synchronize()


def test_list_is_kept_and_notices_new_memory():
    log("grad list")
    gs = grads(MIXED)
    outs = [torch.empty_like(g) for g in gs]
    held = nm.nm_grad_list(gs, outs)
    for step in range(3):
        for g in gs:
            g.mul_(0.5)
        norm, out = nm.nm_grad_clip(held, 0.25)
        want, ref = nm.nm_grad_clip(gs, 0.25, out=[torch.empty_like(g) for g in gs])
        torch.cuda.synchronize()
        assert torch.equal(norm, want) and all(torch.equal(a, b) for a, b in zip(out, ref)) and out[0] is outs[0]
        assert torch.equal(nm.nm_grad_norm(held), want)
        gs[step].data = gs[step].clone() * 3        # other memory under the same tensor
    with pytest.raises(ValueError):
        nm.nm_grad_clip(held, 1.0, out=outs)
    # a parameter that requires its gradient, as an optimizer holds it
    w = torch.nn.Parameter(torch.randn(40, 3, device="cuda"))
    (w * w).sum().backward()
    norm, _ = nm.nm_grad_clip([w.grad], 1.0)
    torch.cuda.synchronize()
    assert abs(float(torch.linalg.vector_norm(w.grad)) - 1.0) < 1e-5 and float(norm) > 1.0


def test_refusals():
    g = torch.randn(8, 8, device="cuda")
    with pytest.raises(ValueError, match="contiguous"):
        nm.nm_grad_norm([g.t()[:, :3]])
    with pytest.raises(ValueError):
        nm.nm_grad_clip([g], 1.0, out=[torch.empty(8, 7, device="cuda")])
    with pytest.raises(ValueError):
        nm.nm_grad_clip([g], 1.0, out=[g.half()])
    for bad in (-1.0, float("nan")):
        with pytest.raises(nm.NMError):
            nm.nm_grad_clip([g], bad)


def test_equal_calls_streams_and_graphs():
    log("grad equal calls, side stream, graph")
    gs = grads(MIXED + [((1 << 20,), "bf16"), ((300, 999), "f32")])
    outs = [torch.empty_like(g) for g in gs]
    held = nm.nm_grad_list(gs, outs)
    first, _ = nm.nm_grad_clip(held, 1.0)
    kept = [o.clone() for o in outs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second, _ = nm.nm_grad_clip(held, 1.0)
    torch.cuda.synchronize()
    assert torch.equal(first, second) and all(torch.equal(a, b) for a, b in zip(kept, outs))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm, _ = nm.nm_grad_clip(held, 1.0)
    for i in range(4):
        for j, g in enumerate(gs):
            g.copy_(grads([(tuple(g.shape), {v: k for k, v in DT.items()}[g.dtype])], 100 * i + j)[0])
        graph.replay()
        want, ref = nm.nm_grad_clip(gs, 1.0, out=[torch.empty_like(g) for g in gs])
        torch.cuda.synchronize()
        assert torch.equal(norm, want) and all(torch.equal(a, b) for a, b in zip(outs, ref))
