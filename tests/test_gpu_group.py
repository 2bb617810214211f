"""Products grouped by expert on MI355X (nm_group_spmm, _dx, _dw) against the float64 oracle.

Bounds: products of two 16-bit floats are exact in fp32; n of them summed in any
order with unit 2^-23 (allowing round-toward-zero) are off by at most n 2^-23 of the
sum of their magnitudes, plus half a step of the output's type.
"""
import numpy as np
import pytest

import nm_inputs
import structured_sparse_gemm_nm_amd as nm
from oracle import nm_experts as E
from oracle import nm_oracle as O
from gpu_util import bits_of, log, to_dev, torch_dtype

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

PAT = [(2, 4), (1, 4), (1, 8)]
ROUND = {"bf16": (2.0 ** -8, 1e-38), "f16": (2.0 ** -11, 2.0 ** -24), "f32": (2.0 ** -24, 1e-38)}


def within(got, ref, size, terms, out):
    assert got.shape == ref.shape and np.isfinite(got).all()
    rel, tiny = ROUND[out]
    bound = terms * 2.0 ** -23 * size + np.abs(ref) * rel + tiny + 1e-30
    worst = (np.abs(got - ref) / bound).max() if ref.size else 0.0
    assert worst <= 1.0, f"{worst:.2f} times the bound"


class Case:
    def __init__(self, lengths, R, K, pat, dt, before=0, behind=0, pad=0, seed=0, pack_on_gpu=False):
        self.n, self.m = pat
        self.R, self.K, self.dt = R, K, dt
        self.T = before + sum(lengths) + behind
        self.offsets = np.cumsum([before, *lengths]).astype(np.int32)
        seed = seed * 7919 + R * 31 + K + self.T
        w = nm_inputs.normal_half((len(lengths) * R, K), 0.05, dt, 90, 0, seed)
        if pack_on_gpu:      # large weights: the pack kernels have tests of their own
            v, i = nm.nm_compress(to_dev(w, dt), self.n, self.m)
            v, i = bits_of(v), i.cpu().numpy().view(np.uint32)
        else:
            v, i = O.prune_pack(w, self.n, self.m)
        self.values, self.idx = v.reshape(len(lengths), R, -1), i.reshape(len(lengths), R, -1)
        self.act = nm_inputs.normal_half((self.T, K), 1.0, dt, 90, 1, seed)
        self.g = nm_inputs.normal_half((self.T, R), 0.5, dt, 90, 2, seed)
        self.d_values, self.d_off = to_dev(self.values, dt), torch.from_numpy(self.offsets).cuda()
        self.d_idx = torch.from_numpy(self.idx.view(np.int32)).cuda()
        self.d_act, self.d_g = self.padded(self.act, pad), self.padded(self.g, pad)

    def padded(self, bits, pad):
        """On the device, rows `pad` elements further apart; what lies between is NaN."""
        t = torch.full((bits.shape[0], bits.shape[1] + pad), float("nan"), dtype=torch_dtype(self.dt), device="cuda")
        t[:, : bits.shape[1]] = to_dev(bits, self.dt)
        return t[:, : bits.shape[1]]

    def outputs(self, cols, out, ldpad):
        """A sentinel-filled output with room between and behind its rows."""
        t = {"f32": torch.float32}.get(out) or torch_dtype(out)
        whole = torch.full((self.T + 3, cols + ldpad), 77.0, dtype=t, device="cuda")
        return whole, whole[: self.T, :cols]

    def untouched(self, whole, owned, cols):
        w = whole.float().cpu().numpy()
        assert (w[self.T:] == 77.0).all() and (w[:, cols:] == 77.0).all() and (w[: self.T][~owned] == 77.0).all()

    def forward(self, out="f32", ldpad=0):
        whole, y = self.outputs(self.R, out, ldpad)
        nm.nm_group_spmm(self.d_values, self.d_idx, self.d_act, self.d_off, self.K, self.n, self.m, out_dtype=y.dtype, out=y)
        torch.cuda.synchronize()
        ref, size, owned = E.group_ref(self.values, self.idx, self.K, self.n, self.m, self.act, self.offsets, self.dt)
        within(y.double().cpu().numpy()[owned], ref[owned], size[owned], self.K * self.n // self.m, out)
        self.untouched(whole, owned, self.R)

    def backward(self, out="f32", ldpad=0):
        whole, dx = self.outputs(self.K, out, ldpad)
        nm.nm_group_spmm_dx(self.d_values, self.d_idx, self.d_g, self.d_off, self.K, self.n, self.m, out_dtype=dx.dtype, out=dx)
        dw = nm.nm_group_spmm_dw(self.d_idx, self.d_g, self.d_act, self.d_off, self.K, self.n, self.m, out_dtype=dx.dtype)
        torch.cuda.synchronize()
        ref, size, owned = E.group_dx_ref(self.values, self.idx, self.K, self.n, self.m, self.g, self.offsets, self.dt)
        within(dx.double().cpu().numpy()[owned], ref[owned], size[owned], self.R, out)
        self.untouched(whole, owned, self.K)
        ref, size = E.group_dw_ref(self.idx, self.K, self.n, self.m, self.g, self.act, self.offsets, self.dt)
        within(dw.double().cpu().numpy(), ref, size, self.T, out)


# lengths that take the few-row kernels, the tiles of 64 and of 128 tokens
LENGTHS = {"token": [0, 1, 0, 1], "few": [3, 0, 17, 1, 5], "mid": [33, 2, 0, 20], "tile64": [64, 1, 90, 40],
           "tile128": [129, 300, 0, 257], "one": [5], "one_large": [400]}


@pytest.mark.parametrize("lengths", list(LENGTHS))
@pytest.mark.parametrize("pat", PAT)
@pytest.mark.parametrize("dt,out", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32")])
def test_forward(lengths, pat, dt, out):
    log(f"group forward {lengths} {pat} {dt} {out}")
    Case(LENGTHS[lengths], 200, 192, pat, dt).forward(out)


# few tiles and a long reduction: summed in shares, the last one shorter, joined in order
@pytest.mark.parametrize("pat", PAT)
@pytest.mark.parametrize("dt,out", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32")])
@pytest.mark.parametrize("lengths,R,K", [([33, 2, 0, 90], 131, 2208), ([260, 0, 150], 72, 2080), ([70], 6, 8224)])
def test_forward_in_shares(lengths, R, K, pat, dt, out):
    log(f"group shares forward {lengths} {R} {K} {pat} {dt} {out}")
    c = Case(lengths, R, K, pat, dt)
    assert nm._group_need(len(lengths), R, K, *pat, nm.NM_BF16, c.T, nm.NM_F32) > 2 * 4 * c.T * R
    c.forward(out)
    c.forward(out, ldpad=3)


@pytest.mark.parametrize("pat", PAT)
@pytest.mark.parametrize("dt,out", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32")])
@pytest.mark.parametrize("lengths,R,K", [([1, 0, 1], 2056, 96), ([33, 150, 0], 2216, 160), ([1100, 0, 2200], 72, 96),
                                         ([2049], 136, 288)])
def test_backward_in_shares(lengths, R, K, pat, dt, out):
    log(f"group shares backward {lengths} {R} {K} {pat} {dt} {out}")
    c = Case(lengths, R, K, pat, dt)
    assert nm._group_dx_need(len(lengths), R, K, c.T) + nm._group_dw_need(len(lengths), R, K, *pat, c.T) > 0
    c.backward(out)
    c.backward(out, ldpad=8)


# at most 64 tiles of 16 to 31 steps: in three or four shares; one step or one tile past that, in one
@pytest.mark.parametrize("pat", PAT)
@pytest.mark.parametrize("out", ["f16", "f32"])
@pytest.mark.parametrize("lengths,R,K,shared", [([70, 0, 61], 133, 1040, True), ([200], 512, 1936, True),
                                                ([130], 4104, 1040, False), ([200], 72, 960, False)])
def test_forward_in_few_shares(lengths, R, K, shared, pat, out):
    log(f"group few shares forward {lengths} {R} {K} {pat} {out}")
    c = Case(lengths, R, K, pat, "f16")
    need = nm._group_need(len(lengths), R, K, *pat, nm.NM_F16, c.T, nm.NM_F32)
    assert need > 2 * 4 * c.T * R if shared else need == 0
    c.forward(out)


@pytest.mark.parametrize("pat", PAT)
@pytest.mark.parametrize("out", ["f16", "f32"])
@pytest.mark.parametrize("lengths,R,K,dx,dw", [([1, 0, 3], 1032, 96, True, False), ([33, 90], 1992, 1056, True, False),
                                               ([520], 72, 96, False, True), ([300, 724], 1032, 288, True, True),
                                               ([40], 1016, 2080, True, False), ([40], 952, 96, False, False)])
def test_backward_in_few_shares(lengths, R, K, dx, dw, pat, out):
    log(f"group few shares backward {lengths} {R} {K} {pat} {out}")
    c = Case(lengths, R, K, pat, "f16")
    assert (nm._group_dx_need(len(lengths), R, K, c.T) > 0) == dx
    assert (nm._group_dw_need(len(lengths), R, K, *pat, c.T) > 0) == dw
    c.backward(out)


# rows and columns at and past the tiles' edges; K of 16 and odd multiples of it
@pytest.mark.parametrize("R,K", [(1, 16), (15, 48), (17, 64), (127, 80), (128, 128), (129, 144), (257, 1040), (96, 2064), (640, 512)])
@pytest.mark.parametrize("pat", PAT)
@pytest.mark.parametrize("lengths", ["few", "tile128"])
def test_forward_sizes(R, K, pat, lengths):
    log(f"group forward R={R} K={K} {pat} {lengths}")
    Case(LENGTHS[lengths], R, K, pat, "bf16").forward("f32")
    Case(LENGTHS[lengths], R, K, pat, "f16").forward("f16")


@pytest.mark.parametrize("lengths", list(LENGTHS))
@pytest.mark.parametrize("pat", PAT)
@pytest.mark.parametrize("dt,out", [("bf16", "bf16"), ("f16", "f32")])
def test_backward(lengths, pat, dt, out):
    log(f"group backward {lengths} {pat} {dt} {out}")
    Case(LENGTHS[lengths], 136, 160, pat, dt).backward(out)


@pytest.mark.parametrize("R,K", [(8, 32), (120, 96), (264, 544)])
@pytest.mark.parametrize("pat", PAT)
def test_backward_sizes(R, K, pat):
    log(f"group backward R={R} K={K} {pat}")
    Case([70, 0, 131, 3], R, K, pat, "bf16").backward("f32")


@pytest.mark.parametrize("lengths", ["few", "tile64", "tile128"])
def test_rows_of_no_expert_and_strides(lengths):
    """Rows in front of the first and behind the last expert hold NaN and stay as they were;
    rows lie further apart than their width."""
    log(f"group strides {lengths}")
    c = Case(LENGTHS[lengths], 200, 160, (2, 4), "bf16", before=5, behind=9, pad=24)
    lo, hi = c.offsets[0], c.offsets[-1]
    for t in (c.d_act, c.d_g):
        t[:lo] = float("nan")
        t[hi:] = float("nan")
    for ldpad in (0, 1, 8):
        c.forward("bf16", ldpad)
        c.backward("f32", ldpad)


def test_many_experts():
    """More experts than a wave, and than a workgroup, looks at in one go."""
    rng = np.random.default_rng(4)
    for E_, T, R, K in [(70, 90, 24, 32), (1100, 2500, 16, 32), (1100, 60000, 8, 32)]:
        log(f"group experts={E_} T={T}")
        lengths = np.bincount(rng.integers(0, E_, T), minlength=E_)
        lengths[3] = 0
        Case(lengths.tolist(), R, K, (2, 4), "f16").forward("f32")
        if T < 10000:
            Case(lengths.tolist(), R, K, (1, 4), "bf16").backward("bf16")


def test_no_rows_at_all():
    c = Case([0, 0, 0], 64, 64, (2, 4), "bf16", before=0, behind=6)
    log("group no rows")
    c.forward()
    c.backward()
    empty = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    assert nm.nm_group_spmm(c.d_values, c.d_idx, empty, c.d_off, 64).shape == (0, 64)
    assert nm.nm_group_spmm_dx(c.d_values, c.d_idx, empty, c.d_off, 64).shape == (0, 64)
    dw = nm.nm_group_spmm_dw(c.d_idx, empty, empty, c.d_off, 64)
    torch.cuda.synchronize()
    assert dw.shape == (3, 64, 32) and not dw.any()


@pytest.mark.parametrize("offsets", [[-5, 700, 3, 90], [400, 100, 300, 0], [0, 5, 2 ** 31 - 1, -2 ** 31], [0, 300, 0, 300]])
@pytest.mark.parametrize("T", [12, 300])
def test_broken_offsets_stay_inside(offsets, T):
    """Offsets that leave [0, T] or descend: clamped (the rule is run over every small list by
    test_host_offsets); nothing around the outputs changes."""
    log(f"group broken offsets {offsets} T={T}")
    c = Case([T, 0, 0], 136, 160, (2, 4), "bf16")
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    for cols, call in [(136, lambda y: nm.nm_group_spmm(c.d_values, c.d_idx, c.d_act, off, 160, out=y)),
                       (160, lambda y: nm.nm_group_spmm_dx(c.d_values, c.d_idx, c.d_g, off, 160, out=y))]:
        whole = torch.full((T + 600, cols + 8), 77.0, device="cuda")
        call(whole[300: 300 + T, :cols])
        torch.cuda.synchronize()
        w = whole.cpu().numpy()
        assert (w[:300] == 77.0).all() and (w[300 + T:] == 77.0).all() and (w[:, cols:] == 77.0).all()
    assert nm.nm_group_spmm_dw(c.d_idx, c.d_g, c.d_act, off, 160).shape == (3, 136, 80)
    torch.cuda.synchronize()


@pytest.mark.parametrize("lengths", ["few", "tile128"])
def test_nonfinite_stays_with_its_expert(lengths):
    log(f"group nonfinite {lengths}")
    c = Case(LENGTHS[lengths], 136, 160, (2, 4), "bf16")
    clean = [t.clone() for t in (c.d_values, c.d_act, c.d_g)]
    args = (c.d_off, c.K, 2, 4)
    y, dx = (f(c.d_values, c.d_idx, x, *args) for f, x in ((nm.nm_group_spmm, c.d_act), (nm.nm_group_spmm_dx, c.d_g)))
    dw = nm.nm_group_spmm_dw(c.d_idx, c.d_g, c.d_act, *args)
    t = int(c.offsets[0])                  # the first expert's first row
    e1 = 1 if LENGTHS[lengths][1] else 2   # another expert with rows, whose weight is made NaN
    c.d_act[t, 7], c.d_g[t, 9] = float("inf"), float("nan")
    c.d_values[e1, 3, 5] = float("nan")
    y2, dx2 = (f(c.d_values, c.d_idx, x, *args) for f, x in ((nm.nm_group_spmm, c.d_act), (nm.nm_group_spmm_dx, c.d_g)))
    dw2 = nm.nm_group_spmm_dw(c.d_idx, c.d_g, c.d_act, *args)
    torch.cuda.synchronize()
    lo, hi = c.offsets[e1], c.offsets[e1 + 1]
    keep = torch.ones(c.T, dtype=torch.bool)
    keep[t], keep[lo:hi] = False, False
    assert torch.equal(y[keep.cuda()], y2[keep.cuda()]) and torch.equal(dx[keep.cuda()], dx2[keep.cuda()])
    assert not torch.isfinite(y2[t]).all() and torch.isnan(dx2[t]).all()
    assert torch.isnan(y2[lo:hi, 3]).all() and torch.equal(y2[lo:hi, :3], y[lo:hi, :3])
    assert torch.equal(dw[1:], dw2[1:]) and torch.isnan(dw2[0, 9]).all()
    assert len(clean) == 3


def test_equal_calls_and_streams():
    log("group equal calls on another stream")
    c = Case(LENGTHS["tile128"], 264, 544, (1, 4), "f16")
    args = (c.d_off, c.K, 1, 4)

    def all_three():
        return (nm.nm_group_spmm(c.d_values, c.d_idx, c.d_act, *args), nm.nm_group_spmm_dx(c.d_values, c.d_idx, c.d_g, *args),
                nm.nm_group_spmm_dw(c.d_idx, c.d_g, c.d_act, *args))
    first = all_three()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        second = all_three()
    third = all_three()                    # two streams at once, each with its own workspace
    torch.cuda.synchronize()
    for a, b, d in zip(first, second, third):
        assert torch.equal(a, b) and torch.equal(a, d)


@pytest.mark.parametrize("lengths", ["few", "tile128"])
def test_captured_and_replayed_with_other_offsets(lengths):
    """A captured graph follows the offsets that the device holds at each replay."""
    log(f"group graph {lengths}")
    c = Case(LENGTHS[lengths], 136, 160, (2, 4), "bf16")
    args = (c.d_off, c.K, 2, 4)

    def all_three():
        return (nm.nm_group_spmm(c.d_values, c.d_idx, c.d_act, *args), nm.nm_group_spmm_dx(c.d_values, c.d_idx, c.d_g, *args),
                nm.nm_group_spmm_dw(c.d_idx, c.d_g, c.d_act, *args))
    all_three()
    torch.cuda.synchronize()
    graph, other = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = all_three()
    with torch.cuda.graph(other):
        held_other = all_three()
    E_ = len(LENGTHS[lengths])
    for shift in range(4):
        ends = np.sort(np.random.default_rng(shift).integers(0, c.T + 1, E_ - 1))
        c.d_off.copy_(torch.tensor([0, *ends.tolist(), c.T], dtype=torch.int32))
        graph.replay()
        other.replay()
        want = all_three()
        torch.cuda.synchronize()
        for a, b, d in zip(held, held_other, want):
            assert torch.equal(a, d) and torch.equal(b, d)


@pytest.mark.parametrize("T,R,K", [(700, 4104, 256), (130, 72, 2208), (96, 2216, 96), (3300, 72, 96)])
def test_large_and_shared_products_follow_their_offsets(T, R, K):
    """The large tiles' table and the parts of a shared reduction (forward, dX, dW): captured twice and replayed
    with other offsets, broken ones among them; nothing around the outputs changes."""
    log(f"group graph T={T} R={R} K={K}")
    c = Case([T // 2, 0, T - T // 2], R, K, (2, 4), "bf16", before=1, behind=3)
    dt = torch.bfloat16
    outs = [[torch.full((c.T + 20, w + 8), 77.0, dtype=dt, device="cuda") for w in (R, K)] for _ in range(3)]

    def all_three(o):
        nm.nm_group_spmm(c.d_values, c.d_idx, c.d_act, c.d_off, K, out_dtype=dt, out=o[0][10: 10 + c.T, :R])
        nm.nm_group_spmm_dx(c.d_values, c.d_idx, c.d_g, c.d_off, K, out_dtype=dt, out=o[1][10: 10 + c.T, :K])
        return nm.nm_group_spmm_dw(c.d_idx, c.d_g, c.d_act, c.d_off, K, out_dtype=dt)
    all_three(outs[2])
    torch.cuda.synchronize()
    graphs, held = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for graph, o in zip(graphs, outs):
        with torch.cuda.graph(graph):
            held.append(all_three(o))
    for offsets in ([1, 1, 40, T], [0, T, T, T + 4], [5, 9, T, T], [9, 9, 9, 9], [T, 3, 700, -1], [-5, T + 99, 0, 50]):
        for o in outs:
            for y in o:
                y.fill_(77.0)
        c.d_off.copy_(torch.tensor(offsets, dtype=torch.int32))
        for graph in graphs:
            graph.replay()
        want = all_three(outs[2])
        torch.cuda.synchronize()
        whole = offsets == sorted(offsets)
        for k, cols in enumerate((R, K)):
            for o in outs:
                w = o[k].float()
                assert (w[:10] == 77).all() and (w[10 + c.T:] == 77).all() and (w[:, cols:] == 77).all()
                if whole:
                    assert (w[10: 10 + offsets[0]] == 77).all() and (w[10 + offsets[-1]:] == 77).all()
                    assert torch.equal(o[k], outs[2][k])
        if whole:
            assert torch.equal(held[0], want) and torch.equal(held[1], want)


def test_one_expert_is_the_plain_product():
    """All rows of one expert: the same values as nm_spmm, nm_spmm_dx, nm_spmm_dw to rounding."""
    log("group one expert")
    c = Case([333], 264, 512, (2, 4), "bf16")
    y = nm.nm_group_spmm(c.d_values, c.d_idx, c.d_act, c.d_off, 512)
    dx = nm.nm_group_spmm_dx(c.d_values, c.d_idx, c.d_g, c.d_off, 512)
    dw = nm.nm_group_spmm_dw(c.d_idx, c.d_g, c.d_act, c.d_off, 512)
    v, i = c.d_values[0], c.d_idx[0]
    py, pdx, pdw = nm.nm_spmm(v, i, c.d_act, 512), nm.nm_spmm_dx(v, i, c.d_g, 512), nm.nm_spmm_dw(i, c.d_g, c.d_act, 512)
    torch.cuda.synchronize()
    assert torch.equal(dx, pdx) and torch.equal(dw[0], pdw)
    _, size, _ = E.group_ref(c.values, c.idx, 512, 2, 4, c.act, c.offsets, "bf16")
    assert (np.abs((y - py).double().cpu().numpy()) <= 2 * 256 * 2.0 ** -23 * size).all()


@pytest.mark.parametrize("pat", PAT)
def test_wide_gradient_tiles(pat):
    """Rows enough for the wide tiles of dX, with edges in rows, columns and the reduction."""
    log(f"group wide dX {pat}")
    Case([7001, 0, 9003, 1, 6100], 72, 544, pat, "bf16", behind=3).backward("bf16")


@pytest.mark.parametrize("R,K", [(520, 256), (300, 640), (1000, 1152)])
@pytest.mark.parametrize("dt,out", [("bf16", "bf16"), ("f16", "f32")])
def test_large_forward_walks_tiles(R, K, dt, out):
    """2:4 rows enough that workgroups walk from tile to tile, across experts; 640 columns, where each
    tile has its own workgroup."""
    log(f"group walked tiles R={R} K={K} {dt} {out}")
    Case([9000, 1, 0, 6500, 130, 2999], R, K, (2, 4), dt, before=2, behind=5).forward(out, 1 if out == "f32" else 8)


# many experts of few rows, enough steps that workgroups stream; K at and past a wave's units, whole
# pieces and columns past K in every place, 1, 2, 4 and 8 shares of K
@pytest.mark.parametrize("E_,R,K,pat", [(40, 4100, 48, (2, 4)), (64, 2100, 512, (2, 4)), (70, 1100, 528, (2, 4)),
                                        (33, 1030, 1552, (2, 4)), (20, 900, 4096, (2, 4)), (64, 2100, 96, (1, 4)),
                                        (64, 1100, 1056, (1, 4)), (40, 500, 3104, (1, 4)), (64, 2100, 64, (1, 8)),
                                        (64, 1100, 1088, (1, 8)), (40, 500, 3136, (1, 8)), (300, 600, 128, (2, 4))])
def test_streamed_experts(E_, R, K, pat):
    log(f"group streamed E={E_} R={R} K={K} {pat}")
    rng = np.random.default_rng(E_ + K)
    lengths = rng.integers(0, 6, E_)
    lengths[0], lengths[E_ // 2], lengths[-1] = 17, 0, 16      # two tiles, none, a full one
    lengths = np.minimum(lengths, 17)
    c = Case(lengths.tolist(), R, K, pat, "bf16" if E_ % 2 else "f16", before=1, behind=4, pad=8, pack_on_gpu=True)
    c.d_act[:1], c.d_act[-4:] = float("nan"), float("nan")
    c.forward("f32", 3)
    c.forward("bf16" if E_ % 2 else "f16", 8)
    # equal calls give equal bits, and broken offsets change nothing around the output
    args = (c.d_values, c.d_idx, c.d_act)
    ys = [torch.zeros((c.T, R), device="cuda") for _ in range(2)]
    for y in ys:
        nm.nm_group_spmm(*args, c.d_off, K, *pat, out=y)
    whole = torch.full((c.T + 40, R + 4), 77.0, device="cuda")
    bad = c.d_off.clone()
    bad[1::2], bad[::2] = c.T + 9, -3
    nm.nm_group_spmm(*args, bad, K, *pat, out=whole[20: 20 + c.T, :R])
    torch.cuda.synchronize()
    assert torch.equal(ys[0], ys[1])
    w = whole.cpu().numpy()
    assert (w[:20] == 77).all() and (w[20 + c.T:] == 77).all() and (w[:, R:] == 77).all()


@pytest.mark.parametrize("lengths", ["token", "few", "tile64"])
@pytest.mark.parametrize("pat,K", [((2, 4), 8208), ((1, 4), 8240), ((1, 8), 12304)])
def test_long_reductions(lengths, pat, K):
    """K past what a streaming wave keeps, in multiples of 16 only."""
    log(f"group long K={K} {pat} {lengths}")
    Case(LENGTHS[lengths], 70, K, pat, "bf16").forward("f32")
