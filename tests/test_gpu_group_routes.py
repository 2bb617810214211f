"""The kernels of the products grouped by expert that only larger or longer calls reach, against
the float64 oracle with the bounds of test_gpu_group; each case says which kernel it is meant for,
and that is held against the rule, written down here a second time.  Non-finite values in every
pattern, with every kernel."""
import numpy as np
import pytest

import structured_sparse_gemm_nm_amd as nm
from gpu_util import log
from test_gpu_group import PAT, Case

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def route(T, E, R, K, n, m):
    """Which kernel a forward product takes (the rows an expert has on average decide)."""
    least = min(T, E)
    mean = T // least
    if mean <= 8:
        piece, units = {(2, 4): (16, 4), (1, 4): (32, 2), (1, 8): (64, 2)}[n, m]
        cols = 8 * piece
        shares = 1
        while shares * units * cols < K:
            shares *= 2
        step = 16 * (8 // min(shares, 8))
        if K % piece == 0 and K <= 4096 and least * -(-R // step) >= 1024:
            return "stream"
        return "few1_wide" if least * R >= 12288 else "few1"
    if mean <= 24:
        return "few2"
    if mean <= 64:
        return "tile64"
    if n == 2 and K % 128 == 0 and R >= 256 and -(-R // 256) * -(-T // 128) >= 96:
        return "lds"
    return "tile128" if -(-R // 128) * -(-T // 128) >= 256 else "tile64"


def case(want, lengths, R, K, pat, dt, **kw):
    c = Case(lengths, R, K, pat, dt, **kw)
    assert route(c.T, len(lengths), R, K, *pat) == want
    return c


@pytest.mark.parametrize("K", [144, 1040])
@pytest.mark.parametrize("pat", PAT)
@pytest.mark.parametrize("dt,out", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32")])
def test_tiles_of_128_tokens(K, pat, dt, out):
    log(f"group tile128 K={K} {pat} {dt} {out}")
    case("tile128", [5000, 0, 3001, 400], 1100, K, pat, dt, before=2, behind=3, pad=8).forward(out, 3 if out == "f32" else 4)


@pytest.mark.parametrize("pat", PAT)
def test_tiles_of_128_tokens_from_a_table(pat):
    """More experts than a workgroup looks through itself."""
    log(f"group tile128 of 300 experts {pat}")
    lengths = np.bincount(np.random.default_rng(5).integers(0, 300, 30000), minlength=300)
    lengths[3], lengths[200] = 0, lengths[200] + 700
    case("tile128", lengths.tolist(), 200, 80, pat, "bf16", pack_on_gpu=True).forward("bf16")


# K past what a streaming wave keeps, not in whole pieces, or too few steps to stream
@pytest.mark.parametrize("pat,K", [((2, 4), 4112), ((2, 4), 512), ((1, 4), 2064), ((1, 4), 4128), ((1, 4), 544),
                                   ((1, 8), 1056), ((1, 8), 4160), ((1, 8), 576)])
@pytest.mark.parametrize("dt,out", [("bf16", "bf16"), ("f16", "f32")])
def test_waves_of_64_rows(pat, K, dt, out):
    log(f"group few1_wide {pat} K={K} {dt} {out}")
    c = case("few1_wide", [3, 0, 17, 1, 5, 8, 2, 4, 16], 1571, K, pat, dt, before=1, behind=2, pad=8, pack_on_gpu=True)
    c.forward(out, 1)


@pytest.mark.parametrize("E_,R,K,pat", [(40, 900, 3136, (1, 8)), (40, 830, 4096, (1, 8)), (40, 890, 3104, (1, 4)),
                                        (70, 500, 4080, (2, 4))])
def test_streams_of_long_rows(E_, R, K, pat):
    """K in four and eight shares."""
    log(f"group stream E={E_} R={R} K={K} {pat}")
    lengths = np.random.default_rng(E_ + K).integers(1, 6, E_)
    lengths[0], lengths[E_ // 2], lengths[-1] = 17, 0, 16
    c = case("stream", lengths.tolist(), R, K, pat, "bf16", before=1, behind=4, pad=8, pack_on_gpu=True)
    c.forward("f32", 3)
    c.forward("bf16", 8)


ROUTES = {"few1": ([3, 0, 17, 1, 5], 136, 160), "few1_wide": ([3, 0, 17, 1, 5, 8], 3000, 4160),
          "few2": ([33, 20, 0, 20], 136, 160), "tile64": ([129, 300, 0, 257], 136, 160),
          "tile128": ([3000, 0, 3001, 400], 1100, 160), "stream": ([2] * 40 + [0, 17] + [3] * 60, 1571, 192)}


@pytest.mark.parametrize("pat", PAT)
@pytest.mark.parametrize("which", list(ROUTES))
def test_nonfinite_stays_with_its_expert(which, pat):
    """Inf in a row of act, NaN in a row of G and in one expert's weight: the outputs of these rows and
    of this expert, and nothing else."""
    log(f"group nonfinite {which} {pat}")
    lengths, R, K = ROUTES[which]
    c = case(which, lengths, R, K, pat, "bf16", pack_on_gpu=True)
    args = (c.d_off, c.K, *pat)

    def all_three():
        dx = dw = None
        y = nm.nm_group_spmm(c.d_values, c.d_idx, c.d_act, *args)
        if R % 8 == 0:
            dx = nm.nm_group_spmm_dx(c.d_values, c.d_idx, c.d_g, *args)
            dw = nm.nm_group_spmm_dw(c.d_idx, c.d_g, c.d_act, *args)
        return y, dx, dw
    y, dx, dw = all_three()
    t = int(c.offsets[0])                                   # the first expert's first row
    e1 = next(e for e in range(1, len(lengths)) if lengths[e])   # another expert with rows
    c.d_act[t, 7], c.d_g[t, 9] = float("inf"), float("nan")
    c.d_values[e1, 3, 5] = float("nan")
    y2, dx2, dw2 = all_three()
    torch.cuda.synchronize()
    lo, hi = int(c.offsets[e1]), int(c.offsets[e1 + 1])
    keep = torch.ones(c.T, dtype=torch.bool, device="cuda")
    keep[t], keep[lo:hi] = False, False
    assert torch.equal(y[keep], y2[keep]) and torch.isfinite(y).all()
    # column 7 of act meets a stored value of 1 in M / N rows; the others keep their bits
    hit = ~torch.isfinite(y2[t])
    assert hit.any() and not hit.all() and torch.equal(y2[t][~hit], y[t][~hit])
    assert torch.isnan(y2[lo:hi, 3]).all() and torch.equal(y2[lo:hi, :3], y[lo:hi, :3])
    assert torch.equal(y2[lo:hi, 4:], y[lo:hi, 4:])
    if dx is not None:
        assert torch.equal(dx[keep], dx2[keep]) and torch.isnan(dx2[t]).all()
        # one column of W meets the NaN
        assert (torch.isnan(dx2[lo:hi]).sum(1) == 1).all()
        assert torch.equal(dw[1:], dw2[1:]) and torch.isnan(dw2[0, 9]).all()
