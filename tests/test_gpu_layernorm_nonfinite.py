"""Where an Inf or NaN in layer norm's inputs may go, as the header states it."""
import pytest

import structured_sparse_gemm_nm_amd as nm
from gpu_util import log

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
@pytest.mark.parametrize("H", [200, 1543, 20000])
def test_non_finite_reaches_its_row_and_columns_only(H, bad):
    log(f"layernorm non-finite H={H} {bad}")
    T, gen = 9, torch.Generator(device="cuda").manual_seed(H)
    x, dy = (torch.randn((T, H), generator=gen, device="cuda") for _ in range(2))
    w = 1 + 0.1 * torch.randn(H, generator=gen, device="cuda")
    rest = [t for t in range(T) if t != 4]
    y, mean, rstd = nm.nm_layernorm(x, w, stats=True)
    dx, dw, db = nm.nm_layernorm_bwd(dy, x, mean, rstd, w)
    x2 = x.clone()
    x2[4, 7] = bad
    y2, mean2, rstd2 = nm.nm_layernorm(x2, w, stats=True)
    gx, gw, gb = nm.nm_layernorm_bwd(dy, x2, mean2, rstd2, w)
    torch.cuda.synchronize()
    assert y2[4].isnan().all() and gx[4].isnan().all() and gw.isnan().all()
    assert torch.equal(y2[rest], y[rest]) and torch.equal(gx[rest], dx[rest]) and torch.equal(gb, db)
    dy2 = dy.clone()
    dy2[4, 7] = bad
    gx, gw, gb = nm.nm_layernorm_bwd(dy2, x, mean, rstd, w)
    torch.cuda.synchronize()
    others = torch.arange(H, device="cuda") != 7
    assert not gx[4].isfinite().any() and torch.equal(gx[rest], dx[rest])
    assert not gw[7].isfinite() and not gb[7].isfinite()
    assert torch.equal(gw[others], dw[others]) and torch.equal(gb[others], db[others])
