"""The adapters' kernels that only larger or less regular calls reach, against the
float64 oracle with the bounds of test_gpu_adapter.Case."""
import numpy as np
import pytest

import structured_sparse_gemm_nm_amd as nm
from gpu_util import log
from test_gpu_adapter import Case

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("R,T", [(265, 40), (267, 300), (3502, 300)])
def test_rows_that_end_inside_a_piece(R, T):
    # an fp32 Y whose rows lie on 16 bytes while R is no multiple of 4, by the product
    # that writes Y before the term is added to it; nothing outside the rows changes
    log(f"adapter rows R={R} T={T}")
    c = Case(R, 192, T, 9, 3, "bf16")
    ldy = (R + 7) // 4 * 4
    hold = torch.full(((T - 1) * ldy + R + 32,), float("nan"), device="cuda")
    out = hold.as_strided((T, R), (ldy, 1))
    y, _ = c.forward(out=out)
    ref, _ = c.forward()
    assert torch.equal(y, ref)
    gaps = torch.ones_like(hold, dtype=torch.bool)
    gaps.as_strided((T, R), (ldy, 1)).zero_()
    assert hold[gaps].isnan().all()
    c.check_forward(half_out=False)


# few tokens through the kernel that streams rows for the whole chip (2:4, at least 4096
# rows, 2048 < K <= 4096, K % 128 == 0): one to three blocks of 16 rows a workgroup, the
# last ones ragged
@pytest.mark.parametrize("R,K,T,r,na", [(4096, 2176, 1, 16, 2), (4111, 2304, 16, 16, 24), (9003, 2176, 5, 9, 4),
                                        (4100, 4096, 3, 40, 5)])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_few_tokens_streamed(R, K, T, r, na, dt):
    log(f"adapter streamed R={R} K={K} T={T} r={r} n={na} {dt}")
    Case(R, K, T, r, na, dt).check_forward()


# prefill with more 256 x 128 tiles than CUs, so that workgroups walk several tiles with
# the next one's loads in flight across the term; whole and ragged tiles
@pytest.mark.parametrize("R,K,T,r", [(4096, 128, 2100, 16), (4100, 256, 2060, 9), (1024, 128, 9000, 33)])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_prefill_walks_tiles(R, K, T, r, dt):
    log(f"adapter prefill walk R={R} K={K} T={T} r={r} {dt}")
    Case(R, K, T, r, 5, dt).check_forward()


# the expand kernel with 64 columns a wave (at least 256 tiles of 16 x 256), onto what
# nm_spmm's own kernels write
@pytest.mark.parametrize("R,K,T,r,n,m", [(3500, 192, 300, 20, 2, 4), (3501, 192, 300, 7, 2, 4), (1025, 1024, 1100, 12, 1, 4),
                                         (4096, 768, 260, 16, 1, 8)])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_wide_expand(R, K, T, r, n, m, dt):
    log(f"adapter wide expand R={R} K={K} T={T} r={r} {n}:{m} {dt}")
    Case(R, K, T, r, 4, dt, n, m).check_forward()


# gradients with 128 columns a workgroup ((K + R) / 128 x adapters >= 256), ranks in one
# fragment and in two, columns that end inside the last tile
@pytest.mark.parametrize("R,K,T,r,na", [(1024, 1024, 200, 16, 16), (1032, 1056, 77, 9, 17), (1024, 1024, 333, 32, 16),
                                        (520, 544, 150, 20, 40), (1040, 1024, 5000, 24, 16)])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_wide_gradients(R, K, T, r, na, dt):
    log(f"adapter wide gradients R={R} K={K} T={T} r={r} n={na} {dt}")
    Case(R, K, T, r, na, dt).check_backward(half_out=False)


# every pattern through a backward pass of several tiles in both directions
@pytest.mark.parametrize("n,m", nm.PATTERNS)
def test_backward_of_many_tiles(n, m):
    log(f"adapter backward tiles {n}:{m}")
    Case(1096, 672, 700, 24, 4, "bf16", n, m).check_backward()


# the largest ranks: several rounds of 16 (few tokens), 32 (the term) and 64 (gradients)
@pytest.mark.parametrize("T,r", [(9, 256), (40, 256), (300, 129), (130, 200)])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_largest_ranks(T, r, dt):
    log(f"adapter rank {r} T={T} {dt}")
    c = Case(264, 384, T, r, 3, dt)
    c.check_forward()
    c.check_backward()
