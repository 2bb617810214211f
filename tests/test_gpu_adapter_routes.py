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
