"""The sizes that cross entropy refuses, as its header states them; no GPU."""
import ctypes
import os

import pytest

import structured_sparse_gemm_nm_amd as nm

pytestmark = pytest.mark.skipif(not os.path.exists(nm.lib_path()), reason="libnmsparse.so not built")

OK, SHAPE = 0, 2


@pytest.mark.parametrize("T,V,st", [(1 << 22, 1 << 15, OK), (1 << 13, 1 << 24, OK), (1 << 14, 1 << 23, OK),
                                    ((1 << 13) + 16, 1 << 24, SHAPE), (1 << 22, (1 << 15) + 128, SHAPE),
                                    (65536, 1 << 24, SHAPE), (1 << 22, 1 << 24, SHAPE)])
def test_tokens_times_words(T, V, st):
    # ceil(T / 16) ceil(V / 128) <= 2^26
    assert ((T + 15) // 16 * ((V + 127) // 128) <= 1 << 26) == (st == OK)
    b = ctypes.c_size_t()
    assert nm.lib().nm_xent_workspace_size(T, V, 64, nm.NM_BF16, ctypes.byref(b)) == st
    assert nm.lib().nm_xent_bwd_workspace_size(T, V, 64, nm.NM_BF16, 1, 1, ctypes.byref(b)) == st
