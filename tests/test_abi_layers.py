"""C ABI checks, without a GPU, of layer norm, the adapters and cross entropy:
every argument error is caught on the host before any HIP call (fake pointers
are never dereferenced)."""
import ctypes
import os

import pytest

import structured_sparse_gemm_nm_amd as nm

pytestmark = pytest.mark.skipif(not os.path.exists(nm.lib_path()), reason="libnmsparse.so not built")

P = 1 << 32          # fake device addresses, this far apart
OK, NULL, SHAPE, UNSUPPORTED, STRIDE, ALIAS, _, ALIGN = range(8)


def norm(x=P, T=4, H=64, ldx=64, dt=nm.NM_BF16, w=2 * P, b=3 * P, eps=1e-5, y=4 * P, ldy=64, mean=5 * P, rstd=6 * P):
    return nm.lib().nm_layernorm(x, T, H, ldx, dt, w, b, eps, y, ldy, mean, rstd, None)


def norm_bwd(dy=P, ldg=64, x=2 * P, ldx=64, T=4, H=64, dt=nm.NM_BF16, mean=3 * P, rstd=4 * P, w=5 * P, dx=6 * P,
             lddx=64, dw=7 * P, db=8 * P, od=nm.NM_F32, ws=9 * P, ws_bytes=1 << 20):
    return nm.lib().nm_layernorm_bwd(dy, ldg, x, ldx, T, H, dt, mean, rstd, w, dx, lddx, dw, db, od, ws, ws_bytes,
                                     None)


def test_layernorm_errors():
    assert norm(x=None) == NULL and norm(y=None) == NULL and norm(mean=None) == NULL
    assert norm(T=-1) == SHAPE and norm(H=0, ldx=0, ldy=0) == SHAPE and norm(H=1 << 25, ldx=1 << 25, ldy=1 << 25) == SHAPE
    assert norm(eps=-1.0) == SHAPE and norm(eps=float("nan")) == SHAPE
    assert norm(dt=nm.NM_I8) == UNSUPPORTED and norm(dt=nm.NM_FP8) == UNSUPPORTED
    assert norm(ldx=63) == STRIDE and norm(ldy=63) == STRIDE and norm(ldx=1 << 41) == SHAPE
    assert norm(x=P + 1) == ALIGN and norm(mean=5 * P + 2) == ALIGN and norm(w=2 * P + 2, dt=nm.NM_F32) == ALIGN
    assert norm(y=P) == ALIAS and norm(mean=2 * P) == ALIAS and norm(mean=6 * P + 4) == ALIAS
    assert norm(x=None, y=None, T=0) == OK


def test_layernorm_bwd_errors():
    for name in ("dy", "x", "mean", "rstd", "dx", "ws"):
        assert norm_bwd(**{name: None}) == NULL, name
    assert norm_bwd(od=nm.NM_F16) == UNSUPPORTED and norm_bwd(dt=nm.NM_I32) == UNSUPPORTED
    assert norm_bwd(ldg=63) == STRIDE and norm_bwd(lddx=3) == STRIDE
    assert norm_bwd(ws_bytes=16) == SHAPE
    assert norm_bwd(ws=9 * P + 4) == ALIGN and norm_bwd(db=8 * P + 2) == ALIGN and norm_bwd(dy=P + 1) == ALIGN
    assert norm_bwd(dx=2 * P) == ALIAS and norm_bwd(dw=8 * P) == ALIAS and norm_bwd(ws=6 * P) == ALIAS
    assert norm_bwd(dw=None, db=None, dy=None, T=0) == OK


def test_layernorm_workspace_size():
    b = ctypes.c_size_t()
    f = nm.lib().nm_layernorm_bwd_workspace_size
    assert f(4, 64, ctypes.byref(b)) == OK and b.value >= 64 * 8
    assert f(1 << 20, 4096, ctypes.byref(b)) == OK and b.value <= 1 << 26
    assert f(-1, 64, ctypes.byref(b)) == SHAPE and f(4, 64, None) == NULL
