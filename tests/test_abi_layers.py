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


def adapter(values=P, idx=2 * P, R=64, K=64, n=2, m=4, dt=nm.NM_BF16, act=3 * P, T=4, ldx=64, ids=4 * P, A=5 * P,
            B=6 * P, scale=7 * P, na=3, r=8, xa=8 * P, Y=9 * P, ldy=64, od=nm.NM_BF16, ws=10 * P, wsb=1 << 20):
    return nm.lib().nm_adapter_spmm(values, idx, R, K, n, m, dt, act, T, ldx, ids, A, B, scale, na, r, xa, Y, ldy, od,
                                    ws, wsb, None)


def adapter_bwd(values=P, idx=2 * P, R=64, K=64, n=2, m=4, dt=nm.NM_BF16, G=11 * P, ldg=64, act=3 * P, T=4, ldx=64,
                xa=8 * P, ids=4 * P, A=5 * P, B=6 * P, scale=7 * P, na=3, r=8, dX=9 * P, lddx=64, dA=12 * P, dB=13 * P,
                od=nm.NM_BF16, ws=10 * P, wsb=1 << 20):
    return nm.lib().nm_adapter_spmm_bwd(values, idx, R, K, n, m, dt, G, T, ldg, act, ldx, xa, ids, A, B, scale, na, r,
                                        dX, lddx, dA, dB, od, ws, wsb, None)


def test_adapter_errors():
    for name in ("values", "idx", "act", "ids", "A", "B", "scale", "xa", "Y", "ws"):
        assert adapter(**{name: None, "T": 40}) == NULL, name
    assert adapter(dt=nm.NM_I8) == UNSUPPORTED and adapter(od=nm.NM_F16) == UNSUPPORTED and adapter(n=3) == UNSUPPORTED
    assert adapter(r=0) == SHAPE and adapter(r=257) == SHAPE and adapter(na=-1) == SHAPE and adapter(na=65536) == SHAPE
    assert adapter(T=(1 << 24) + 1) == SHAPE and adapter(T=-1) == SHAPE and adapter(K=40, ldx=40) == SHAPE
    assert adapter(R=1 << 23, ldy=1 << 23) == SHAPE and adapter(ldx=1 << 24) == SHAPE
    assert adapter(ldx=56) == STRIDE and adapter(ldy=63) == STRIDE and adapter(ldx=68) == ALIGN
    assert adapter(A=5 * P + 8) == ALIGN and adapter(ids=4 * P + 2) == ALIGN and adapter(xa=8 * P + 4) == ALIGN
    assert adapter(Y=3 * P) == ALIAS and adapter(xa=9 * P) == ALIAS and adapter(Y=7 * P) == ALIAS
    assert adapter(T=0, values=None, idx=None, act=None, ids=None, xa=None, Y=None) == OK


def test_adapter_bwd_errors():
    for name in ("values", "idx", "G", "act", "ids", "A", "B", "scale", "xa", "dA", "dB", "ws"):
        assert adapter_bwd(**{name: None}) == NULL, name
    assert adapter_bwd(R=60, ldg=64) == SHAPE and adapter_bwd(K=48) == SHAPE and adapter_bwd(wsb=16) == SHAPE
    assert adapter_bwd(od=nm.NM_F16) == UNSUPPORTED and adapter_bwd(dt=nm.NM_FP8) == UNSUPPORTED
    assert adapter_bwd(ldg=56) == STRIDE and adapter_bwd(lddx=56) == STRIDE and adapter_bwd(ldx=68) == ALIGN
    assert adapter_bwd(dA=5 * P) == ALIAS and adapter_bwd(dB=12 * P) == ALIAS and adapter_bwd(dX=11 * P) == ALIAS
    assert adapter_bwd(dA=12 * P + 4) == ALIGN
    assert adapter_bwd(T=0, na=0, A=None, B=None, scale=None, dA=None, dB=None, G=None, act=None) == OK


def test_adapter_workspace_sizes():
    b = ctypes.c_size_t()
    fwd, bwd = nm.lib().nm_adapter_spmm_workspace_size, nm.lib().nm_adapter_spmm_bwd_workspace_size
    ref = ctypes.byref(b)
    assert fwd(64, 64, 2, 4, nm.NM_BF16, 40, 64, 3, 8, nm.NM_BF16, ref) == OK and b.value >= 40 * 64 * 4
    assert fwd(64, 64, 2, 4, nm.NM_BF16, 40, 64, 3, 8, nm.NM_F32, ref) == OK and b.value >= 40 * 3 * 8 * 2
    assert fwd(64, 64, 2, 4, nm.NM_BF16, 9, 64, 3, 8, nm.NM_F32, ref) == OK and b.value == 0
    assert bwd(64, 64, 2, 4, nm.NM_BF16, 40, 3, 8, nm.NM_BF16, ref) == OK and b.value >= 40 * 8 * 4
    assert fwd(64, 64, 2, 4, nm.NM_BF16, 40, 64, 3, 8, nm.NM_F16, ref) == UNSUPPORTED
    assert bwd(64, 64, 2, 4, nm.NM_BF16, 40, 3, 8, nm.NM_BF16, None) == NULL


def xent(x=P, T=4, H=64, ldx=64, w=2 * P, V=100, ldw=64, dt=nm.NM_BF16, labels=3 * P, loss=4 * P, lse=5 * P, ws=6 * P,
         wsb=1 << 20):
    return nm.lib().nm_xent(x, T, H, ldx, w, V, ldw, dt, labels, loss, lse, ws, wsb, None)


def xent_bwd(x=P, T=4, H=64, ldx=64, w=2 * P, V=100, ldw=64, dt=nm.NM_BF16, labels=3 * P, lse=5 * P, dloss=7 * P,
             dx=8 * P, lddx=64, dxt=nm.NM_F32, dw=9 * P, lddw=64, dwt=nm.NM_BF16, ws=6 * P, wsb=1 << 24):
    return nm.lib().nm_xent_bwd(x, T, H, ldx, w, V, ldw, dt, labels, lse, dloss, dx, lddx, dxt, dw, lddw, dwt, ws, wsb,
                                None)


def test_xent_errors():
    for name in ("x", "w", "labels", "loss", "lse", "ws"):
        assert xent(**{name: None}) == NULL, name
    assert xent(dt=nm.NM_F32) == UNSUPPORTED
    assert xent(H=60) == SHAPE and xent(H=0) == SHAPE and xent(V=0) == SHAPE and xent(T=-1) == SHAPE
    assert xent(T=1 << 23) == SHAPE and xent(V=1 << 25) == SHAPE and xent(T=1 << 22, V=1 << 24) == SHAPE
    assert xent(ldx=1 << 23) == SHAPE and xent(wsb=8) == SHAPE
    assert xent(ldx=56) == STRIDE and xent(ldw=56) == STRIDE and xent(ldw=68) == ALIGN
    assert xent(x=P + 8) == ALIGN and xent(labels=3 * P + 2) == ALIGN
    assert xent(loss=5 * P) == ALIAS and xent(lse=P) == ALIAS and xent(ws=2 * P) == ALIAS
    assert xent(T=0, x=None, labels=None, loss=None, lse=None, ws=None) == OK


def test_xent_bwd_errors():
    for name in ("x", "w", "labels", "lse", "dloss", "ws"):
        assert xent_bwd(**{name: None}) == NULL, name
    assert xent_bwd(dxt=nm.NM_F16) == UNSUPPORTED and xent_bwd(dwt=nm.NM_F16) == UNSUPPORTED
    assert xent_bwd(lddx=56) == STRIDE and xent_bwd(lddw=66) == ALIGN and xent_bwd(wsb=1000) == SHAPE
    assert xent_bwd(dx=9 * P) == ALIAS and xent_bwd(dw=P) == ALIAS and xent_bwd(ws=8 * P) == ALIAS
    assert xent_bwd(dx=None, dw=None) == OK and xent_bwd(T=0, dw=None) == OK


def test_xent_workspace_sizes():
    b = ctypes.c_size_t()
    L = nm.lib()
    assert L.nm_xent_workspace_size(2048, 32000, 4096, nm.NM_BF16, ctypes.byref(b)) == OK
    assert b.value < 2048 * 32000 // 8                      # far below the logits
    assert L.nm_xent_bwd_workspace_size(4096, 1 << 20, 4096, nm.NM_BF16, 1, 1, ctypes.byref(b)) == OK
    assert b.value < 1 << 30                                # pieces: bounded whatever the vocabulary
    assert L.nm_xent_bwd_workspace_size(4, 100, 60, nm.NM_BF16, 1, 1, ctypes.byref(b)) == SHAPE
    assert L.nm_xent_workspace_size(4, 100, 64, nm.NM_BF16, None) == NULL
