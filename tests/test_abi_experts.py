"""C ABI and binding checks, without a GPU, of the products grouped by expert, the
4-bit floats and the gradients' norm: every argument error is caught on the host
before any HIP call (fake pointers are never dereferenced)."""
import ctypes
import os

import pytest

import structured_sparse_gemm_nm_amd as nm

pytestmark = pytest.mark.skipif(not os.path.exists(nm.lib_path()), reason="libnmsparse.so not built")

P = 1 << 36          # fake device addresses, this far apart
OK, NULL, SHAPE, UNSUPPORTED, STRIDE, ALIAS, _, ALIGN = range(8)
INF, NAN = float("inf"), float("nan")


def group(values=P, idx=2 * P, E=3, R=64, K=64, n=2, m=4, dt=nm.NM_BF16, act=3 * P, T=4, ldx=64, off=4 * P, Y=5 * P,
          ldy=64, od=nm.NM_BF16, ws=6 * P, wsb=1 << 20):
    return nm.lib().nm_group_spmm(values, idx, E, R, K, n, m, dt, act, T, ldx, off, Y, ldy, od, ws, wsb, None)


def group_dx(values=P, idx=2 * P, E=3, R=64, K=64, n=2, m=4, dt=nm.NM_BF16, G=3 * P, T=4, ldg=64, off=4 * P, dX=5 * P,
             lddx=64, od=nm.NM_BF16, ws=6 * P, wsb=1 << 20):
    return nm.lib().nm_group_spmm_dx(values, idx, E, R, K, n, m, dt, G, T, ldg, off, dX, lddx, od, ws, wsb, None)


def group_dw(idx=2 * P, E=3, R=64, K=64, n=2, m=4, dt=nm.NM_BF16, G=3 * P, T=4, ldg=64, act=7 * P, ldx=64, off=4 * P,
             dW=5 * P, od=nm.NM_BF16, ws=6 * P, wsb=1 << 24):
    return nm.lib().nm_group_spmm_dw(idx, E, R, K, n, m, dt, G, T, ldg, act, ldx, off, dW, od, ws, wsb, None)


@pytest.mark.parametrize("call", [group, group_dx, group_dw])
def test_group_errors(call):
    assert call(dt=nm.NM_I8) == UNSUPPORTED and call(od=nm.NM_F16) == UNSUPPORTED and call(n=3) == UNSUPPORTED
    assert call(E=0) == SHAPE and call(E=65536) == SHAPE and call(T=-1) == SHAPE and call(T=(1 << 24) + 1) == SHAPE
    assert call(K=40, **({"ldx": 64} if call is not group_dx else {})) == SHAPE
    assert call(idx=None) == NULL and call(off=None) == NULL and call(off=4 * P + 2) == ALIGN
    assert call(idx=2 * P + 4) == ALIGN
    if call is not group_dw:
        many = dict(E=300, T=30000)          # enough experts for a table
        assert call(ws=None, **many) == NULL and call(wsb=16, **many) == SHAPE
        assert call(ws=6 * P + 8, **many) == ALIGN and call(ws=P, **many) == ALIAS
        assert call(values=None) == NULL and call(values=P + 8) == ALIGN


def test_group_shapes_strides_and_aliases():
    assert group(act=None) == NULL and group(Y=None) == NULL
    assert group(R=1 << 23, ldy=1 << 23) == SHAPE and group(ldx=1 << 23) == SHAPE
    assert group(ldx=56) == STRIDE and group(ldy=63) == STRIDE and group(ldx=68) == ALIGN and group(act=3 * P + 8) == ALIGN
    assert group(Y=3 * P) == ALIAS and group(Y=4 * P) == ALIAS
    # the second and third expert's weights are inputs too
    assert group(Y=P + 64 * 32 * 2 * 2 + 16) == ALIAS
    assert group(T=0, values=None, act=None, Y=None, ws=None, off=None) == OK and group(R=0, ldy=0, values=None) == OK
    assert group_dx(G=None) == NULL and group_dx(dX=None) == NULL and group_dx(R=60) == SHAPE
    assert group_dx(K=48) == SHAPE and group_dx(ldg=56) == STRIDE and group_dx(lddx=56) == STRIDE
    assert group_dx(ldg=68) == ALIGN and group_dx(dX=3 * P) == ALIAS and group_dx(ldg=1 << 23) == SHAPE
    assert group_dx(T=0, G=None, dX=None, ws=None) == OK
    assert group_dw(G=None) == NULL and group_dw(act=None) == NULL and group_dw(dW=None) == NULL
    assert group_dw(R=60) == SHAPE and group_dw(K=48) == SHAPE and group_dw(ldx=56) == STRIDE and group_dw(ldg=68) == ALIGN
    assert group_dw(T=1 << 20, ldg=1 << 12) == SHAPE and group_dw(dW=7 * P) == ALIAS and group_dw(dW=2 * P) == ALIAS
    assert group_dw(R=0, dW=None, idx=None) == OK
    # many tokens, few tiles: partial sums
    assert group_dw(T=8192, ws=None) == NULL and group_dw(T=8192, wsb=64) == SHAPE and group_dw(T=8192, ws=6 * P + 8) == ALIGN
    assert group_dw(T=8192, ws=3 * P) == ALIAS


def test_group_workspace_sizes():
    b = ctypes.c_size_t()
    ref = ctypes.byref(b)
    f = nm.lib().nm_group_spmm_workspace_size
    assert f(300, 64, 64, 2, 4, nm.NM_BF16, 30000, nm.NM_F32, ref) == OK and 0 < b.value < 1 << 16
    assert f(8, 2048, 256, 2, 4, nm.NM_BF16, 2000, nm.NM_F32, ref) == OK and 0 < b.value < 1 << 16
    assert f(8, 64, 64, 2, 4, nm.NM_BF16, 8, nm.NM_F32, ref) == OK and b.value == 0
    assert f(8, 64, 64, 2, 4, nm.NM_BF16, 0, nm.NM_F32, ref) == OK and b.value == 0
    assert f(0, 64, 64, 2, 4, nm.NM_BF16, 10, nm.NM_F32, ref) == SHAPE
    assert f(8, 64, 64, 2, 4, nm.NM_BF16, 10, nm.NM_F32, None) == NULL
    g = nm.lib().nm_group_spmm_dx_workspace_size
    assert g(300, 64, 64, 1000, ref) == OK and 0 < b.value < 1 << 16 and g(8, 64, 64, 1000, ref) == OK and b.value == 0
    assert g(8, 4096, 64, 100, ref) == OK and 2 * 100 * 64 * 4 <= b.value < 1 << 24       # in shares
    w = nm.lib().nm_group_spmm_dw_workspace_size
    assert w(8, 64, 64, 2, 4, 1000, ref) == OK and b.value == 0
    assert w(2, 64, 64, 2, 4, 8192, ref) == OK and b.value == 16 * 2 * 64 * 32 * 4
    assert w(2, 64, 64, 2, 4, -1, ref) == SHAPE and w(2, 64, 64, 3, 4, 5, ref) == UNSUPPORTED and w(2, 64, 64, 2, 4, 5, None) == NULL
    assert g(8, 64, 64, -1, ref) == SHAPE and g(1 << 20, 64, 64, 5, ref) == SHAPE and g(8, 64, 64, 10, None) == NULL


def test_experts_without_rows_of_weight():
    """R = 0 is a valid, empty weight however many tokens there are: nothing to share out."""
    b = ctypes.c_size_t(1)
    ref = ctypes.byref(b)
    for T in (0, 1, 1 << 14, 1 << 24):
        assert nm.lib().nm_group_spmm_dw_workspace_size(2, 0, 64, 2, 4, T, ref) == OK and b.value == 0
        assert nm.lib().nm_group_spmm_workspace_size(2, 0, 64, 2, 4, nm.NM_BF16, T, nm.NM_F32, ref) == OK and b.value == 0
        assert nm.lib().nm_group_spmm_dx_workspace_size(2, 0, 64, T, ref) == OK
        assert group_dw(R=0, T=T, ldg=8, dW=None, idx=None) == OK


def quantize(x=P, T=4, K=64, ldx=64, dt=nm.NM_BF16, q=2 * P, s=3 * P):
    return nm.lib().nm_mx_quantize(x, T, K, ldx, dt, q, s, None)


def dequantize(q=2 * P, s=3 * P, T=4, K=64, y=P, ldy=64, dt=nm.NM_BF16):
    return nm.lib().nm_mx_dequantize(q, s, T, K, y, ldy, dt, None)


def gemm(wq=P, ws=2 * P, E=1, R=64, K=64, xq=3 * P, xs=4 * P, T=4, off=None, Y=5 * P, ldy=64, od=nm.NM_BF16,
         wk=6 * P, wkb=1 << 20):
    return nm.lib().nm_mx_gemm(wq, ws, E, R, K, xq, xs, T, off, Y, ldy, od, wk, wkb, None)


def test_mx_errors():
    for call in (quantize, dequantize):
        assert call(q=None) == NULL and call(s=None) == NULL
        assert call(dt=nm.NM_I8) == UNSUPPORTED and call(T=-1) == SHAPE and call(T=(1 << 24) + 1) == SHAPE
        assert call(q=2 * P + 4) == ALIGN and call(s=3 * P + 8) == ALIGN
        assert call(T=0, q=None, s=None) == OK
    assert quantize(x=None) == NULL and quantize(K=48) == SHAPE and quantize(K=0, ldx=0) == SHAPE
    assert quantize(ldx=63) == STRIDE and quantize(x=P + 1) == ALIGN and quantize(x=P + 2, dt=nm.NM_F32) == ALIGN
    assert quantize(q=P) == ALIAS and quantize(s=2 * P) == ALIAS and quantize(K=1 << 23, ldx=1 << 23) == SHAPE
    assert dequantize(y=None) == NULL and dequantize(ldy=63) == STRIDE and dequantize(y=3 * P) == ALIAS
    for name in ("wq", "ws", "xq", "xs", "Y"):
        assert gemm(**{name: None}) == NULL, name
    assert gemm(E=2) == SHAPE
    assert gemm(E=0, off=7 * P) == SHAPE and gemm(E=65536, off=7 * P) == SHAPE and gemm(K=80) == SHAPE
    assert gemm(R=(1 << 22) + 1, ldy=1 << 23) == SHAPE and gemm(T=-1) == SHAPE and gemm(od=nm.NM_I32) == UNSUPPORTED
    assert gemm(ldy=63) == STRIDE and gemm(xq=3 * P + 8) == ALIGN and gemm(off=7 * P + 1) == ALIGN
    assert gemm(Y=P) == ALIAS and gemm(Y=4 * P) == ALIAS and gemm(Y=7 * P, off=7 * P) == ALIAS
    assert gemm(T=0, xq=None) == OK and gemm(R=0, ldy=0, wq=None) == OK


def test_mx_sizes():
    a, b = ctypes.c_size_t(), ctypes.c_size_t()
    f = nm.lib().nm_mx_sizes
    assert f(5, 288, ctypes.byref(a), ctypes.byref(b)) == OK and (a.value, b.value) == (5 * 144, 2 * 5 * 8)
    assert f(5, 288, None, None) == OK and f(5, 30, None, None) == SHAPE and f(-1, 32, None, None) == SHAPE
    g = nm.lib().nm_mx_gemm_workspace_size
    assert g(1, 64, 64, 4, 0, nm.NM_F32, ctypes.byref(a)) == OK and g(1, 64, 64, 4, 0, nm.NM_F32, None) == NULL
    assert g(2, 64, 64, 4, 0, nm.NM_F32, ctypes.byref(a)) == SHAPE
    assert g(2, 64, 64, 4, 1, nm.NM_F32, ctypes.byref(a)) == OK and a.value < 1 << 16


def grads(ptrs=(P, 2 * P), counts=(10, 20), dts=(nm.NM_F32, nm.NM_BF16), out=(3 * P, 4 * P), norm=5 * P, ws=6 * P,
          wsb=1 << 20, max_norm=1.0, eps=1e-6, clip=True):
    n = len(ptrs)
    vp = ctypes.c_void_p * n
    a = (vp(*ptrs), (ctypes.c_int64 * n)(*counts), (ctypes.c_int * n)(*dts), n)
    if not clip:
        return nm.lib().nm_grad_norm(*a, norm, ws, wsb, None)
    return nm.lib().nm_grad_clip(*a, max_norm, eps, None if out is None else vp(*out), norm, ws, wsb, None)


def test_grad_errors():
    for clip in (False, True):
        assert grads(norm=None, clip=clip) == NULL and grads(ws=None, clip=clip) == NULL
        assert grads(ptrs=(P, None), clip=clip) == NULL and grads(wsb=64, clip=clip) == SHAPE
        assert grads(counts=(-1, 20), clip=clip) == SHAPE and grads(counts=((1 << 36) + 1, 20), clip=clip) == SHAPE
        assert grads(dts=(nm.NM_F32, nm.NM_I8), clip=clip) == UNSUPPORTED
        assert grads(ptrs=(P + 2, 2 * P), clip=clip) == ALIGN and grads(ws=6 * P + 8, clip=clip) == ALIGN
        assert grads(norm=5 * P + 2, clip=clip) == ALIGN
        assert grads(norm=P + 36, clip=clip) == ALIAS and grads(ws=2 * P + 32 - (1 << 10), clip=clip) == ALIAS
    assert grads(out=None) == NULL and grads(out=(3 * P, None)) == NULL and grads(out=(3 * P, 4 * P + 1)) == ALIGN
    assert grads(max_norm=-1.0) == SHAPE and grads(max_norm=NAN) == SHAPE and grads(eps=-1.0) == SHAPE
    assert grads(eps=INF) == SHAPE and grads(eps=NAN) == SHAPE


def test_grad_aliases():
    assert grads(out=(P, 2 * P), norm=P + 8) == ALIAS
    assert grads(out=(2 * P, P)) == ALIAS                      # each into the other
    assert grads(out=(P + 4, 4 * P)) == ALIAS                  # into itself, but shifted
    assert grads(out=(3 * P, 3 * P + 36)) == ALIAS             # outputs over one another
    assert grads(ptrs=(P, P), dts=(0, 0), out=(P, P), counts=(10, 10)) == ALIAS     # one tensor twice, in place
    assert grads(ptrs=(P, P + 8), dts=(0, 0), out=(P, P + 8), counts=(10, 10)) == ALIAS
    assert grads(out=(3 * P, 5 * P)) == ALIAS and grads(out=(6 * P + 64, 4 * P)) == ALIAS
    assert grads(out=(2 * P + 39, 4 * P), dts=(nm.NM_BF16, nm.NM_BF16)) == ALIGN
    assert grads(out=(2 * P + 38, 4 * P), dts=(nm.NM_BF16, nm.NM_BF16)) == ALIAS    # its last element


def test_grad_workspace_size():
    b = ctypes.c_size_t()
    f = nm.lib().nm_grad_workspace_size
    assert f(0, ctypes.byref(b)) == OK and f(500, ctypes.byref(b)) == OK and b.value < 1 << 18
    assert f(16385, ctypes.byref(b)) == SHAPE and f(-1, ctypes.byref(b)) == SHAPE and f(1, None) == NULL


# ---- the binding's own checks come before anything touches a device

torch = pytest.importorskip("torch")


def test_binding_refuses_cpu_tensors_and_wrong_shapes():
    bf = torch.bfloat16
    idx = torch.zeros(2, 16, 2, dtype=torch.int32)
    values, act = torch.zeros(2, 16, 32, dtype=bf), torch.zeros(5, 64, dtype=bf)
    offsets = torch.tensor([0, 2, 5], dtype=torch.int32)
    with pytest.raises(ValueError, match="HIP device"):
        nm.nm_group_spmm(values, idx, act, offsets, 64)
    for bad in (offsets[:2], offsets.long(), torch.zeros(6, dtype=torch.int32)[::2]):
        with pytest.raises(ValueError, match="offsets"):
            nm.nm_group_spmm(values, idx, act, bad, 64)
    with pytest.raises(ValueError, match="idx"):
        nm.nm_group_spmm(values, idx[:, :, :1], act, offsets, 64)
    with pytest.raises(TypeError):
        nm.nm_group_spmm(values, idx, act.float(), offsets, 64)
    with pytest.raises(ValueError, match="HIP device"):
        nm.nm_mx_quantize(act)
    with pytest.raises(ValueError, match="HIP device"):
        nm.nm_grad_norm([act])
    with pytest.raises(ValueError, match="outputs for"):
        nm.nm_grad_list([act], [])
    with pytest.raises(TypeError, match="gradients are"):
        nm.nm_grad_list([idx])
    q, s = torch.zeros(5, 32, dtype=torch.uint8), torch.zeros(1, 5, 8, dtype=torch.uint8)
    with pytest.raises(ValueError, match="HIP device"):
        nm.nm_mx_gemm(q, s, q, s)
    with pytest.raises(ValueError, match="xscale"):
        nm.nm_mx_gemm(q, s, q, s[:, :4])
    with pytest.raises(ValueError, match="wq"):
        nm.nm_mx_gemm(q, s, q, s, offsets)
