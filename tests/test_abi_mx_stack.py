"""C ABI checks, without a GPU, of stacks of 4-bit matrices: the scales of one matrix of a
stack begin on 8 bytes only, and the calls that take them say so.  Fake pointers are never
dereferenced: a call that passes the check of alignment is stopped by the next one."""
import ctypes
import os

import pytest

import structured_sparse_gemm_nm_amd as nm

pytestmark = pytest.mark.skipif(not os.path.exists(nm.lib_path()), reason="libnmsparse.so not built")

P = 1 << 36          # fake device addresses, this far apart
OK, NULL, SHAPE, UNSUPPORTED, STRIDE, ALIAS, _, ALIGN = range(8)


def quantize(x=P, E=3, R=101, K=256, ldx=256, stride=101 * 256, dt=nm.NM_BF16, q=2 * P, s=3 * P):
    return nm.lib().nm_mx_quantize_stack(x, E, R, K, ldx, stride, dt, q, s, None)


def dequantize(q=2 * P, s=3 * P, E=3, R=101, K=256, y=P, ldy=256, stride=101 * 256, dt=nm.NM_BF16):
    return nm.lib().nm_mx_dequantize_stack(q, s, E, R, K, y, ldy, stride, dt, None)


def gemm(ws=2 * P, xs=4 * P, Y=5 * P, E=1, off=None):
    return nm.lib().nm_mx_gemm(P, ws, E, 101, 256, 3 * P, xs, 101, off, Y, 101, nm.NM_F32, None, 0, None)


def test_scales_of_a_stack_begin_on_eight_bytes():
    one = ctypes.c_size_t()
    assert nm.lib().nm_mx_sizes(101, 256, None, ctypes.byref(one)) == OK
    second = 3 * P + one.value                    # the second matrix's scales, all three of odd sizes
    assert second % 16 == 8
    # past the alignment, into the check of what overlaps
    assert quantize(E=1, s=second, q=second - 8 - 64) == ALIAS and quantize(E=1, s=second - 4) == ALIGN
    assert dequantize(E=1, s=second, y=second) == ALIAS and dequantize(E=1, s=second - 4) == ALIGN
    second += P
    assert gemm(xs=second, Y=second - 8) == ALIAS and gemm(xs=second - 4) == ALIGN
    assert gemm(ws=second, xs=7 * P, Y=second - 8) == ALIAS and gemm(ws=second - 4) == ALIGN


def test_stack_refusals():
    for call in (quantize, dequantize):
        assert call(E=-1) == SHAPE and call(E=(1 << 24) + 1) == SHAPE and call(R=-1) == SHAPE and call(K=48) == SHAPE
        assert call(stride=-1) == STRIDE and call(stride=1 << 40) == SHAPE and call(E=1 << 24, stride=1 << 17) == SHAPE
        assert call(E=1 << 24, R=1 << 10, stride=0) == SHAPE
        assert call(dt=nm.NM_I8) == UNSUPPORTED and call(q=2 * P + 8) == ALIGN
        assert call(q=None) == NULL and call(s=None) == NULL
        assert call(E=0, q=None, s=None) == OK and call(R=0, q=None, s=None) == OK
    assert quantize(x=None) == NULL and quantize(ldx=255) == STRIDE and quantize(x=P + 1) == ALIGN
    assert dequantize(y=None) == NULL and dequantize(ldy=255) == STRIDE and dequantize(y=P + 1) == ALIGN
    # what is written must not overlap; what is read may
    assert dequantize(stride=101 * 256 - 1) == STRIDE and dequantize(stride=0) == STRIDE
    assert quantize(stride=0, q=P + 100 * 256 * 2) == ALIAS and quantize(stride=8, q=P + 100 * 256 * 2 + 512 + 16) == ALIAS
    # the last matrix counts
    assert quantize(q=P + 3 * 101 * 256 * 2 - 16) == ALIAS and quantize(s=2 * P + 3 * 101 * 128 - 8) == ALIAS
    assert dequantize(y=2 * P + 3 * 101 * 128 - 2) == ALIAS and dequantize(y=3 * P + 3 * 101 * 8 - 2) == ALIAS
