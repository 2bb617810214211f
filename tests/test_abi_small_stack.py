"""The checks of long lists of gradients, without a GPU, on a thread whose stack is small: they
return a status, and two threads at once do not disturb each other.  Fake pointers are never
dereferenced; every call here is one that is refused."""
import ctypes
import os
import subprocess
import sys
import threading

import pytest

import structured_sparse_gemm_nm_amd as nm

pytestmark = pytest.mark.skipif(not os.path.exists(nm.lib_path()), reason="libnmsparse.so not built")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 36          # fake device addresses, this far apart
OK, NULL, SHAPE, UNSUPPORTED, STRIDE, ALIAS, _, ALIGN = range(8)


def call(n, last_out=None, norm=5 * P, clip=True):
    """A list of n tensors of 64 values into others, in descending order; the last output at last_out."""
    vp = ctypes.c_void_p * n
    grads = vp(*(P + 256 * i for i in range(n)))
    outs = [3 * P + 256 * (n - i) for i in range(n)]
    if last_out is not None:
        outs[-1] = last_out
    a = (grads, (ctypes.c_int64 * n)(*[64] * n), (ctypes.c_int * n)(*[nm.NM_F32] * n), n)
    if not clip:
        return nm.lib().nm_grad_norm(*a, norm, 6 * P, 1 << 24, None)
    return nm.lib().nm_grad_clip(*a, 1.0, 1e-6, vp(*outs), norm, 6 * P, 1 << 24, None)


def refusals():
    for n in (1, 254, 255, 256, 5000, 16384):
        assert call(n, last_out=P + 4) == ALIAS and call(n, norm=P + 256 * (n - 1) + 60) == ALIAS
        assert call(n, last_out=3 * P + 256 * n + 1) == ALIGN
        if n > 1:
            assert call(n, last_out=3 * P + 256 * n - 4) == ALIAS and call(n, last_out=P) == ALIAS
        assert call(n, norm=P + 256 * (n - 1) + 60, clip=False) == ALIAS


def test_lists_of_every_length():
    refusals()


SMALL = """
import sys, threading
sys.path[:0] = [{root!r}, {tests!r}]
import test_abi_small_stack as t
t.refusals()                               # (what is imported or built on first use is there)
bad = []
def run():
    try:
        t.refusals()
    except BaseException as e:
        bad.append(e)
threading.stack_size(160 * 1024)
x = threading.Thread(target=run)
x.start()
x.join()
assert not bad, bad
print("done")
"""


def test_small_stack():
    """In a process of its own: a stack that overflows ends it."""
    code = SMALL.format(root=ROOT, tests=os.path.dirname(os.path.abspath(__file__)))
    res = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert res.returncode == 0 and "done" in res.stdout, (res.returncode, res.stderr[-2000:])


def test_threads_at_once():
    bad = []

    def run():
        try:
            for _ in range(3):
                refusals()
        except BaseException as e:
            bad.append(e)
    threads = [threading.Thread(target=run) for _ in range(4)]
    for x in threads:
        x.start()
    for x in threads:
        x.join()
    assert not bad, bad
