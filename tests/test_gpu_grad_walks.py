"""Norm and clipping of lists so large that workgroups walk from chunk to chunk, forward in the
norm and backward in the clipping, across tensors; of so many parts that their sum is taken by a
launch of its own; and of as many tensors as a launch takes and one more.  Bounds as in
test_gpu_grad (fewer than 2^28 squares a list)."""
import numpy as np
import pytest

from gpu_util import log
from test_gpu_grad import check, grads

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

CHUNK = 32768        # bytes a workgroup takes at a time; a launch has at most 2048 workgroups


def chunks(gs):
    return sum(-(-g.numel() * g.element_size() // CHUNK) for g in gs)


@pytest.mark.parametrize("in_place", [False, True])
def test_walks_over_uneven_tensors(in_place):
    """About 165 MB: large tensors with runs of small and empty ones between them, every type."""
    log(f"grad walks in_place={in_place}")
    rng = np.random.default_rng(7)
    small = [((int(k),), ["bf16", "f32", "f16"][i % 3]) for i, k in enumerate(rng.integers(0, 40000, 60))]
    shapes = [((9000001,), "f32"), *small[:20], ((30000007,), "bf16"), ((0,), "f16"), ((1,), "f32"), *small[20:40],
              ((3001, 3333), "f16"), *small[40:], ((5500, 1001), "f32"), ((3,), "bf16")]
    gs = grads(shapes, 3, 0.01)
    assert chunks(gs) > 2 * 2048 and len(gs) <= 170          # one launch, every workgroup twice and more
    check(gs, 0.7, in_place=in_place)


@pytest.mark.parametrize("in_place", [False, True])
def test_sums_of_many_parts(in_place):
    """600 tensors of 8 to 10 chunks: three launches of the norm, 4096 parts and more."""
    log(f"grad many parts in_place={in_place}")
    rng = np.random.default_rng(8)
    shapes = [((int(k) // (4 if i % 3 == 0 else 2),), ["f32", "bf16", "f16"][i % 3])
              for i, k in enumerate(rng.integers(8 * CHUNK - 5000, 10 * CHUNK, 600))]
    gs = grads(shapes, 4, 0.01)
    parts = sum(min(2048, chunks(gs[i: i + 262])) for i in range(0, len(gs), 262))
    assert parts > 4096
    check(gs, 0.7, in_place=in_place)


@pytest.mark.parametrize("count", [170, 171, 262, 263, 340, 341, 524, 525])
def test_as_many_tensors_as_a_launch_takes(count):
    log(f"grad {count} tensors")
    rng = np.random.default_rng(count)
    shapes = [((int(k),), ["f32", "bf16", "f16"][i % 3]) for i, k in enumerate(rng.integers(1, 3000, count))]
    check(grads(shapes, count), 1.0)
    check(grads(shapes, count), 1.0, in_place=True)
    # empty tensors take no place in a launch
    some = [s for i, s in enumerate(shapes) for s in ([s, ((0,), "f16")] if i % 5 == 0 else [s])]
    check(grads(some, count), 1.0)
