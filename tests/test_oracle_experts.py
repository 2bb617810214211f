"""Pins of the oracle of grouped products, 4-bit floats and gradient norms, without a GPU."""
import numpy as np
import pytest

from oracle import nm_experts as E
from oracle import nm_oracle as O


def test_rows_of_offsets():
    assert E.rows_of([0, 2, 2, 5], 5) == [(0, 2), (2, 2), (2, 5)]
    assert E.rows_of([-3, 9, 1, 7], 5) == [(0, 5), (5, 5), (1, 5)]


def packed(E_, R, K, n, m, seed):
    w = np.random.default_rng(seed).standard_normal((E_, R, K)).astype(np.float16).view(np.uint16)
    p = [O.prune_pack(w[e], n, m) for e in range(E_)]
    return np.stack([q[0] for q in p]), np.stack([q[1] for q in p])


@pytest.mark.parametrize("n,m", [(2, 4), (1, 4), (1, 8)])
def test_group_gradients_against_differences(n, m):
    rng = np.random.default_rng(5)
    K, R, T, offsets = 32, 8, 6, [0, 2, 2, 6]
    values, idx = packed(3, R, K, n, m, 3)
    act = rng.standard_normal((T, K)).astype(np.float16).view(np.uint16)
    g = rng.standard_normal((T, R)).astype(np.float16).view(np.uint16)
    G = O.half_bits_to_f64(g, "f16")
    y, _, owned = E.group_ref(values, idx, K, n, m, act, offsets, "f16")
    assert owned.all()
    dx, _, _ = E.group_dx_ref(values, idx, K, n, m, g, offsets, "f16")
    dw, _ = E.group_dw_ref(idx, K, n, m, g, act, offsets, "f16")
    assert not dw[1].any()
    # the loss sum G Y is linear in act and in every stored weight: differences are exact but for rounding
    x = O.half_bits_to_f64(act, "f16")
    for t, k in [(0, 3), (1, 31), (4, 0), (5, 17)]:
        e = 0 if t < 2 else 2
        w = O.half_bits_to_f64(O.decompress(values[e], idx[e], K, n, m), "f16")
        step = np.zeros_like(x)
        step[t, k] = 0.5
        diff = (G[t] @ (w @ (x[t] + step[t])) - G[t] @ (w @ (x[t] - step[t])))
        assert abs(diff - dx[t, k]) < 1e-10
    for e, r, s in [(0, 0, 0), (2, 7, 1), (2, 3, K // m * n - 1)]:
        v = values[e].copy()
        loss = []
        for sign in (1, -1):
            w64 = O.half_bits_to_f64(v, "f16")
            w64[r, s] += 0.5 * sign
            dense = np.zeros((R, K))
            from oracle.nm_train import stored_columns
            np.put_along_axis(dense, stored_columns(idx[e], K, n, m), w64, 1)
            lo, hi = E.rows_of(offsets, T)[e]
            loss.append((G[lo:hi] * (x[lo:hi] @ dense.T)).sum())
        assert abs(loss[0] - loss[1] - dw[e, r, s]) < 1e-10


def test_mx_worked_block():
    x = np.zeros((1, 32))
    x[0, :9] = [7.9, -0.25, 0.2500001, 0.75, 1.25, 1.75, 2.5, -3.5, 5.0]
    code, byte = E.mx_quantize_ref(x)
    assert byte[0, 0] == 127                   # largest 7.9: exponent 2, less 2
    want = [6.0, -0.0, 0.5, 1.0, 1.0, 2.0, 2.0, -4.0, 4.0]
    got = E.mx_values_ref(code, byte)[0]
    assert got[:9].tolist() == want and not got[9:].any()
    assert code[0, 1] == 8                     # the sign of a zero stays


def test_mx_against_a_search_of_all_values():
    rng = np.random.default_rng(11)
    x = rng.standard_normal((40, 64)) * 2.0 ** rng.integers(-140, 126, (40, 1))
    x = x.astype(np.float32).astype(np.float64)
    code, byte = E.mx_quantize_ref(x)
    got = E.mx_values_ref(code, byte)
    for t in range(40):
        for b in range(2):
            blk = x[t, 32 * b: 32 * b + 32]
            s = 2.0 ** max(np.floor(np.log2(np.abs(blk).max())) - 2, -127)
            cand = np.concatenate([E.E2M1, -E.E2M1]) * s
            best = np.abs(blk[:, None] - cand).min(axis=1)
            assert (np.abs(blk - got[t, 32 * b: 32 * b + 32]) == best).all()


def test_mx_blocks_of_zeros_and_nonfinite():
    x = np.zeros((3, 32))
    x[1, 4], x[2, 7] = np.inf, np.nan
    code, byte = E.mx_quantize_ref(x)
    assert byte.ravel().tolist() == [0, 255, 255] and not code.any()
    assert not E.mx_values_ref(code, byte)[0].any() and np.isnan(E.mx_values_ref(code, byte)[1:]).all()


def test_mx_pack_layout():
    rng = np.random.default_rng(2)
    code = rng.integers(0, 16, (5, 288)).astype(np.uint8)
    byte = rng.integers(0, 255, (5, 9)).astype(np.uint8)
    q, scale = E.mx_pack_ref(code, byte)
    assert q.shape == (5, 144) and scale.shape == (2, 5, 8)
    assert q[3, 7] == code[3, 14] + 16 * code[3, 15]
    assert scale[1, 4, 0] == byte[4, 8] and scale[0, 2, 5] == byte[2, 5] and not scale[1, :, 1:].any()


def test_grad_clip_by_hand():
    g = [np.array([3.0, 0.0]), np.array([[4.0]]), np.zeros(0)]
    norm, out = E.grad_clip_ref(g, 1.0, 0.0)
    assert norm == 5.0 and np.allclose(out[0], [0.6, 0.0], atol=1e-15) and np.allclose(out[1], 0.8, atol=1e-15)
    assert E.grad_clip_ref(g, 10.0, 0.0)[1][1] == 4.0
    assert E.grad_clip_ref([np.zeros(2)], 0.0, 0.0)[0] == 0.0 and E.grad_clip_ref([], 1.0, 1e-6)[0] == 0.0
