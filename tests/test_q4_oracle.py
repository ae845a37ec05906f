"""Pins of the 4-bit oracle, on the CPU."""
import numpy as np
import pytest

from oracle import q4_oracle as q4


def test_values_of_the_codes():
    assert q4.e2m1_table().tolist() == [0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6]


def test_hand_made_group():
    x = np.zeros((1, 32))
    x[0, :6] = [6.0, -3.0, 0.25, 0.75, 5.0, -0.3]
    q, s = q4.q4_encode(x)
    assert s.tolist() == [[127]]
    # 6 -> 7; -3 -> 13; .25 is half way between 0 and .5: even 0; .75 between .5 and 1: even 2;
    # 5 between 4 and 6: even 6; -.3 -> -.5: 9
    assert q[0, :3].tolist() == [7 | 13 << 4, 0 | 2 << 4, 6 | 9 << 4]
    x[0, 0] = 6.5                                     # past 6: the next power of two
    assert q4.q4_encode(x)[1].tolist() == [[128]]


def test_groups_of_zeros_and_not_finite():
    x = np.zeros((3, 64))
    x[1, 40], x[2, 3] = np.inf, np.nan
    x[2, 60] = -12.0
    q, s = q4.q4_encode(x)
    assert s.tolist() == [[2, 2], [2, 255], [255, 128]]
    v = q4.q4_decode(q, s)
    assert np.isnan(v[1, 32:]).all() and np.isnan(v[2, :32]).all() and (v[0] == 0).all()
    assert v[2, 60] == -12.0


def test_encode_is_the_identity_on_the_form():
    rng = np.random.default_rng(0)
    code = rng.integers(0, 16, (40, 64))
    code[:, ::32] = 7                                 # a largest value in every group
    v = q4.e2m1_table()[code] * np.exp2(rng.integers(-120, 120, (40, 2))).repeat(32, 1)
    q, s = q4.q4_encode(v)
    assert np.array_equal(q4.q4_decode(q, s), v)


def test_nearest_by_brute_force():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((50, 32)) * np.exp2(rng.integers(-30, 30, (50, 1)))
    q, s = q4.q4_encode(x)
    v = q4.q4_decode(q, s)
    unit = np.exp2(s.astype(float) - 127)
    best = np.abs(x[..., None] / unit[..., None] - q4.e2m1_table()).min(-1)
    assert np.allclose(np.abs(x - v) / unit, best, rtol=0, atol=1e-12)
    top = np.abs(x).max(1, keepdims=True)
    assert ((top <= 6 * unit) & (top > 3 * unit)).all()


@pytest.mark.parametrize("offsets", [None, [0, 2, 2, 5]])
def test_products_are_the_dense_ones(offsets):
    rng = np.random.default_rng(2)
    E = 1 if offsets is None else 3
    forms = [q4.q4_encode(rng.standard_normal((6, 64))) for _ in range(E)]
    wq, ws = (np.stack(f) for f in zip(*forms))
    x, dy = rng.standard_normal((6, 64)), rng.standard_normal((6, 6))
    if offsets is None:
        wq, ws = wq[0], ws[0]
        W = q4.q4_decode(wq, ws)
        assert np.allclose(q4.matmul_q4(x, wq, ws), x @ W.T) and np.allclose(q4.matmul_q4_t(dy, wq, ws), dy @ W)
        return
    y, dx = q4.matmul_q4(x, wq, ws, offsets), q4.matmul_q4_t(dy, wq, ws, offsets)
    for t, e in enumerate([0, 0, 2, 2, 2]):
        W = q4.q4_decode(wq[e], ws[e])
        assert np.allclose(y[t], W @ x[t]) and np.allclose(dx[t], dy[t] @ W)
    assert np.isnan(y[5]).all() and np.isnan(dx[5]).all()


def test_routing_by_hand():
    expert = np.array([[2, 0], [0, 0], [-1, 2], [7, 1]])
    order, inverse, offsets = q4.expert_sort(expert, 3)
    assert order.tolist() == [1, 2, 3, 7, 0, 5, 4, 6]
    assert inverse.tolist() == [[4, 0], [1, 2], [6, 5], [7, 3]]
    assert offsets.tolist() == [0, 3, 4, 6]
    x = np.array([[1.0], [10.0], [100.0], [1000.0]])
    xs = q4.expert_send(x, inverse, offsets, np.full((8, 1), -5.0))
    assert xs[:, 0].tolist() == [1, 10, 10, 1000, 1, 100, -5, -5]
    w = np.array([[0.5, 2.0], [1.0, 3.0], [9.0, 1.0], [9.0, 4.0]])
    assert q4.expert_return(xs, inverse, offsets, w)[:, 0].tolist() == [2.5, 40.0, 100.0, 4000.0]
    assert q4.expert_return(xs, inverse, offsets, None)[:, 0].tolist() == [2, 20, 100, 1000]


def test_return_gradient_by_differences():
    rng = np.random.default_rng(3)
    expert = np.array([[0, 1], [1, 1], [-1, 0]])
    _, inverse, offsets = q4.expert_sort(expert, 2)
    ys, w, dy = rng.standard_normal((6, 4)), rng.standard_normal((3, 2)), rng.standard_normal((3, 4))
    d_ys, d_w = q4.expert_return_bwd(dy, ys, inverse, offsets, w, np.zeros((6, 4)))
    loss = lambda a, b: (dy * q4.expert_return(a, inverse, offsets, b)).sum()  # noqa: E731
    h = 1e-6
    for arr, grad, other in ((ys, d_ys, "ys"), (w, d_w, "w")):
        for i in np.ndindex(arr.shape):
            up, dn = arr.copy(), arr.copy()
            up[i] += h
            dn[i] -= h
            a, b = ((up, w), (dn, w)) if other == "ys" else ((ys, up), (ys, dn))
            assert abs((loss(*a) - loss(*b)) / (2 * h) - grad[i]) < 1e-8
