"""Gradients of the 4-bit weight's products and layer against the formula and against
differences, and the experts' sort of either index type.

Tolerances: an element of dx is off by its fp32 sum, 2^-23 (out + 64) sum |dy| |w|, and half
a bf16 step, 2^-8 of the value.  A difference of two results is a sum of T out
independent roundings, each of at most 2^-8 of its result and so of standard deviation
2^-8 / sqrt(3) of it: eight standard deviations of the sum, and the fp32 sums' bound.
"""
import numpy as np
import pytest
import torch

from oracle import q4_oracle as q4
from parameter_efficient_fine_gb300 import ops

from gpu_util import DEV, assert_no_device_error, to_f64

pytestmark = pytest.mark.gpu

BF, I32, I64 = torch.bfloat16, torch.int32, torch.int64


def _rnd(seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    return lambda *s: torch.randn(*s, generator=gen, device=DEV)


def _weight(rnd, *shape):
    q, s = ops.q4_store(rnd(*shape) / shape[-1] ** 0.5)
    return q, s, q4.q4_decode(q.cpu().numpy(), s.cpu().numpy())


@pytest.mark.parametrize("T", [1, 5, 40, 200])
def test_gradient_of_a_product_element_by_element(T):
    rnd = _rnd(T)
    wq, ws, W = _weight(rnd, 272, 544)
    x, dy = rnd(T, 544).to(BF).requires_grad_(True), rnd(T, 272).to(BF)
    ops.matmul_q4(x, wq, ws).backward(dy)
    d = to_f64(dy)
    ref = d @ W
    bound = (1 + 2.0 ** -8) * 2.0 ** -23 * (272 + 64) * (np.abs(d) @ np.abs(W)) + 2.0 ** -8 * np.abs(ref)
    err = lambda g: (np.abs(g - ref) > bound).mean()  # noqa: E731
    assert err(to_f64(x.grad)) == 0
    # what the bound is for: no gradient, another sign, another weight's are far outside
    assert err(0 * ref) > 0.99 and err(-ref) > 0.99 and err(d @ np.roll(W, 1, 0)) > 0.9
    assert_no_device_error()


@pytest.mark.parametrize("T", [1, 5, 40, 200])
def test_gradient_of_a_product_against_a_difference(T):
    rnd = _rnd(T + 50)
    wq, ws, W = _weight(rnd, 272, 544)
    x, dy = rnd(T, 544).to(BF), rnd(T, 272).to(BF)
    # a direction in which the product moves along dy, so that the sides are large
    step = torch.from_numpy(to_f64(dy) @ W).to(DEV)
    hi, lo = (x.double() + step).to(BF), (x.double() - step).to(BF)
    leaf = x.clone().requires_grad_(True)
    ops.matmul_q4(leaf, wq, ws).backward(dy)
    y1, y0 = to_f64(ops.matmul_q4(hi, wq, ws)), to_f64(ops.matmul_q4(lo, wq, ws))
    d, dx = to_f64(dy), to_f64(hi) - to_f64(lo)
    left, right = ((y1 - y0) * d).sum(), (dx * to_f64(leaf.grad)).sum()
    step_of = 2.0 ** -8 / np.sqrt(3)
    spread = step_of * np.sqrt((((np.abs(y1) ** 2 + np.abs(y0) ** 2)) * d ** 2).sum() + ((dx * to_f64(leaf.grad)) ** 2).sum())
    sums = 2.0 ** -23 * (544 + 64) * ((np.abs(to_f64(hi)) + np.abs(to_f64(lo))) @ np.abs(W).T * np.abs(d)).sum()
    bound = 8 * spread + 2 * sums
    assert abs(left - right) <= bound
    assert abs(right) > 4 * bound                      # so neither 0 nor -right would pass


def test_gradient_of_experts_element_by_element():
    rnd = _rnd(3)
    T, E = 60, 4
    wq, ws, W = _weight(rnd, E, 144, 160)
    off = [0, 5, 5, 40, 55]                            # rows behind the last expert's
    offsets = torch.tensor(off, dtype=I32, device=DEV)
    x, dy = rnd(T, 160).to(BF).requires_grad_(True), rnd(T, 144).to(BF)
    ops.matmul_q4(x, wq, ws, offsets).backward(dy)
    d, ref, mag = to_f64(dy), np.zeros((T, 160)), np.zeros((T, 160))
    for e in range(E):
        rows = slice(off[e], off[e + 1])
        ref[rows], mag[rows] = d[rows] @ W[e], np.abs(d[rows]) @ np.abs(W[e])
    bound = (1 + 2.0 ** -8) * 2.0 ** -23 * (144 + 64) * mag + 2.0 ** -8 * np.abs(ref)
    assert (np.abs(to_f64(x.grad) - ref) <= bound).all()
    assert not x.grad[55:].any()


@pytest.mark.parametrize("T,out,inp,r", [(37, 272, 128, 24), (300, 528, 416, 72)])
def test_gradient_of_a_against_x_itself(T, out, inp, r):
    """x is kept in 8 bits for dA = dxa^T x: E4M3 with a scale per 128 columns, whose random part is
    0.026 of a value; with the bf16 chain, 0.035 of the norm, as for d_mag."""
    rnd = _rnd(T)
    wq, ws, W = _weight(rnd, out, inp)
    A, B, s = (rnd(r, inp) / inp ** 0.5).requires_grad_(True), 0.1 * rnd(out, r), 2.0
    m = torch.ones(out, device=DEV)
    norm, _ = ops.norm_factored(ops.q4_load(wq, ws, torch.float32), A.detach(), B, m, s)
    m = norm * (1 + 0.02 * rnd(out))
    x, dy, g = rnd(T, inp).to(BF), rnd(T, out).to(BF), m / norm
    ops.dora_linear_q4(x, wq, ws, A, B, m, g, norm, s).backward(dy)
    ref = (s * (to_f64(g) * to_f64(dy)) @ to_f64(B)).T @ to_f64(x)
    err = np.linalg.norm(to_f64(A.grad) - ref) / np.linalg.norm(ref)
    assert err <= 0.035, err


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (50, 3, 5), (700, 6, 60), (9000, 2, 16)])
def test_either_index_type_sorts_alike(T, k, E):
    gen = torch.Generator(device=DEV).manual_seed(T)
    expert = torch.randint(-2, E + 2, (T, k), generator=gen, device=DEV)
    assert expert.dtype == I64 and (T == 1 or ((expert < 0) | (expert >= E)).any())
    wide = expert.clone()
    wide[expert < 0] = -(1 << 40)                      # outside any 32-bit reading of them
    wide[expert >= E] = (1 << 32) + 1
    got = [ops.expert_sort(e, E) for e in (expert, expert.to(I32), wide)]
    order, inverse, offsets = q4.expert_sort(expert.cpu().numpy(), E)
    for o, i, f in got:
        assert np.array_equal(o.cpu().numpy(), order) and np.array_equal(i.cpu().numpy(), inverse)
        assert np.array_equal(f.cpu().numpy(), offsets)
