"""GPU parity of the experts' sort, send and return with their oracle, through the C ABI.

Tolerances: indexes and sent rows are equal; y is an fp32 sum of k products and one
rounding, d_ys one product and one rounding, d_weight an fp32 sum over cols terms:
2^-24 per addition or product of the sum of magnitudes, and half a step of the result's
type (bf16 2^-8; fp32 2^-24).
"""
import numpy as np
import pytest
import torch

import parameter_efficient_fine_gb300 as dora
from oracle import q4_oracle as q4

from gpu_util import DEV, check_bound, f32_dev, to_f64
from test_gpu_guards import Guarded
from test_gpu_q4 import act, act_to_f64

pytestmark = pytest.mark.gpu

I32 = torch.int32


def sort(expert, experts):
    T, k = expert.shape
    order = torch.full((T * k,), -9, dtype=I32, device=DEV)
    inverse = torch.full((T, k), -9, dtype=I32, device=DEV)
    offsets = torch.full((experts + 1,), -9, dtype=I32, device=DEV)
    dora.dora_expert_sort(expert, experts, order, inverse, offsets)
    return order, inverse, offsets


def entries(rng, T, k, E, kind):
    e = rng.integers(0, E, (T, k))
    if kind == "padded":
        e[rng.random((T, k)) < 0.3] = -1
        e[T // 2] = E
    elif kind == "one":
        e[:] = E - 1
    elif kind == "none":
        e[:] = np.where(rng.random((T, k)) < 0.5, -1, E + 3)
    return e


CASES = [(1, 1, 1), (1, 8, 64), (3, 2, 2), (17, 3, 5), (63, 6, 60), (128, 8, 300), (1000, 4, 33), (5000, 7, 16), (333, 1, 4096), (4097, 1, 3), (8192, 8, 64),
         (20001, 2, 1024), (5000, 1, 1025), (16384, 3, 200)]


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("kind", ["some", "padded", "one", "none"])
@pytest.mark.parametrize("T,k,E", CASES)
def test_sort(T, k, E, kind, dtype):
    e = entries(np.random.default_rng(T + k + E), T, k, E, kind)
    if dtype == torch.int64 and kind == "padded":
        e[0, 0] = 2 ** 32                              # would be expert 0 in 32 bits
    got = sort(torch.from_numpy(e).to(DEV, dtype), E)
    for g, r in zip(got, q4.expert_sort(e, E)):
        assert np.array_equal(g.cpu().numpy(), r)


def test_sort_of_nothing():
    _, _, offsets = sort(torch.empty(0, 4, dtype=I32, device=DEV), 7)
    assert offsets.tolist() == [0] * 8


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["some", "padded", "none"])
@pytest.mark.parametrize("T,k,E,cols", [(1, 1, 1, 1), (1, 8, 64, 4096), (2, 3, 4, 7), (17, 3, 5, 1000), (63, 6, 60, 264),
                                        (40, 9, 8, 101), (300, 2, 3, 64), (5, 4, 4, 5000), (700, 5, 9, 24)])
def test_send_return_and_gradient(T, k, E, cols, kind, dtype):
    rng = np.random.default_rng(T + cols)
    e = entries(rng, T, k, E, kind)
    _, inverse, offsets = sort(torch.from_numpy(e).to(DEV, I32), E)
    inv, off = inverse.cpu().numpy(), offsets.cpu().numpy()
    hx, x = act(rng.standard_normal((T, cols)), dtype)
    hs, ys = act(rng.standard_normal((T * k, cols)), dtype)
    w = rng.standard_normal((T, k)).astype(np.float32)
    wd = f32_dev(w)
    half = 2.0 ** (-8 if dtype == "bf16" else -24)
    size = T * k * cols * x.element_size()
    xb, db = Guarded(size), Guarded(size)
    xs, d_ys = xb.view(x.dtype, (T * k, cols)), db.view(x.dtype, (T * k, cols))
    xs.fill_(3.0)
    d_ys.fill_(3.0)
    dora.dora_expert_send(x, inverse, offsets, xs)
    x64, s64 = act_to_f64(hx), act_to_f64(hs)
    assert np.array_equal(to_f64(xs), q4.expert_send(x64, inv, off, np.full((T * k, cols), 3.0)))
    y = torch.full_like(x, float("nan"))
    for weight, host in ((wd, w), (None, None)):
        dora.dora_expert_return(ys, inverse, offsets, weight, y)
        ref = q4.expert_return(s64, inv, off, host)
        mag = q4.expert_return(np.abs(s64), inv, off, None if host is None else np.abs(host))
        check_bound("y", to_f64(y), ref, half * np.abs(ref) + 2.0 ** -23 * (k + 1) * mag)
    d_w = torch.full((T, k), float("nan"), device=DEV)
    dora.dora_expert_return_bwd(x, ys, inverse, offsets, wd, d_ys, d_w)
    d_ref, w_ref = q4.expert_return_bwd(x64, s64, inv, off, w, np.full((T * k, cols), 3.0))
    _, w_mag = q4.expert_return_bwd(np.abs(x64), np.abs(s64), inv, off, w, np.zeros((T * k, cols)))
    check_bound("d_ys", to_f64(d_ys), d_ref, (half + 2.0 ** -24) * np.abs(d_ref))
    check_bound("d_weight", to_f64(d_w), w_ref, 2.0 ** -24 * (cols + 16) * w_mag)
    torch.cuda.synchronize()
    xb.check("xs")
    db.check("d_ys")


def test_rows_of_no_expert_are_not_read():
    """NaN behind the last expert's rows and in the weights of entries that have none."""
    e = torch.tensor([[0, -1], [5, 1], [-1, -1]], dtype=I32, device=DEV)
    _, inverse, offsets = sort(e, 2)
    ys = torch.ones(6, 16, device=DEV)
    ys[2:] = float("nan")
    w = torch.tensor([[2.0, float("nan")], [float("inf"), 3.0], [float("nan")] * 2], device=DEV)
    y = torch.empty(3, 16, device=DEV)
    dora.dora_expert_return(ys, inverse, offsets, w, y)
    assert y[:, 0].tolist() == [2.0, 3.0, 0.0]
    d_ys, d_w = torch.full_like(ys, 7.0), torch.empty(3, 2, device=DEV)
    dora.dora_expert_return_bwd(y, ys, inverse, offsets, w, d_ys, d_w)
    assert d_w.tolist() == [[32.0, 0.0], [0.0, 48.0], [0.0, 0.0]]
    assert d_ys[:, 0].tolist() == [4.0, 9.0, 7.0, 7.0, 7.0, 7.0]


def test_indexes_past_the_rows_stay_inside():
    inverse = torch.tensor([[0, 2 ** 31 - 1], [-5, 1], [4, 6]], dtype=I32, device=DEV)
    for last in (6, 1000, -3):
        offsets = torch.tensor([0, last], dtype=I32, device=DEV)
        b = Guarded(6 * 8 * 4)
        xs = b.view(torch.float32, (6, 8))
        dora.dora_expert_send(torch.ones(3, 8, device=DEV), inverse, offsets, xs)
        y = torch.empty(3, 8, device=DEV)
        dora.dora_expert_return(torch.ones(6, 8, device=DEV), inverse, offsets, None, y)
        torch.cuda.synchronize()
        b.check("xs")
        assert y[:, 0].tolist() == ([0.0, 0.0, 0.0] if last < 0 else [1.0, 1.0, 1.0])


def test_unaligned_rows_take_the_same_values():
    rng = np.random.default_rng(0)
    e = entries(rng, 20, 3, 4, "padded")
    _, inverse, offsets = sort(torch.from_numpy(e).to(DEV, I32), 4)
    x = torch.randn(20, 64, device=DEV).bfloat16()
    shifted = torch.empty(20 * 64 + 1, dtype=x.dtype, device=DEV)[1:].view(20, 64)
    shifted.copy_(x)
    a, b = torch.zeros(60, 64, dtype=x.dtype, device=DEV), torch.zeros(60, 64, dtype=x.dtype, device=DEV)
    dora.dora_expert_send(x, inverse, offsets, a)
    dora.dora_expert_send(shifted, inverse, offsets, b)
    assert torch.equal(a, b)


def test_rows_past_32_bits():
    """More than 2^31 elements of sorted rows; the last tokens' against torch."""
    T, k, E, cols = 70000, 8, 16, 4096
    torch.manual_seed(2)
    expert = torch.randint(0, E, (T, k), dtype=I32, device=DEV)
    _, inverse, offsets = sort(expert, E)
    x = torch.randn(T, cols, device=DEV).to(torch.bfloat16)
    xs = torch.empty(T * k, cols, dtype=torch.bfloat16, device=DEV)
    dora.dora_expert_send(x, inverse, offsets, xs)
    some = torch.cat([torch.arange(0, T, 997), torch.arange(T - 5, T)]).to(DEV)
    at = inverse[some].long()
    assert torch.equal(xs[at], x[some][:, None].expand(-1, k, -1))
    assert int(at.max()) * cols > 2 ** 31
    w = torch.rand(T, k, device=DEV)
    y = torch.empty_like(x)
    dora.dora_expert_return(xs, inverse, offsets, w, y)
    d, dw = torch.empty_like(xs), torch.empty_like(w)
    dora.dora_expert_return_bwd(x, xs, inverse, offsets, w, d, dw)
    rows, ws, xd = xs[at].double(), w[some].double(), x[some].double()
    ref, mag = (ws[:, :, None] * rows).sum(1), (ws[:, :, None] * rows.abs()).sum(1)
    assert ((y[some].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + (1 + 2.0 ** -8) * 2 * k * 2.0 ** -24 * mag).all()
    ref = ws[:, :, None] * xd[:, None]
    assert ((d[at].double() - ref).abs() <= (2.0 ** -8 + 2.0 ** -23) * ref.abs()).all()
    ref, mag = (rows * xd[:, None]).sum(-1), (rows * xd[:, None]).abs().sum(-1)
    assert ((dw[some].double() - ref).abs() <= 2 * cols * 2.0 ** -24 * mag).all()
