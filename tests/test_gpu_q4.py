"""GPU parity of the 4-bit weight's operators with their fp64 oracle, through the C ABI.

Tolerances, each from the arithmetic:
  * the form: equal bytes (division by a power of two is exact); its values: equal bits.
  * y and dx of the products: W's values are exact in the operands; the sums are fp32
    and may round toward zero, K + 64 additions at the very most, so
    2^-23 (K + 64) sum |x| |w|, and one rounding to bf16, half a step: 2^-8 of the value.
    x W^T of few tokens takes x as two 8-bit pieces: within 2^-14 of a scale unit, of which a
    group's largest magnitude is more than 224, so 2^-21 of that for each of its 32 elements.
"""
import numpy as np
import pytest
import torch

import parameter_efficient_fine_gb300 as dora
from oracle import q4_oracle as q4
from parameter_efficient_fine_gb300 import workloads as wl

from gpu_util import DEV, act_to_dev, act_to_f64, assert_no_device_error, check_bound, to_f64
from test_gpu_guards import Guarded

pytestmark = pytest.mark.gpu

U8 = torch.uint8
BF16 = torch.bfloat16


def u8_dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def act(a, dtype="bf16"):
    """float64 values rounded to the activation type: the host bits and the device tensor."""
    h = wl.f32_to_bf16_bits(a.astype(np.float32)) if dtype == "bf16" else a.astype(np.float32)
    return h, act_to_dev(h)


def spread(rng, shape):
    """Normal values over many binades, a few loud columns, a row and a group of zeros."""
    x = rng.standard_normal(shape) * 2.0 ** rng.integers(-12, 12, size=(shape[0], 1))
    x[:, :: 37] *= 50.0
    x[shape[0] // 2] = 0.0
    x[0, :32] = 0.0
    return x


def store(x):
    q = torch.full((*x.shape[:-1], x.shape[-1] // 2), 0x5a, dtype=U8, device=DEV)
    sc = torch.full((*x.shape[:-1], x.shape[-1] // 32), 0x5a, dtype=U8, device=DEV)
    dora.dora_q4_store(x, q, sc)
    return q, sc


# ---- store and load ---------------------------------------------------------
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 32), (1, 4096), (3, 96), (5, 160), (33, 2080), (300, 992), (2000, 416)])
def test_store_and_load(rows, cols, dtype):
    h, x = act(spread(np.random.default_rng(rows * 7 + cols), (rows, cols)), dtype)
    q, sc = store(x)
    q_ref, sc_ref = q4.q4_encode(act_to_f64(h))
    assert np.array_equal(sc.cpu().numpy(), sc_ref)
    assert np.array_equal(q.cpu().numpy(), q_ref)
    back = torch.full_like(x, float("nan"))
    dora.dora_q4_load(q, sc, back)
    assert np.array_equal(to_f64(back), q4.q4_decode(q_ref, sc_ref))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_store_borders_not_finite_and_extreme(dtype):
    x = np.ones((9, 64))
    x[0, 3], x[1, 40], x[2, :] = np.nan, np.inf, -np.inf
    x[3, :] = 3.38e38                              # the largest binade
    x[4, :] = 1e-38
    x[5, :] = np.float64(np.finfo(np.float32).tiny)
    x[6, :8] = [6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]    # every tie
    x[6, 32:40] = [-6.0, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5.0]
    x[7, ::2], x[7, 1::2] = 6.0, 6.03125
    x[8, :] = -0.0
    h, d = act(x, dtype)
    q, sc = store(d)
    q_ref, sc_ref = q4.q4_encode(act_to_f64(h))
    assert np.array_equal(sc.cpu().numpy(), sc_ref) and np.array_equal(q.cpu().numpy(), q_ref)
    back = torch.empty_like(d)
    dora.dora_q4_load(q, sc, back)
    with np.errstate(over="ignore", invalid="ignore"):
        ref = q4.q4_decode(q_ref, sc_ref).astype(np.float32).astype(np.float64)
    assert np.array_equal(to_f64(back), ref, equal_nan=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_every_code_and_scale_loads_to_its_value(dtype):
    q = torch.arange(256, dtype=torch.int32, device=DEV).to(U8).repeat(256, 1)
    sc = torch.arange(256, dtype=torch.int32, device=DEV).to(U8)[:, None].repeat(1, 16).contiguous()
    x = torch.empty(256, 512, device=DEV, dtype=BF16 if dtype == "bf16" else torch.float32)
    dora.dora_q4_load(q, sc, x)
    with np.errstate(over="ignore", invalid="ignore"):
        ref = q4.q4_decode(q.cpu().numpy(), sc.cpu().numpy()).astype(np.float32).astype(np.float64)
    assert np.array_equal(to_f64(x), ref, equal_nan=True)


def test_store_and_load_write_nothing_else():
    rows, cols = 37, 160
    _, x = act(spread(np.random.default_rng(5), (rows, cols)))
    qb, sb, xb = Guarded(rows * cols // 2), Guarded(rows * cols // 32), Guarded(rows * cols * 2)
    q, sc, back = qb.view(U8, (rows, cols // 2)), sb.view(U8, (rows, cols // 32)), xb.view(BF16, (rows, cols))
    dora.dora_q4_store(x, q, sc)
    dora.dora_q4_load(q, sc, back)
    torch.cuda.synchronize()
    for b, n in ((qb, "q"), (sb, "scale"), (xb, "x")):
        b.check(n)


# ---- products ---------------------------------------------------------------
def weight(rng, out, inp, experts=None):
    """Bytes of a weight (or a stack): normal values, groups of very different scale, a group of zeros."""
    n = experts or 1
    W = rng.standard_normal((n * out, inp)) / np.sqrt(inp)
    W *= np.repeat(2.0 ** rng.integers(-3, 4, (n * out, inp // 32)), 32, axis=1)
    W[0, :32] = 0.0
    q, s = q4.q4_encode(W)
    if experts:
        return q.reshape(n, out, -1), s.reshape(n, out, -1)
    return q, s


def sum_bound(x, wq, ws, K, t, offsets=None):
    f = q4.matmul_q4_t if t else q4.matmul_q4
    wabs, xabs = wq & 0x77, np.abs(x)
    bound = 2.0 ** -23 * (K + 64) * f(xabs, wabs, ws, offsets)
    if not t:
        top = xabs.reshape(len(x), -1, 32).max(-1).repeat(32, -1)
        bound += 2.0 ** -21 * f(top, wabs, ws, offsets)
    return bound


def product(x, wq, ws, y, t, offsets=None):
    """The call with a guarded workspace of just the size that it names."""
    out, inp = wq.shape[-2], 2 * wq.shape[-1]
    size = dora.dora_matmul_q4_t_workspace if t else dora.dora_matmul_q4_workspace
    n = size(x.shape[0], out, inp, 1 if offsets is None else wq.shape[0])
    b = Guarded(n)
    (dora.dora_matmul_q4_t if t else dora.dora_matmul_q4)(x, wq, ws, y, offsets, b.view(U8, (n,)))
    b.check("workspace")


def run(x, wq, ws, t, offsets=None, fill=float("nan")):
    n = 2 * wq.shape[-1] if t else wq.shape[-2]
    y = torch.full((x.shape[0], n), fill, dtype=BF16, device=DEV)
    product(x, wq, ws, y, t, offsets)
    return y


def check_product(x, h, wq, ws, t, offsets=None):
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device=DEV)
    y = to_f64(run(x, u8_dev(wq), u8_dev(ws), t, off))
    v = act_to_f64(h)
    ref = (q4.matmul_q4_t if t else q4.matmul_q4)(v, wq, ws, offsets)
    sums = sum_bound(v, wq, ws, v.shape[1], t, offsets)
    left = np.isnan(ref)
    assert np.array_equal(np.isnan(y), left)
    check_bound("product", y[~left], ref[~left], ((1 + 2.0 ** -8) * sums + 2.0 ** -8 * np.abs(ref) + 1e-37)[~left])
    assert_no_device_error()


@pytest.mark.parametrize("t", [False, True], ids=["xWt", "dyW"])
@pytest.mark.parametrize("T,out,inp", [
    (1, 16, 32), (1, 512, 512), (1, 1040, 2080), (2, 272, 1120), (3, 4096, 256), (7, 128, 128), (8, 256, 4096),
    (9, 48, 160), (16, 400, 640), (17, 256, 256), (31, 528, 992), (33, 64, 96), (40, 2048, 512), (64, 272, 384), (65, 272, 544),
    (100, 1040, 2080), (100, 400, 1152), (128, 4096, 128), (129, 256, 1024), (200, 144, 8192), (257, 512, 160), (70, 4096, 160), (150, 160, 4096), (300, 784, 288), (1000, 272, 736)])
def test_products(T, out, inp, t):
    rng = np.random.default_rng(T * 31 + out + inp)
    wq, ws = weight(rng, out, inp)
    h, x = act(spread(rng, (T, out if t else inp)))
    check_product(x, h, wq, ws, t)


@pytest.mark.parametrize("T,out,inp", [(1, 272, 4608), (5, 144, 8320), (40, 272, 4608), (64, 528, 2560)])
def test_parts_of_k_that_start_anywhere(T, out, inp):
    """Few tokens: CTAs whose first block of k is no multiple of four, and rows of scales
    that are no multiple of 16 bytes."""
    rng = np.random.default_rng(T + inp)
    wq, ws = weight(rng, out, inp)
    h, x = act(spread(rng, (T, inp)))
    check_product(x, h, wq, ws, False)


@pytest.mark.parametrize("t", [False, True], ids=["xWt", "dyW"])
def test_tiles_of_every_width_in_turn(t):
    """More tiles than the device holds pairs of CTAs, each a few blocks of k that the
    conversion groups do not divide, their tokens from one to a full tile."""
    rng = np.random.default_rng(11)
    offsets = np.cumsum([0, 1, 33, 64, 65, 97, 129, 160, 0, 191, 224, 256]).tolist()
    out, inp = (544, 4096) if t else (4096, 544)
    wq, ws = weight(rng, out, inp, len(offsets) - 1)
    h, x = act(spread(rng, (offsets[-1], out if t else inp)))
    check_product(x, h, wq, ws, t, offsets)


EXPERTS = [
    ([0, 1], 64, 96), ([0, 0, 3, 3, 4, 4], 272, 544), ([0, 5, 5, 40, 41, 300], 144, 160), ([0] * 40 + [2, 2, 9, 9], 256, 384),
    ([0, 700, 701, 701], 400, 256), ([0, 30, 30, 100, 130], 272, 640), ([0, 1, 300, 301], 144, 384), ([0, 8, 16, 24, 32, 40, 48, 56, 64], 512, 1024), (list(range(0, 78, 2)), 48, 2080),
    # few tokens, some experts with more than a tile holds
    ([0, 0, 1, 3, 43, 46, 46, 63, 72], 272, 384), ([0, 30, 31, 33, 36, 38], 144, 1024), ([0, 0, 0, 0, 150, 160], 272, 544),
    ([0, 0, 20, 20, 20, 20], 528, 4096)]


@pytest.mark.parametrize("t", [False, True], ids=["xWt", "dyW"])
@pytest.mark.parametrize("behind", [0, 5])
@pytest.mark.parametrize("offsets,out,inp", EXPERTS, ids=[str(i) for i in range(len(EXPERTS))])
def test_experts(offsets, out, inp, behind, t):
    rng = np.random.default_rng(len(offsets) + out + behind)
    wq, ws = weight(rng, out, inp, len(offsets) - 1)
    h, x = act(spread(rng, (offsets[-1] + behind, out if t else inp)))
    check_product(x, h, wq, ws, t, offsets)


@pytest.mark.parametrize("t", [False, True], ids=["xWt", "dyW"])
@pytest.mark.parametrize("offsets", [[0, 0, 0, 0], [3, 3, 3, 3], [-7, 2, 1, 100], [5, 2, 4, 4]])
def test_offsets_past_the_rows_stay_inside(offsets, t):
    rng = np.random.default_rng(9)
    T, out, inp = 6, 144, 160
    wq, ws = weight(rng, out, inp, 3)
    n = inp if t else out
    _, x = act(spread(rng, (T, out if t else inp)))
    yb = Guarded(T * n * 2)
    y = yb.view(BF16, (T, n))
    product(x, u8_dev(wq), u8_dev(ws), y, t, torch.tensor(offsets, dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    yb.check("y")
    assert_no_device_error()


@pytest.mark.parametrize("t", [False, True], ids=["xWt", "dyW"])
@pytest.mark.parametrize("T", [1, 20, 70, 300])
def test_every_code_and_scale_in_a_product(T, t):
    """One weight of every code at scales from the smallest to the largest that a
    product of this size leaves finite; row by row so that each value is seen alone."""
    scales = [0, 1, 2, 3, 60, 126, 127, 128, 129, 130, 200, 250, 252]
    out, inp = 16 * len(scales), 128
    code = np.arange(out)[:, None] + np.arange(inp)[None] // 2
    wq = ((code[:, 0::2] % 16) | ((code[:, 1::2] + 5) % 16) << 4).astype(np.uint8)
    ws = np.repeat(np.array(scales, np.uint8), 16)[:, None].repeat(inp // 32, 1)
    W = q4.q4_decode(wq, ws)
    n, k = (inp, out) if t else (out, inp)
    x = np.zeros((T, k))
    x[np.arange(T), (np.arange(T) * 7) % k] = 1.0       # picks a row or a column of W
    _, d = act(x)
    y = to_f64(run(d, u8_dev(wq), u8_dev(ws), t))
    ref = x @ (W if t else W.T)
    # a result below the smallest normal number may be flushed in a product
    tiny = np.abs(ref) < 2.0 ** -126
    assert np.array_equal(y[~tiny], ref[~tiny])
    assert np.all(np.abs(y[tiny]) < 2.0 ** -126)


@pytest.mark.parametrize("t", [False, True], ids=["xWt", "dyW"])
@pytest.mark.parametrize("T", [1, 12, 40, 300])
def test_not_finite(T, t):
    """A NaN group of W reaches every result that it is part of and no other; a row of
    x that is not finite no other row."""
    rng = np.random.default_rng(T)
    out, inp = 272, 320
    wq, ws = weight(rng, out, inp)
    ws[5, 3] = 255
    n, k = (inp, out) if t else (out, inp)
    h, _ = act(spread(rng, (T, k)))
    x = act_to_dev(h)
    bad = T // 2 if T > 1 else None
    if bad is not None:
        x[bad, 7], x[bad - 1, 9] = float("inf"), float("nan")
    y = to_f64(run(x, u8_dev(wq), u8_dev(ws), t))
    hit = np.zeros((T, n), bool)
    hit[:, slice(96, 128) if t else 5] = True
    if bad is not None:
        hit[[bad - 1, bad]] = True
        assert not np.isfinite(y[bad]).any() or not t      # an infinity may meet a zero or not: NaN or infinite
        assert np.isnan(y[bad - 1]).all()
    assert np.isnan(y[:, slice(96, 128) if t else 5]).all()
    assert np.isfinite(y[~hit]).all()


@pytest.mark.parametrize("t", [False, True], ids=["xWt", "dyW"])
@pytest.mark.parametrize("T", [1, 30, 150])
def test_same_bits_again_and_nothing_else_written(T, t):
    rng = np.random.default_rng(T)
    out, inp = 1040, 1120
    wq, ws = (u8_dev(v) for v in weight(rng, out, inp))
    _, x = act(spread(rng, (T, out if t else inp)))
    n = inp if t else out
    first = run(x, wq, ws, t)
    for _ in range(3):
        yb = Guarded(T * n * 2)
        y = yb.view(BF16, (T, n))
        product(x, wq, ws, y, t)
        torch.cuda.synchronize()
        yb.check("y")
        assert torch.equal(y.view(torch.int16), first.view(torch.int16))
    assert_no_device_error()


@pytest.mark.parametrize("T,out,inp,t", [(600, 1024, 8192, False), (129, 4096, 8192, False), (1000, 4096, 4096, True),
                                         (600, 4096, 1024, True), (5, 1040, 8192, False), (50, 1040, 8224, False)])
def test_many_calls_give_the_same_bits(T, out, inp, t):
    """Long rings of copies, conversions and products, over and over with other work
    between: a slot that was given back too early would show as another result."""
    torch.manual_seed(T)
    wq = torch.randint(0, 256, (out, inp // 2), dtype=U8, device=DEV)
    ws = torch.randint(115, 125, (out, inp // 32), dtype=U8, device=DEV)
    x = torch.randn(T, out if t else inp, device=DEV).to(BF16)
    big = torch.empty(200 << 20, dtype=U8, device=DEV)
    first = run(x, wq, ws, t)
    for i in range(60):
        if i % 3 == 0:
            big.fill_(i)                                 # out of L2
        assert torch.equal(run(x, wq, ws, t), first), i
    assert_no_device_error()


@pytest.mark.parametrize("t", [False, True], ids=["xWt", "dyW"])
@pytest.mark.parametrize("T", [1, 24, 600])
def test_error_of_a_row_is_what_rounding_leaves(T, t):
    """Sums held in few bits would show here and not in the element-wise bound: the
    norm of a row's error is what rounding to bf16 leaves, 2^-8 / sqrt(3) of the
    row's norm at most, and 2^-9 or less over random mantissas."""
    rng = np.random.default_rng(3)
    out, inp = 1024, 8192
    if t:
        out, inp = inp, out
    wq, ws = weight(rng, out, inp)
    h, x = act(rng.standard_normal((T, out if t else inp)))
    y = to_f64(run(x, u8_dev(wq), u8_dev(ws), t))
    ref = (q4.matmul_q4_t if t else q4.matmul_q4)(act_to_f64(h), wq, ws)
    err = np.linalg.norm(y - ref, axis=1) / np.linalg.norm(ref, axis=1)
    assert err.max() <= 1.1 * 2.0 ** -9, err.max()


@pytest.mark.parametrize("t", [False, True], ids=["xWt", "dyW"])
@pytest.mark.parametrize("T", [7, 4700])
def test_a_stack_past_32_bits(T, t):
    """More than 2^32 values, 2^31 bytes, the tokens at the first and the last expert: a
    row's error as above."""
    E, n = 66, 8192
    torch.manual_seed(T)
    wq = torch.randint(0, 256, (E, n, n // 2), dtype=U8, device=DEV)
    ws = torch.randint(110, 118, (E, n, n // 32), dtype=U8, device=DEV)
    offsets = torch.full((E + 1,), 3, dtype=torch.int32, device=DEV)
    offsets[0], offsets[E] = 0, T
    x = torch.randn(T, n, device=DEV).to(BF16)
    y = run(x, wq, ws, t, offsets)
    assert_no_device_error()
    W = torch.empty(n, n, device=DEV)
    for e, rows in ((0, slice(0, 3)), (E - 1, slice(3, None, 1 + T // 50))):
        dora.dora_q4_load(wq[e], ws[e], W)
        ref = x[rows].double() @ (W if t else W.t()).double()
        err = (y[rows].double() - ref).norm(dim=1) / ref.norm(dim=1)
        assert err.max() <= 1.1 * 2.0 ** -9, (e, err.max())


def test_a_result_past_32_bits():
    T, out, inp = 70000, 32768, 64
    torch.manual_seed(1)
    wq = torch.randint(0, 256, (out, inp // 2), dtype=U8, device=DEV)
    ws = torch.randint(110, 118, (out, inp // 32), dtype=U8, device=DEV)
    x = torch.randn(T, inp, device=DEV).to(BF16)
    y = run(x, wq, ws, False)
    assert_no_device_error()
    W = torch.empty(out, inp, device=DEV)
    dora.dora_q4_load(wq, ws, W)
    rows = slice(0, None, 1021)
    ref = x[rows].double() @ W.t().double()
    err = (y[rows].double() - ref).norm(dim=1) / ref.norm(dim=1)
    assert err.max() <= 1.1 * 2.0 ** -9, err.max()
    assert not y.isnan().any()
