"""x enters the products with a 4-bit weight as it is, however many tokens there are.

A row of W with one value that is not zero picks a column of x: every other product is
zero, so y is that column's value times W's, rounded once to bf16 (half a step, so the
same bits as the 64-bit product rounded), whatever else the row of x holds.
"""
import numpy as np
import pytest
import torch

from oracle import q4_oracle as q4
from parameter_efficient_fine_gb300 import ops, workloads as wl

from gpu_util import DEV, act_to_dev, act_to_f64, assert_no_device_error, check_bound, to_f64
from test_gpu_q4 import BF16, run, u8_dev, weight

pytestmark = pytest.mark.gpu

TOKENS = [1, 3, 8, 9, 16, 17, 32, 40, 64, 65, 200]       # every kernel and tile, and both sides of their limits
WIDTHS = [384, 416, 2080]                                # rows of whole blocks of 128, and not


def bits(v):
    """float64 values rounded to bf16, as bits."""
    return wl.f32_to_bf16_bits(v.astype(np.float32))


def picks(rng, out, inp, byte=127):
    """A weight whose row f has one value that is not zero, and (column, value) of each."""
    col, code = rng.integers(0, inp, out), rng.integers(1, 8, out) + 8 * rng.integers(0, 2, out)
    c = np.zeros((out, inp), np.uint8)
    c[np.arange(out), col] = code
    wq, ws = c[:, 0::2] | c[:, 1::2] << 4, np.full((out, inp // 32), byte, np.uint8)
    return wq, ws, col, q4.e2m1_table()[code] * 2.0 ** (byte - 127)


def same_values(got, want):
    """Equal, but that a result below the smallest normal number may be flushed."""
    tiny = np.abs(want) < 2.0 ** -126
    assert np.array_equal(got[~tiny], want[~tiny])
    assert np.all(np.abs(got[tiny]) <= 2.0 ** -126)


def rounded(v):
    """float64 values as the bf16 that they round to, widened again."""
    return act_to_f64(bits(v))


@pytest.mark.parametrize("inp", WIDTHS)
@pytest.mark.parametrize("T", TOKENS)
@pytest.mark.parametrize("least", [-8, -14, -17, -24, -40, -100])
def test_a_column_comes_out_as_it_is(T, inp, least):
    """Values of any mantissa from 2^least to 1, neighbours of very different size."""
    rng = np.random.default_rng(T * 7 + inp - least)
    wq, ws, col, w = picks(rng, 528, inp)
    x = act_to_f64(bits(rng.choice([-1.0, 1.0], (T, inp)) * 2.0 ** rng.uniform(least, 0, (T, inp))))
    y = to_f64(run(act_to_dev(bits(x)), u8_dev(wq), u8_dev(ws), False))
    same_values(y, rounded(x[:, col] * w))
    assert_no_device_error()


@pytest.mark.parametrize("inp", WIDTHS)
@pytest.mark.parametrize("T", TOKENS)
def test_every_finite_value_among_any_others(T, inp):
    rng = np.random.default_rng(T + inp)
    wq, ws, col, w = picks(rng, 528, inp)
    pattern = rng.integers(0, 1 << 16, (T, inp)).astype(np.uint16)
    pattern[(pattern & 0x7f80) == 0x7f80] = 0
    x = act_to_f64(pattern)
    y = to_f64(run(act_to_dev(pattern), u8_dev(wq), u8_dev(ws), False))
    with np.errstate(over="ignore"):
        same_values(y, rounded(x[:, col] * w))
    assert_no_device_error()


@pytest.mark.parametrize("inp", [384, 416])
@pytest.mark.parametrize("T", TOKENS)
@pytest.mark.parametrize("top", [-126, -118, -110, -105])
def test_small_groups_beside_a_large_scale(T, inp, top):
    """Groups whose largest magnitude is near the smallest number, times a W that brings the
    result back: nothing of x is lost below."""
    rng = np.random.default_rng(T + top + inp)
    wq, ws, col, w = picks(rng, 272, inp, byte=227)
    # whole numbers of 2^-133, the smallest bf16
    k = rng.integers(-(1 << 7), 1 << 7, (T, inp)) * 2.0 ** rng.integers(0, top + 127, (T, inp))
    x = k * 2.0 ** -133
    x = act_to_f64(bits(x))
    y = to_f64(run(act_to_dev(bits(x)), u8_dev(wq), u8_dev(ws), False))
    same_values(y, rounded(x[:, col] * w))


@pytest.mark.parametrize("loud", [1e3, 1e5, 1e6, 1e12, 1e30])
@pytest.mark.parametrize("T,inp", [(1, 2048), (5, 2080), (8, 2048), (12, 2048), (30, 2080), (64, 2048), (64, 2080), (100, 2048)])
def test_loud_columns_beside_zeros_of_the_weight(T, inp, loud):
    """Sums: columns that are far louder meet zeros of W, so the result is the others' alone."""
    rng = np.random.default_rng(T + inp)
    wq, ws = weight(rng, 272, inp)
    x = rng.standard_normal((T, inp))
    cols = np.arange(0, inp, 96) + 6
    x[:, cols] *= loud
    wq[:, cols // 2] &= 0xf0                           # even columns lie in the low half
    h = bits(x)
    v = act_to_f64(h)
    y = to_f64(run(act_to_dev(h), u8_dev(wq), u8_dev(ws), False))
    ref = q4.matmul_q4(v, wq, ws)
    sums = 2.0 ** -23 * (inp + 64) * q4.matmul_q4(np.abs(v), wq & 0x77, ws)
    check_bound("y", y, ref, (1 + 2.0 ** -8) * sums + 2.0 ** -8 * np.abs(ref))


@pytest.mark.parametrize("t", [False, True], ids=["xWt", "dyW"])
@pytest.mark.parametrize("inp", [384, 416])
@pytest.mark.parametrize("T", TOKENS)
def test_infinities_are_added_as_the_formula_says(T, inp, t):
    """inf times a value is inf of that sign, times zero NaN; two of different signs NaN."""
    rng = np.random.default_rng(T + inp)
    wq, ws = weight(rng, 272, inp)
    x = rng.standard_normal((T, 272 if t else inp))
    x[0, 5] = np.inf
    if T > 2:
        x[1, [7, 70]] = np.inf, -np.inf
        x[T - 1, 33] = -np.inf
    h = bits(x)
    y = to_f64(run(act_to_dev(h), u8_dev(wq), u8_dev(ws), t))
    v, W = act_to_f64(h), q4.q4_decode(wq, ws)
    with np.errstate(invalid="ignore"):
        ref = sum(v[:, k, None] * (W if t else W.T)[k][None] for k in range(v.shape[1]))
    bad = ~np.isfinite(ref)
    assert np.array_equal(y[bad], ref[bad], equal_nan=True)
    assert np.isfinite(y[~bad]).all() and (~bad).any() == (T > 3)
    assert_no_device_error()


@pytest.mark.parametrize("inp", [384, 416])
@pytest.mark.parametrize("T", TOKENS)
def test_a_nan_reaches_its_own_row_and_no_other(T, inp):
    rng = np.random.default_rng(T + inp)
    wq, ws = weight(rng, 272, inp)
    x = rng.standard_normal((T, inp))
    x[T // 2, 40] = np.nan
    y = to_f64(run(act_to_dev(bits(x)), u8_dev(wq), u8_dev(ws), False))
    rest = np.arange(T) != T // 2
    assert np.isnan(y[T // 2]).all() and np.isfinite(y[rest]).all()


EXPERTS = [[0, 3, 3, 8, 9], [0, 5, 30, 31, 60], [0, 64, 100, 100, 180], [0, 0, 70, 71, 200], [0, 200, 300, 400, 700]]


@pytest.mark.parametrize("inp", [384, 416])
@pytest.mark.parametrize("offsets", EXPERTS, ids=[str(i) for i in range(len(EXPERTS))])
def test_columns_of_experts_come_out_as_they_are(offsets, inp):
    rng = np.random.default_rng(offsets[-1] + inp)
    E, T, out = len(offsets) - 1, offsets[-1], 272
    wq, ws, col, w = picks(rng, E * out, inp)
    x = act_to_f64(bits(rng.choice([-1.0, 1.0], (T, inp)) * 2.0 ** rng.uniform(-40, 0, (T, inp))))
    off = torch.tensor(offsets, dtype=torch.int32, device=DEV)
    y = to_f64(run(act_to_dev(bits(x)), u8_dev(wq.reshape(E, out, -1)), u8_dev(ws.reshape(E, out, -1)), False, off))
    for e in range(E):
        rows, f = slice(offsets[e], offsets[e + 1]), slice(e * out, (e + 1) * out)
        same_values(y[rows], rounded(x[rows][:, col[f]] * w[f]))


@pytest.mark.parametrize("T,experts", [(1, 0), (8, 0), (9, 0), (16, 0), (20, 0), (32, 0), (33, 0), (200, 0), (6, 3), (20, 3), (40, 3), (200, 3)])
def test_a_weight_that_starts_16_bytes_into_its_memory(T, experts):
    """16-byte alignment is what the products ask for; rows of whole blocks of 128 take
    another way into shared memory where W is on 32 bytes."""
    rng = np.random.default_rng(T + experts)
    E, out, inp = max(experts, 1), 272, 512
    wq, ws, col, w = picks(rng, E * out, inp)
    x = act_to_f64(bits(rng.choice([-1.0, 1.0], (T, inp)) * 2.0 ** rng.uniform(-20, 0, (T, inp))))
    shape = (E, out) if experts else (out,)
    offsets = np.linspace(0, T, E + 1).astype(int)
    off = torch.tensor(offsets, dtype=torch.int32, device=DEV) if experts else None
    d = act_to_dev(bits(x))
    plain = u8_dev(wq).reshape(*shape, -1)
    raw = torch.zeros(wq.size + 32, dtype=torch.uint8, device=DEV)
    moved = raw[16:16 + wq.size].view(plain.shape)
    moved.copy_(plain)
    assert moved.data_ptr() % 32 == 16
    scales = u8_dev(ws).reshape(*shape, -1)
    y = to_f64(run(d, moved, scales, False, off))
    for e in range(E):
        rows, f = slice(offsets[e], offsets[e + 1]), slice(e * out, (e + 1) * out)
        same_values(y[rows], rounded(x[rows][:, col[f]] * w[f]))
    # sums: the same within what sums of either order leave
    wq, ws = weight(rng, out, inp, experts or None)
    h = bits(rng.standard_normal((T, inp)))
    moved.copy_(u8_dev(wq))
    y = to_f64(run(act_to_dev(h), moved, u8_dev(ws), False, off))
    v = act_to_f64(h)
    offs = offsets.tolist() if experts else None
    ref = q4.matmul_q4(v, wq, ws, offs)
    sums = 2.0 ** -23 * (inp + 64) * q4.matmul_q4(np.abs(v), wq & 0x77, ws, offs)
    check_bound("y", y, ref, (1 + 2.0 ** -8) * sums + 2.0 ** -8 * np.abs(ref))
    assert_no_device_error()


@pytest.mark.parametrize("T", [2, 8, 20])
def test_long_rows(T):
    """More blocks of k a CTA than it has bits for: 262, groups that no pieces hold among them."""
    rng = np.random.default_rng(T)
    inp = 128 * 2100
    x = rng.standard_normal((T, inp))
    odd = rng.choice(inp // 32, 60, replace=False)
    odd[:4] = 0, 1024, 2100 * 4 - 1, 1028             # the first and the last; blocks that share a bit
    for t in range(T):
        x[t, 32 * odd + rng.integers(0, 32, 60)] *= 2.0 ** rng.integers(20, 90, 60)
    x = act_to_f64(bits(x))
    wq, ws, col, w = picks(rng, 144, inp)
    wq[:] = 0
    col[:120] = 32 * odd[rng.integers(0, 60, 120)] + rng.integers(0, 32, 120)
    code = rng.integers(1, 8, 144)
    wq[np.arange(144), col // 2] = code << (4 * (col % 2))
    w = q4.e2m1_table()[code]
    y = to_f64(run(act_to_dev(bits(x)), u8_dev(wq), u8_dev(ws), False))
    same_values(y, rounded(x[:, col] * w))
    assert_no_device_error()


def loud(seed, T, inp):
    """Hidden states with loud columns, and a few values that are far louder."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(T, inp, generator=gen, device=DEV)
    x *= torch.where(torch.rand(inp, generator=gen, device=DEV) < 0.01, 24.0, 1.0)
    return torch.where(torch.rand(T, inp, generator=gen, device=DEV) < 2e-5, x * 2.0 ** 50, x).to(BF16)


@pytest.mark.parametrize("T,inp", [(1, 4096), (8, 4096), (8, 4128), (13, 4096), (30, 4096)])
def test_replayed_calls_and_calls_at_once(T, inp):
    """The same bits from a captured call with other inputs, and from calls on several streams,
    each with its own workspace."""
    rng = np.random.default_rng(T)
    wq, ws = (u8_dev(v) for v in weight(rng, 1040, inp))
    xs = [loud(i, T, inp) for i in range(4)]
    want = [ops.matmul_q4(x, wq, ws) for x in xs]
    torch.cuda.synchronize()
    x = xs[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = ops.matmul_q4(x, wq, ws)
    for i in (1, 2, 3, 0):
        x.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[i])
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(10):
        got = []
        for a, st in zip(xs, streams):
            with torch.cuda.stream(st):
                got.append(ops.matmul_q4(a, wq, ws))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert_no_device_error()


@pytest.mark.parametrize("T", [1, 8, 12, 30])
def test_a_chain_of_calls_reads_what_the_one_before_wrote(T):
    """Launches that overlap the end of the one before: x of each call is the result of the last,
    read once more from memory for its finer pieces."""
    rng = np.random.default_rng(T)
    wq, ws = (u8_dev(v) for v in weight(rng, 1024, 1024))
    big = loud(9, T, 1024)
    want = None
    for _ in range(20):
        y = big
        for i in range(8):
            y = ops.matmul_q4(y, wq, ws)
            if want is None:
                torch.cuda.synchronize()
        want = y if want is None else want
        assert torch.equal(y, want)
