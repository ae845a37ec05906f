"""GPU parity of the 8-bit operators with their fp64 oracle, through the C ABI.

Tolerances, each from the arithmetic:
  * the 8-bit form: equal bytes (division by a power of two is exact, v's two
    fp32 roundings are part of its definition); its values: equal bits.
  * y, d_base, d_lora of the compose: bitwise dora_compose_fwd's and _bwd's.
  * d_mag: fp32 sums of at most T + 16 terms,
        |err| <= 2^-24 (T + 16) sum_t |dy| |v| / n.
  * dA: exact products, sums in fp32 that may round toward zero: a chain of
    T + 64 additions at the very most, so |err| <= 2^-23 (T + 64) sum |dxa| |x|;
    and, since the sums are cut into short chains, ||err||_F <= 1e-6 ||ref||_F
    (the error of a random sum grows with the root of its length: chains of 16
    matrix instructions and 60 partial sums stay below 16 2^-24).
  * y and dx of the products: the same bound with K additions, and one
    rounding to bf16, 2^-9 of the value (2^-8 with the bound's own slack).
"""
import numpy as np
import pytest
import torch

import parameter_efficient_fine_gb300 as dora
from oracle import q8_oracle as q8
from parameter_efficient_fine_gb300 import workloads as wl

from gpu_util import DEV, act_to_dev, act_to_f64, assert_no_device_error, check_bound, f32_dev, run_bwd, run_fwd, to_f64
from test_gpu_guards import Guarded

pytestmark = pytest.mark.gpu

U8 = torch.uint8


def form(rows, cols, block_rows=1):
    """Empty 8-bit form, filled with a byte that no result can keep by chance."""
    return (torch.full((rows, cols), 0x5a, dtype=U8, device=DEV),
            torch.full((-(-rows // block_rows), -(-cols // 128)), 0x5a, dtype=U8, device=DEV))


def u8_dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def workspace(n):
    return torch.empty(max(n, 1), dtype=U8, device=DEV)


def act(a, dtype):
    """float64 values rounded to the activation type: the host bits and the device tensor."""
    h = wl.f32_to_bf16_bits(a.astype(np.float32)) if dtype == "bf16" else a.astype(np.float32)
    return h, act_to_dev(h)


def store(x, block_rows=1):
    q, sc = form(*x.shape, block_rows)
    dora.dora_q8_store(x, block_rows, q, sc)
    return q, sc


def spread(rng, shape):
    """Normal values over many binades, a few loud columns, a row and a block of zeros."""
    x = rng.standard_normal(shape) * 2.0 ** rng.integers(-12, 12, size=(shape[0], 1))
    x[:, :: 37] *= 50.0
    x[shape[0] // 2] = 0.0
    x[0, :128] = 0.0
    return x


# ---- store and load ---------------------------------------------------------
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols,block_rows", [
    (1, 1, 1), (1, 128, 1), (1, 4096, 1), (3, 127, 1), (5, 129, 1), (7, 1003, 1), (33, 264, 1), (300, 1000, 1),
    (2000, 392, 1), (1, 1, 128), (128, 128, 128), (130, 264, 128), (500, 1003, 128),
])
def test_store_and_load(rows, cols, block_rows, dtype):
    h, x = act(spread(np.random.default_rng(rows * 7 + cols), (rows, cols)), dtype)
    q, sc = store(x, block_rows)
    q_ref, sc_ref = q8.q8_encode(act_to_f64(h), block_rows)
    assert np.array_equal(sc.cpu().numpy(), sc_ref)
    assert np.array_equal(q.cpu().numpy(), q_ref)
    back = torch.full_like(x, float("nan"))
    dora.dora_q8_load(q, sc, block_rows, back)
    assert np.array_equal(to_f64(back), q8.q8_decode(q_ref, sc_ref, block_rows))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cols", [256, 250])
def test_store_not_finite_and_extreme(cols, dtype):
    x = np.ones((8, cols))
    x[0, 3], x[1, 200], x[2, :] = np.nan, np.inf, -np.inf
    x[3, :] = 3.38e38                              # the largest binade
    x[4, :] = 1e-38
    x[5, :] = np.float64(np.finfo(np.float32).tiny)
    x[6, ::2], x[6, 1::2] = 448.0, 449.0 if dtype == "f32" else 452.0
    x[7, :] = -0.0
    h, d = act(x, dtype)
    q, sc = store(d)
    q_ref, sc_ref = q8.q8_encode(act_to_f64(h))
    assert np.array_equal(sc.cpu().numpy(), sc_ref) and np.array_equal(q.cpu().numpy(), q_ref)
    back = torch.empty_like(d)
    dora.dora_q8_load(q, sc, 1, back)
    ref = q8.q8_decode(q_ref, sc_ref)
    with np.errstate(over="ignore"):
        assert np.array_equal(to_f64(back), ref.astype(np.float32).astype(np.float64), equal_nan=True)


def test_every_e4m3_byte_loads_to_its_value():
    q = torch.arange(256, dtype=torch.int32, device=DEV).to(U8).repeat(245, 1)
    sc = torch.arange(10, 255, dtype=torch.int32, device=DEV).to(U8)[:, None].repeat(1, 2).contiguous()
    x = torch.empty(245, 256, device=DEV)
    dora.dora_q8_load(q, sc, 1, x)
    ref = q8.q8_decode(q.cpu().numpy(), sc.cpu().numpy())
    with np.errstate(over="ignore"):
        assert np.array_equal(x.cpu().numpy(), ref.astype(np.float32), equal_nan=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_unaligned_pointers_take_the_same_values(dtype):
    rows, cols = 9, 512
    h, x = act(spread(np.random.default_rng(1), (rows, cols)), dtype)
    q_ref, sc_ref = store(x)
    flat = torch.empty(rows * cols + 1, dtype=x.dtype, device=DEV)
    off = flat[1:].view(rows, cols)
    off.copy_(x)
    qf = torch.empty(rows * cols + 3, dtype=U8, device=DEV)
    q, sc = qf[3:].view(rows, cols), torch.empty_like(sc_ref)
    dora.dora_q8_store(off, 1, q, sc)
    assert torch.equal(q, q_ref) and torch.equal(sc, sc_ref)
    off.zero_()
    dora.dora_q8_load(q, sc, 1, off)
    back = torch.empty_like(x)
    dora.dora_q8_load(q_ref, sc_ref, 1, back)
    assert torch.equal(off, back)


def shifted(x, by):
    """x's values in rows that start `by` elements past an aligned address."""
    flat = torch.empty(x.numel() + by, dtype=x.dtype, device=DEV)
    flat[by:] = x.reshape(-1)
    return flat[by:].view(x.shape)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,out", [(1, 512), (2, 256), (3, 17), (40, 130), (70, 384), (301, 1000)])
@pytest.mark.parametrize("by", [1, 2, 5])
def test_any_alignment_gives_the_same_bits(T, out, by, dtype):
    """Every operand at its own odd address against the same values in rows of
    whole 16-byte pieces, padded with columns that the result does not read."""
    rng = np.random.default_rng(T + out)
    wide = -(-out // 128) * 128
    base, lora, dy = (act(spread(rng, (T, wide)), dtype)[1] for _ in range(3))
    for x in (base, lora, dy):
        x[:, out:] = 0                             # leaves a block's scale as it is
    g, n = f32_dev(rng.uniform(0.5, 1.5, wide)), f32_dev(rng.uniform(0.5, 2.0, wide))
    y, (q, sc) = torch.empty_like(base), form(T, wide)
    dora.dora_compose_fwd_q8(base, lora, g, 0.75, y, q, sc)
    db, dl, dm = torch.empty_like(base), torch.empty_like(base), torch.empty(wide, device=DEV)
    ws = workspace(dora.dora_compose_bwd_q8_workspace(T, wide))
    dora.dora_compose_bwd_q8(dy, q, sc, g, n, 0.75, db, dl, dm, ws)
    ref = (y, q, db, dl)

    cut = [x[:, :out].contiguous() for x in (base, lora, dy)]
    b2, l2, dy2 = (shifted(x, by + k) for k, x in enumerate(cut))
    g2, n2 = g[:out].contiguous(), n[:out].contiguous()
    y2, q2 = shifted(torch.empty_like(cut[0]), by), shifted(torch.empty(T, out, dtype=U8, device=DEV), 2 * by + 1)
    sc2 = torch.empty_like(sc)
    dora.dora_compose_fwd_q8(b2, l2, g2, 0.75, y2, q2, sc2)
    db2, dl2 = (shifted(torch.empty_like(cut[0]), by + k) for k in (2, 1))
    dm2 = torch.empty(out, device=DEV)
    ws = workspace(dora.dora_compose_bwd_q8_workspace(T, out))
    dora.dora_compose_bwd_q8(dy2, q2, sc2, g2, n2, 0.75, db2, dl2, dm2, ws)
    for a, b in zip(ref, (y2, q2, db2, dl2)):
        assert torch.equal(a[:, :out], b)
    assert torch.equal(sc, sc2)
    v = torch.from_numpy(q8.q8_decode(q2.cpu().numpy(), sc2.cpu().numpy())).to(DEV)
    size = (dy2.double().abs() * v.abs()).sum(0) / n2.double()
    exact = (dy2.double() * v).sum(0) / n2.double()
    assert ((dm2.double() - exact).abs() <= 2.0 ** -24 * (T + 16) * size).all()
    back, back2 = torch.empty_like(base), shifted(torch.empty_like(cut[0]), by + 3)
    dora.dora_q8_load(q, sc, 1, back)
    dora.dora_q8_load(q2, sc2, 1, back2)
    assert torch.equal(back[:, :out], back2)


def test_offsets_past_32_bits():
    rows, cols = 300000, 14400                     # 4.3e9 elements
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device=DEV)
    x[:1000].normal_()
    for k in range(1000, rows, 1000):
        torch.mul(x[:1000], 1.0 + k / rows, out=x[k:k + 1000])
    q, sc = store(x)
    back = torch.empty_like(x)
    dora.dora_q8_load(q, sc, 1, back)
    for at in (0, 149130, 149131, 298261, rows - 7):
        h = x[at:at + 7].double().cpu().numpy()
        q_ref, sc_ref = q8.q8_encode(h)
        assert np.array_equal(q[at:at + 7].cpu().numpy(), q_ref) and np.array_equal(sc[at:at + 7].cpu().numpy(), sc_ref)
        assert np.array_equal(to_f64(back[at:at + 7]), q8.q8_decode(q_ref, sc_ref))


# ---- compose ----------------------------------------------------------------
def _compose_inputs(T, out, dtype, seed):
    rng = np.random.default_rng(seed)
    f = {k: act(rng.standard_normal((T, out)) * a, dtype) for k, a in (("base", 1.0), ("lora", 0.2), ("dy", 1.0))}
    g = (1 + rng.uniform(-0.05, 0.05, out)).astype(np.float32)
    n = rng.uniform(0.5, 2.0, out).astype(np.float32)
    return f, g, n, float(np.float32(32.0 / np.sqrt(48)))


COMPOSE = [(1, 1), (1, 8192), (3, 127), (37, 104), (33, 1003), (300, 520), (1500, 1000), (777, 2056)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,out", COMPOSE)
def test_compose_forward(T, out, dtype):
    f, g, n, s = _compose_inputs(T, out, dtype, T + out)
    base, lora, gd = f["base"][1], f["lora"][1], f32_dev(g)
    y = torch.full_like(base, float("nan"))
    q, sc = form(T, out)
    dora.dora_compose_fwd_q8(base, lora, gd, s, y, q, sc)
    assert torch.equal(y, run_fwd(base, lora, gd, s))
    _, (q_ref, sc_ref) = q8.compose_fwd_q8(act_to_f64(f["base"][0]), act_to_f64(f["lora"][0]), g, s)
    assert np.array_equal(sc.cpu().numpy(), sc_ref) and np.array_equal(q.cpu().numpy(), q_ref)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,out", COMPOSE)
def test_compose_backward(T, out, dtype):
    f, g, n, s = _compose_inputs(T, out, dtype, T + out + 1)
    dy, gd, nd = f["dy"][1], f32_dev(g), f32_dev(n)
    q_h, sc_h = q8.q8_encode(act_to_f64(f["base"][0]) + s * act_to_f64(f["lora"][0]))
    db, dl, dm = torch.empty_like(dy), torch.empty_like(dy), torch.full((out,), float("nan"), device=DEV)
    args = (dy, u8_dev(q_h), u8_dev(sc_h), gd, nd, s, db, dl, dm)
    ws = workspace(dora.dora_compose_bwd_q8_workspace(T, out))
    dora.dora_compose_bwd_q8(*args, ws)
    db_ref, dl_ref, _ = run_bwd(dy, f["base"][1], f["lora"][1], gd, nd, s)
    assert torch.equal(db, db_ref) and torch.equal(dl, dl_ref)
    d64, v = act_to_f64(f["dy"][0]), q8.q8_decode(q_h, sc_h)
    _, _, dm_ref = q8.compose_bwd_q8(d64, q_h, sc_h, g, n, s)
    check_bound("d_mag", to_f64(dm), dm_ref, 2.0 ** -24 * (T + 16) * (np.abs(d64) * np.abs(v)).sum(0) / n + 1e-30)
    first = dm.clone()
    dora.dora_compose_bwd_q8(*args, ws.fill_(0xff))
    assert torch.equal(first, dm)


def test_compose_backward_without_tokens():
    dm = torch.full((40,), float("nan"), device=DEV)
    e = torch.empty(0, 40, device=DEV)
    g = torch.ones(40, device=DEV)
    dora.dora_compose_bwd_q8(e, torch.empty(0, 40, dtype=U8, device=DEV), torch.empty(0, 1, dtype=U8, device=DEV), g, g,
                             1.0, e, e, dm, workspace(dora.dora_compose_bwd_q8_workspace(0, 40)))
    assert torch.equal(dm, torch.zeros_like(dm))


def test_d_mag_is_the_difference_quotient():
    """y is linear in m (g = m / n), so L = <dy, y> has exact difference quotients where v
    is exact in 8 bits: small integers."""
    rng = np.random.default_rng(3)
    T, out, s = 64, 256, 0.5
    base = rng.integers(-4, 5, (T, out)).astype(np.float64)
    lora = 2.0 * rng.integers(-3, 4, (T, out))     # v an integer of at most 7: 3 bits
    dy = rng.integers(-3, 4, (T, out)).astype(np.float64)
    n, m = rng.uniform(0.5, 2.0, out), rng.uniform(0.5, 2.0, out)
    b, l, d = (act_to_dev(a.astype(np.float32)) for a in (base, lora, dy))
    q, sc = form(T, out)
    gd, nd = f32_dev(m / n), f32_dev(n)
    dora.dora_compose_fwd_q8(b, l, gd, s, torch.empty_like(b), q, sc)
    dm = torch.empty(out, device=DEV)
    dora.dora_compose_bwd_q8(d, q, sc, gd, nd, s, torch.empty_like(d), torch.empty_like(d), dm,
                             workspace(dora.dora_compose_bwd_q8_workspace(T, out)))
    loss = lambda mm: (dy * (mm / n) * (base + s * lora)).sum(0)  # noqa: E731  (per column)
    quotient = (loss(m + 0.25) - loss(m - 0.25)) / 0.5
    np.testing.assert_allclose(to_f64(dm), quotient, rtol=1e-5, atol=1e-5)


# ---- the gradient of A ------------------------------------------------------
GRAD = [(1, 16, 8), (2, 128, 16), (17, 272, 24), (64, 128, 64), (255, 512, 8), (256, 512, 16), (257, 1040, 40),
        (1000, 144, 384), (513, 2064, 136), (4100, 256, 264), (640, 528, 1024), (130, 4096, 512), (6000, 400, 72)]


def _grad_inputs(T, inp, r, seed):
    rng = np.random.default_rng(seed)
    q, sc = q8.q8_encode(spread(rng, (T, inp)).astype(np.float32))
    dxa = act_to_f64(wl.f32_to_bf16_bits(rng.standard_normal((T, r)).astype(np.float32)))
    return q, sc, dxa


def run_grad(q, sc, dxa, ws_fill=None):
    T, r = dxa.shape
    inp = q.shape[1]
    dA = torch.full((r, inp), float("nan"), device=DEV)
    ws = workspace(dora.dora_lora_grad_q8_workspace(T, inp, r))
    if ws_fill is not None:
        ws.fill_(ws_fill)
    dora.dora_lora_grad_q8(dxa, q, sc, dA, ws)
    return dA


@pytest.mark.parametrize("T,inp,r", GRAD)
def test_lora_grad(T, inp, r):
    q, sc, dxa = _grad_inputs(T, inp, r, T + inp + r)
    qd, scd, dd = u8_dev(q), u8_dev(sc), act_to_dev(wl.f32_to_bf16_bits(dxa.astype(np.float32)))
    dA = run_grad(qd, scd, dd)
    assert_no_device_error()
    ref, mag = q8.lora_grad_q8(dxa, q, sc), np.abs(dxa).T @ np.abs(q8.q8_decode(q, sc))
    got = to_f64(dA)
    check_bound("dA", got, ref, 2.0 ** -23 * (T + 64) * mag + 1e-37)
    assert np.linalg.norm(got - ref) <= 1e-6 * np.linalg.norm(ref)
    assert torch.equal(dA, run_grad(qd, scd, dd, 0xff))


@pytest.mark.parametrize("T,inp,r", [
    (20000, 144, 24), (9000, 528, 72), (2700, 4112, 200), (5000, 2064, 392), (16300, 1040, 16), (3000, 8192, 136),
])
def test_lora_grad_of_cut_runs(T, inp, r):
    """Sizes at which a CTA's run of 128 tokens begins and ends inside a tile, at
    any place of a window, and a tile has up to dozens of parts; twice the same bits."""
    rng = np.random.default_rng(T + inp + r)
    dxa = torch.from_numpy(rng.standard_normal((T, r))).to(DEV).bfloat16()
    q, sc = store(torch.from_numpy(rng.standard_normal((T, inp))).to(DEV).bfloat16())
    ws = workspace(dora.dora_lora_grad_q8_workspace(T, inp, r))
    got = [torch.full((r, inp), float("nan"), device=DEV) for _ in range(2)]
    for dA in got:
        dora.dora_lora_grad_q8(dxa, q, sc, dA, ws)
    x = torch.empty(T, inp, device=DEV)
    dora.dora_q8_load(q, sc, 1, x)
    assert_no_device_error()
    ref = dxa.double().t() @ x.double()
    size = dxa.double().abs().t() @ x.double().abs()
    err = (got[0].double() - ref).abs()
    assert (err <= 2.0 ** -23 * (T + 64) * size).all() and err.norm() <= 1e-6 * ref.norm()
    assert torch.equal(got[0], got[1])


def test_lora_grad_without_tokens():
    dA = run_grad(torch.empty(0, 144, dtype=U8, device=DEV), torch.empty(0, 2, dtype=U8, device=DEV),
                  torch.empty(0, 24, dtype=torch.bfloat16, device=DEV))
    assert torch.equal(dA, torch.zeros_like(dA))


def test_lora_grad_keeps_nan_in_its_column_and_extreme_scales():
    T, inp, r = 300, 256, 16
    q, sc, dxa = _grad_inputs(T, inp, r, 11)
    q[77, 33] = 0x7f
    sc[:, 1] = np.where(np.arange(T) % 2, 10, 20)            # tiny values: still normal floats
    dA = to_f64(run_grad(u8_dev(q), u8_dev(sc), act_to_dev(wl.f32_to_bf16_bits(dxa.astype(np.float32)))))
    assert np.isnan(dA[:, 33]).all()
    keep = np.arange(inp) != 33
    assert np.isfinite(dA[:, keep]).all()
    q[77, 33] = 0
    ref, mag = q8.lora_grad_q8(dxa, q, sc), np.abs(dxa).T @ np.abs(q8.q8_decode(q, sc))
    check_bound("dA", dA[:, keep], ref[:, keep], (2.0 ** -23 * (T + 64) * mag + 1e-37)[:, keep])
    sc[:, :] = 127 + 110                                     # values near the top of the range
    dxa *= 2.0 ** -20
    dA = to_f64(run_grad(u8_dev(q), u8_dev(sc), act_to_dev(wl.f32_to_bf16_bits(dxa.astype(np.float32)))))
    ref = q8.lora_grad_q8(dxa, q, sc)
    assert np.linalg.norm((dA - ref) / 2.0 ** 90) <= 1e-6 * np.linalg.norm(ref / 2.0 ** 90)


def test_lora_grad_is_the_difference_quotient():
    """xa = x A^T is linear in A: <dxa, x (A + h E)^T> - <dxa, x (A - h E)^T> = 2 h <dA, E>."""
    T, inp, r = 200, 144, 24
    q, sc, dxa = _grad_inputs(T, inp, r, 5)
    dA = to_f64(run_grad(u8_dev(q), u8_dev(sc), act_to_dev(wl.f32_to_bf16_bits(dxa.astype(np.float32)))))
    x = q8.q8_decode(q, sc)
    rng = np.random.default_rng(6)
    A = rng.standard_normal((r, inp))
    for _ in range(4):
        E = rng.standard_normal((r, inp))
        quotient = ((dxa * (x @ (A + 0.5 * E).T)).sum() - (dxa * (x @ (A - 0.5 * E).T)).sum())
        bound = 2.0 ** -23 * (T + 64) * ((np.abs(dxa).T @ np.abs(x)) * np.abs(E)).sum()
        assert abs(quotient - (dA * E).sum()) <= bound


# ---- the products -----------------------------------------------------------
MATMUL = [(1, 16, 16), (1, 128, 8192), (2, 4096, 272), (7, 400, 1040), (16, 144, 128), (17, 256, 512), (33, 1024, 4096),
          (64, 528, 2064), (65, 272, 384), (127, 144, 656), (128, 128, 128), (129, 400, 272), (200, 2064, 144),
          (257, 1040, 1040), (300, 520 + 8, 784), (1000, 384, 2304), (1025, 2304, 400)]


def _matmul_inputs(T, out, inp, trans, seed):
    rng = np.random.default_rng(seed)
    w = rng.standard_normal((out, inp)) * 2.0 ** rng.integers(-3, 3, size=(out, 1))
    wq, wsc = q8.q8_encode(w.astype(np.float32), 128)
    q, sc = q8.q8_encode(spread(rng, (T, out if trans else inp)).astype(np.float32))
    return q, sc, wq, wsc


def run_matmul(q, sc, wq, wsc, trans, ws_fill=None):
    out, inp = wq.shape
    T = q.shape[0]
    y = torch.full((T, inp if trans else out), float("nan"), dtype=torch.bfloat16, device=DEV)
    size, call = ((dora.dora_matmul_q8_t_workspace, dora.dora_matmul_q8_t) if trans else
                  (dora.dora_matmul_q8_workspace, dora.dora_matmul_q8))
    ws = workspace(size(T, out, inp))
    if ws_fill is not None:
        ws.fill_(ws_fill)
    call(q, sc, wq, wsc, y, ws)
    return y


def check_product(name, got, q, sc, wq, wsc, trans):
    f = q8.matmul_q8_t if trans else q8.matmul_q8
    x, w = q8.q8_decode(q, sc), q8.q8_decode(wq, wsc, 128)
    mag = np.abs(x) @ (np.abs(w) if trans else np.abs(w).T)
    check_bound(name, got, f(q, sc, wq, wsc), 2.0 ** -8 * np.abs(f(q, sc, wq, wsc)) + 2.0 ** -23 * x.shape[1] * mag + 1e-37)


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("T,out,inp", MATMUL)
def test_matmul(T, out, inp, trans):
    h = _matmul_inputs(T, out, inp, trans, T + out + inp)
    d = [u8_dev(a) for a in h]
    y = run_matmul(*d, trans)
    assert_no_device_error()
    check_product("y", to_f64(y), *h, trans)
    assert torch.equal(y, run_matmul(*d, trans, 0xff))


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("T,feat,k", [
    (2500, 2064, 272),       # odd numbers of everything; a last feature tile of 16, k of 2 blocks and a bit
    (1120, 4096, 128),       # whole tiles, one k block
    (1121, 4112, 384),       # one token over, one 16 of features over
    (7000, 784, 1552),       # few features; k ends inside a group of four blocks
    (225, 20000, 528),       # two token tiles, the last of one token
])
def test_matmul_many_tiles(T, feat, k, trans):
    """Enough tiles for the kernel on CTA pairs."""
    out, inp = (k, feat) if trans else (feat, k)
    h = _matmul_inputs(T, out, inp, trans, T + feat)
    d = [u8_dev(a) for a in h]
    y = run_matmul(*d, trans)
    assert_no_device_error()
    check_product("y", to_f64(y), *h, trans)
    assert torch.equal(y, run_matmul(*d, trans, 0xff))
    h[0][T // 2, 5] = 0x7f
    z = run_matmul(*[u8_dev(a) for a in h], trans)
    assert torch.isnan(z[T // 2]).all()
    z[T // 2] = y[T // 2]
    assert torch.equal(z, y)


def _drawn(k):
    rng = np.random.default_rng(20261206 + k)
    return int(np.exp(rng.uniform(0, np.log(1500)))), 16 * int(rng.integers(1, 120)), 16 * int(rng.integers(1, 120))


@pytest.mark.parametrize("k", range(16))
def test_matmul_drawn(k):
    T, out, inp = _drawn(k)
    for trans in (False, True):
        h = _matmul_inputs(T, out, inp, trans, 100 + k)
        y = run_matmul(*[u8_dev(a) for a in h], trans)
        check_product("y", to_f64(y), *h, trans)
    assert_no_device_error()


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("T", [1, 300])
def test_matmul_nan_stays_in_its_row(T, trans):
    out, inp = 272, 400
    h = _matmul_inputs(T, out, inp, trans, 4)
    clean = run_matmul(*[u8_dev(a) for a in h], trans)
    h[0][T // 2, 5] = 0x7f
    y = run_matmul(*[u8_dev(a) for a in h], trans)
    assert torch.isnan(y[T // 2]).all()
    y[T // 2] = clean[T // 2]
    assert torch.equal(y, clean)


@pytest.mark.parametrize("T", [3, 200])
def test_matmul_t_is_the_gradient_of_matmul(T):
    """y is linear in x: the quotient of <dy, y> along e is <dx, e>, with dy and e exact in 8 bits."""
    out, inp = 400, 272
    q, sc, wq, wsc = _matmul_inputs(T, out, inp, False, 8)
    rng = np.random.default_rng(9)
    dyq, dysc = q8.q8_encode(rng.integers(-8, 9, (T, out)).astype(np.float64))
    dx = to_f64(run_matmul(*[u8_dev(a) for a in (dyq, dysc, wq, wsc)], True))
    x, w, dy = q8.q8_decode(q, sc), q8.q8_decode(wq, wsc, 128), q8.q8_decode(dyq, dysc)
    e = rng.standard_normal((T, inp))
    quotient = ((dy * ((x + 0.5 * e) @ w.T)).sum() - (dy * ((x - 0.5 * e) @ w.T)).sum())
    bound = (2.0 ** -8 * np.abs(dx) * np.abs(e) + 2.0 ** -23 * out * (np.abs(dy) @ np.abs(w)) * np.abs(e)).sum()
    assert abs(quotient - (dx * e).sum()) <= bound


@pytest.mark.parametrize("trans", [False, True])
def test_full_size_rows(trans):
    """The high-rank layer, 15360 tokens: sampled rows and columns."""
    rng = np.random.default_rng(12)
    T, out, inp = 15360, 8192, 8192
    gen = torch.Generator(device=DEV).manual_seed(12)
    x, w = torch.randn(T, inp, generator=gen, device=DEV), torch.randn(out, inp, generator=gen, device=DEV) / 90
    q, sc = store(x)
    wq, wsc = store(w, 128)
    y = run_matmul(q, sc, wq, wsc, trans)
    assert_no_device_error()
    rows = np.sort(rng.choice(T, 40, replace=False))
    rows[0], rows[-1] = 0, T - 1
    h = [q.cpu().numpy()[rows], sc.cpu().numpy()[rows], wq.cpu().numpy(), wsc.cpu().numpy()]
    check_product("y", to_f64(y)[rows], *h, trans)


# ---- together, and their surroundings ---------------------------------------
def test_other_streams_and_graph_replay():
    T, out, inp, r = 300, 272, 400, 24
    q, sc, wq, wsc = (u8_dev(a) for a in _matmul_inputs(T, out, inp, False, 21))
    x = torch.randn(T, inp, device=DEV, dtype=torch.bfloat16)
    dxa = torch.randn(T, r, device=DEV, dtype=torch.bfloat16)
    y, dA = torch.empty(T, out, dtype=torch.bfloat16, device=DEV), torch.empty(r, inp, device=DEV)
    g, n = torch.rand(out, device=DEV) + 0.5, torch.rand(out, device=DEV) + 0.5
    vq, vsc = form(T, out)
    z, db, dl, dm = (torch.empty(T, out, dtype=torch.bfloat16, device=DEV) for _ in range(4))
    dm = torch.empty(out, device=DEV)
    dx = torch.empty(T, inp, dtype=torch.bfloat16, device=DEV)
    w1, w2, w3, w4 = (workspace(k) for k in (
        dora.dora_matmul_q8_workspace(T, out, inp), dora.dora_lora_grad_q8_workspace(T, inp, r),
        dora.dora_compose_bwd_q8_workspace(T, out), dora.dora_matmul_q8_t_workspace(T, out, inp)))

    def step():
        dora.dora_q8_store(x, 1, q, sc)
        dora.dora_matmul_q8(q, sc, wq, wsc, y, w1)
        dora.dora_compose_fwd_q8(y, y, g, 0.5, z, vq, vsc)
        dora.dora_compose_bwd_q8(z, vq, vsc, g, n, 0.5, db, dl, dm, w3)
        dora.dora_lora_grad_q8(dxa, q, sc, dA, w2)
        dora.dora_q8_store(db, 1, vq, vsc)
        dora.dora_matmul_q8_t(vq, vsc, wq, wsc, dx, w4)
        return [t.clone() for t in (y, z, db, dl, dm, dA, dx)]

    ref = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for a in (y, z, db, dl, dm, dA, dx):
            a.fill_(7.0)
        got = step()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out_g = step()
    for _ in range(3):
        for a in (y, z, db, dl, dm, dA, dx):
            a.fill_(7.0)
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, out_g))
    assert_no_device_error()


@pytest.mark.parametrize("T,out,inp,r", [(1, 144, 272, 8), (37, 272, 144, 24), (130, 528, 400, 136), (700, 1040, 656, 264)])
def test_writes_stay_in_bounds(T, out, inp, r):
    h = _matmul_inputs(T, out, inp, False, 31)
    q, sc, wq, wsc = (u8_dev(a) for a in h)
    dyq, dysc = store(torch.randn(T, out, device=DEV))
    dxa = torch.randn(T, r, device=DEV, dtype=torch.bfloat16)
    b = {"y": Guarded(T * out * 2), "dx": Guarded(T * inp * 2), "dA": Guarded(r * inp * 4), "q": Guarded(T * out),
         "scale": Guarded(T * -(-out // 128)), "z": Guarded(T * out * 2), "x": Guarded(T * out * 2)}
    n = {"w1": dora.dora_matmul_q8_workspace(T, out, inp), "w2": dora.dora_matmul_q8_t_workspace(T, out, inp),
         "w3": dora.dora_lora_grad_q8_workspace(T, inp, r)}
    b |= {k: Guarded(v) for k, v in n.items()}
    ws = {k: b[k].view(U8, (v,)) for k, v in n.items()}
    bf = torch.bfloat16
    y = b["y"].view(bf, (T, out))
    dora.dora_matmul_q8(q, sc, wq, wsc, y, ws["w1"])
    dora.dora_matmul_q8_t(dyq, dysc, wq, wsc, b["dx"].view(bf, (T, inp)), ws["w2"])
    dora.dora_lora_grad_q8(dxa, q, sc, b["dA"].view(torch.float32, (r, inp)), ws["w3"])
    vq, vsc = b["q"].view(U8, (T, out)), b["scale"].view(U8, (T, -(-out // 128)))
    dora.dora_compose_fwd_q8(y, y, torch.ones(out, device=DEV), 1.0, b["z"].view(bf, (T, out)), vq, vsc)
    dora.dora_q8_load(vq, vsc, 1, b["x"].view(bf, (T, out)))
    torch.cuda.synchronize()
    for k, v in b.items():
        v.check(k)
    assert_no_device_error()
