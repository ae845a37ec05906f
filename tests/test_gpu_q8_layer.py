"""The layer on an 8-bit weight (ops.dora_linear_q8): its output and gradients
against a fp64 evaluation of the same layer on the values that it rounds to
8 bits, through autograd and under torch.compile; what it keeps in memory; the
kernels' failure path."""
import numpy as np
import pytest
import torch

import parameter_efficient_fine_gb300 as dora
from oracle import q8_oracle as q8
from parameter_efficient_fine_gb300 import ops

from gpu_util import DEV, assert_no_device_error, to_f64

pytestmark = pytest.mark.gpu


def _layer(T, out, inp, r, seed, dtype=torch.float32):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen, device=DEV)  # noqa: E731
    W0 = rnd(out, inp) / inp ** 0.5
    wq, wscale = ops.q8_store(W0, 128)
    A, B = (rnd(r, inp) / inp ** 0.5).to(dtype), (0.1 * rnd(out, r)).to(dtype)
    W = ops.q8_load(wq, wscale, 128, torch.bfloat16)
    s = 2.0
    norm = (W.float() + s * (B.float() @ A.float())).norm(dim=1)
    m = norm * (1 + 0.02 * rnd(out))
    return dict(x=rnd(T, inp).bfloat16(), wq=wq, wscale=wscale, A=A, B=B, m=m, g=m / norm, norm=norm, s=s), rnd(T, out).bfloat16()


def _reference(d, dy):
    """fp64, with x and W0 as their 8-bit values in the base product and dA."""
    f = {k: to_f64(v) for k, v in d.items() if k in ("x", "A", "B", "g", "norm")}
    x8 = q8.q8_decode(*q8.q8_encode(f["x"]))
    w8 = q8.q8_decode(d["wq"].cpu().numpy(), d["wscale"].cpu().numpy(), 128)
    dy, s = to_f64(dy), d["s"]
    v = x8 @ w8.T + s * (f["x"] @ f["A"].T @ f["B"].T)
    d_base = f["g"] * dy
    d_lora = s * d_base
    dxa = d_lora @ f["B"]
    return {"y": f["g"] * v, "x": d_base @ w8 + dxa @ f["A"], "A": dxa.T @ x8, "B": d_lora.T @ (f["x"] @ f["A"].T),
            "m": (dy * v).sum(0) / f["norm"]}


def _near(name, got, ref, tol):
    err = np.linalg.norm(to_f64(got) - ref) / np.linalg.norm(ref)
    assert err <= tol, f"{name}: {err:.2e} > {tol:.0e}"


# one rounding to bf16 is 2^-9 at most, its random part 0.0017 of a value; the
# bf16 chain of a term has up to three of them.  E4M3 rounds by 2^-4 at most,
# with a random part of 0.026: it enters dx through d_base and d_mag through v
TOL = {"y": 0.006, "x": 0.035, "A": 0.008, "B": 0.008, "m": 0.035}


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,out,inp,r", [(1, 144, 272, 8), (37, 272, 144, 24), (300, 528, 400, 72), (1500, 1024, 768, 64)])
def test_layer_forward_and_backward(T, out, inp, r, dtype):
    d, dy = _layer(T, out, inp, r, T + r, dtype)
    for k in ("x", "A", "B", "m"):
        d[k].requires_grad_(True)
    y = ops.dora_linear_q8(**d)
    y.backward(dy)
    assert_no_device_error()
    ref = _reference(d, dy)
    _near("y", y, ref["y"], TOL["y"])
    for k in ("x", "A", "B", "m"):
        assert d[k].grad.dtype == d[k].dtype
        _near("d" + k, d[k].grad, ref[k], TOL[k])


def test_layer_compiles_and_skips_what_needs_no_gradient():
    d, dy = _layer(300, 528, 400, 72, 5)
    d["A"].requires_grad_(True)
    f = torch.compile(lambda **k: ops.dora_linear_q8(**k), fullgraph=True, backend="aot_eager")
    y = f(**d)
    y.backward(dy)
    grad, d["A"].grad = d["A"].grad.clone(), None
    z = ops.dora_linear_q8(**d)
    z.backward(dy)
    assert torch.equal(y, z) and torch.equal(grad, d["A"].grad)
    assert d["x"].grad is None and d["m"].grad is None


def test_layer_keeps_two_bytes_an_element():
    """From forward to backward: x and v in 8 bits with their scales, and xa."""
    T, out, inp, r = 4096, 1024, 1024, 64
    d, _ = _layer(T, out, inp, r, 6)
    d["A"].requires_grad_(True)
    kept = []
    with torch.autograd.graph.saved_tensors_hooks(lambda t: kept.append(t) or t, lambda t: t):
        ops.dora_linear_q8(**d)
    own = {t.data_ptr() for t in d.values() if isinstance(t, torch.Tensor)}
    size = sum(t.numel() * t.element_size() for t in kept if t.data_ptr() not in own)
    assert 0 < size <= T * (inp + out) * (1 + 1 / 128) + 2 * T * r


def test_compose_q8_matches_compose_where_v_is_exact():
    gen = torch.Generator(device=DEV).manual_seed(7)
    base = torch.randint(-4, 5, (200, 384), generator=gen, device=DEV).float().requires_grad_(True)
    lora = (2.0 * torch.randint(-3, 4, (200, 384), generator=gen, device=DEV)).float().requires_grad_(True)
    m = torch.rand(384, generator=gen, device=DEV).requires_grad_(True)
    norm = torch.rand(384, generator=gen, device=DEV) + 0.5
    g, dy = (m / norm).detach(), torch.randn(200, 384, generator=gen, device=DEV)
    out = []
    for f in (lambda: ops.compose(base, lora, m, g, norm, 0.5), lambda: ops.compose_q8(base, lora, m, g, norm, 0.5)[0]):
        y = f()
        out.append([y, *torch.autograd.grad(y, (base, lora, m), dy)])
    for a, b in zip(*out[:2]):
        torch.testing.assert_close(a, b, rtol=2e-6, atol=2e-6)


@pytest.mark.parametrize("call", ["matmul", "pairs", "grad"])
def test_withheld_loads_end_in_an_error(call):
    """The kernels' waits give up, record a code and leave the context usable."""
    u8 = torch.uint8
    T, out, inp = {"matmul": (20, 256, 512), "pairs": (2000, 2560, 512), "grad": (300, 0, 256)}[call]
    q, sc = ops.q8_store(torch.randn(T, inp, device=DEV), 1)
    ws = torch.empty(1 << 24, dtype=u8, device=DEV)
    if call == "grad":
        dxa, dA = torch.randn(T, 16, device=DEV).bfloat16(), torch.empty(16, inp, device=DEV)
        run = lambda: dora.dora_lora_grad_q8(dxa, q, sc, dA, ws)  # noqa: E731
        res = dA
    else:
        wq, wsc = ops.q8_store(torch.randn(out, inp, device=DEV), 128)
        res = torch.empty(T, out, device=DEV, dtype=torch.bfloat16)
        run = lambda: dora.dora_matmul_q8(q, sc, wq, wsc, res, ws)  # noqa: E731
    run()
    good = res.clone()
    assert_no_device_error()
    dora.dora_test_stall_loads(True, 20_000_000)
    try:
        run()
        torch.cuda.synchronize()
        assert dora.dora_device_error() != 0
    finally:
        dora.dora_test_stall_loads(False)
    run()
    assert_no_device_error()
    assert torch.equal(res, good)
