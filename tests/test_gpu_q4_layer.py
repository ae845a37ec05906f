"""The operators on a 4-bit weight and the experts' routing as they are used together:
the DoRA layer (ops.dora_linear_q4), experts with their activation, their gradients
through autograd, torch.compile, graphs, streams, and the kernels' failure path.

Tolerances on norms: one rounding to bf16 is 2^-8 of a value at most, its random part
0.0017; the bf16 chain of a term has up to four of them, 0.0034, taken twice for what a
chain's rounded factors add.  x and v in 8 bits (E4M3) have a random part of 0.026,
which enters dA and d_mag.
"""
import numpy as np
import pytest
import torch

import parameter_efficient_fine_gb300 as dora
from oracle import q4_oracle as q4
from oracle import q8_oracle as q8
from parameter_efficient_fine_gb300 import ops

from gpu_util import DEV, assert_no_device_error, to_f64

pytestmark = pytest.mark.gpu

BF, U8, I32 = torch.bfloat16, torch.uint8, torch.int32


def _near(name, got, ref, tol):
    err = np.linalg.norm(to_f64(got) - ref) / np.linalg.norm(ref)
    assert err <= tol, f"{name}: {err:.2e} > {tol:.0e}"


def _rnd(seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    return lambda *s: torch.randn(*s, generator=gen, device=DEV)


def _values(q, scale):
    return q4.q4_decode(q.cpu().numpy(), scale.cpu().numpy())


# ---- the DoRA layer ---------------------------------------------------------
def _layer(T, out, inp, r, seed, dtype=torch.float32):
    rnd = _rnd(seed)
    wq, wscale = ops.q4_store(rnd(out, inp) / inp ** 0.5)
    A, B = (rnd(r, inp) / inp ** 0.5).to(dtype), (0.1 * rnd(out, r)).to(dtype)
    W = ops.q4_load(wq, wscale, torch.float32)
    s = 2.0
    m = torch.ones(out, device=DEV)
    norm, _ = ops.norm_factored(W, A.float(), B.float(), m, s)
    m = norm * (1 + 0.02 * rnd(out))
    return dict(x=rnd(T, inp).to(BF), wq=wq, wscale=wscale, A=A, B=B, m=m, g=m / norm, norm=norm, s=s), rnd(T, out).to(BF)


def _reference(d, dy):
    """fp64, with x in dA and v in d_mag as the form keeps them, which is part of their tolerance."""
    f = {k: to_f64(v) for k, v in d.items() if k in ("x", "A", "B", "g", "norm")}
    W, dy, s = _values(d["wq"], d["wscale"]), to_f64(dy), d["s"]
    v = f["x"] @ W.T + s * (f["x"] @ f["A"].T @ f["B"].T)
    d_base = f["g"] * dy
    dxa = s * d_base @ f["B"]
    x8 = q8.q8_decode(*q8.q8_encode(f["x"]))
    return {"y": f["g"] * v, "x": d_base @ W + dxa @ f["A"], "A": dxa.T @ x8, "B": s * d_base.T @ (f["x"] @ f["A"].T),
            "m": (dy * v).sum(0) / f["norm"]}


TOL = {"y": 0.007, "x": 0.008, "A": 0.008, "B": 0.008, "m": 0.035}


@pytest.mark.parametrize("dtype", [torch.float32, BF])
@pytest.mark.parametrize("T,out,inp,r", [(1, 144, 288, 8), (12, 272, 160, 16), (37, 272, 128, 24), (300, 528, 416, 72), (1500, 1024, 768, 64)])
def test_layer_forward_and_backward(T, out, inp, r, dtype):
    d, dy = _layer(T, out, inp, r, T + r, dtype)
    served = ops.dora_linear_q4(**d)                # nothing takes a gradient: nothing is kept
    for k in ("x", "A", "B", "m"):
        d[k].requires_grad_(True)
    y = ops.dora_linear_q4(**d)
    assert torch.equal(served, y)
    y.backward(dy)
    assert_no_device_error()
    ref = _reference(d, dy)
    _near("y", y, ref["y"], TOL["y"])
    for k in ("x", "A", "B", "m"):
        assert d[k].grad.dtype == d[k].dtype
        _near("d" + k, d[k].grad, ref[k], TOL[k])


def test_layer_compiles_and_skips_what_needs_no_gradient():
    d, dy = _layer(300, 528, 416, 72, 5)
    d["A"].requires_grad_(True)
    f = torch.compile(lambda **k: ops.dora_linear_q4(**k), fullgraph=True, backend="aot_eager")
    y = f(**d)
    y.backward(dy)
    grad, d["A"].grad = d["A"].grad.clone(), None
    z = ops.dora_linear_q4(**d)
    z.backward(dy)
    assert torch.equal(y, z) and torch.equal(grad, d["A"].grad)
    assert d["x"].grad is None and d["m"].grad is None


def test_layer_keeps_two_bytes_an_element():
    T, out, inp, r = 4096, 1024, 1024, 64
    d, _ = _layer(T, out, inp, r, 6)
    d["A"].requires_grad_(True)
    kept = []
    with torch.autograd.graph.saved_tensors_hooks(lambda t: kept.append(t) or t, lambda t: t):
        ops.dora_linear_q4(**d)
    own = {t.data_ptr() for t in d.values() if isinstance(t, torch.Tensor)}
    size = sum(t.numel() * t.element_size() for t in kept if t.data_ptr() not in own)
    assert 0 < size <= T * (inp + out) * (1 + 1 / 128) + 2 * T * r


def test_norm_of_the_4_bit_weight_from_bfloat16_is_exact():
    """q4_load to bfloat16 loses nothing: the bf16 norm's input is the form's values."""
    d, _ = _layer(1, 272, 544, 16, 8)
    a, b = (ops.q4_load(d["wq"], d["wscale"], t).float() for t in (BF, torch.float32))
    assert torch.equal(a, b)


# ---- experts ----------------------------------------------------------------
def _experts(T, k, E, inp, hid, seed, padded=False):
    rnd = _rnd(seed)
    x = rnd(T, inp).to(BF)
    gate, up = (ops.q4_store(rnd(E, hid, inp) / inp ** 0.5) for _ in range(2))
    down = ops.q4_store(rnd(E, inp, hid) / hid ** 0.5)
    score = rnd(T, E)
    weight, expert = score.softmax(-1).topk(k, dim=-1)
    if padded:
        expert = expert.clone()
        expert[T - T // 4:] = -1
        expert[0, 0] = expert[0, -1]                  # the same expert twice
    return x, expert, weight.contiguous(), gate, up, down


def _mlp(x, expert, weight, gate, up, down):
    """Experts as a model calls them: one sort, one send, three products, one return."""
    _, inverse, offsets = ops.expert_sort(expert, gate[0].shape[0])
    xs = ops.expert_send(x, inverse, offsets)
    hs = torch.nn.functional.silu(ops.matmul_q4(xs, *gate, offsets)) * ops.matmul_q4(xs, *up, offsets)
    return ops.expert_return(ops.matmul_q4(hs, *down, offsets), inverse, offsets, weight)


def _mlp_reference(x, expert, weight, gate, up, down, dy):
    x, w = x.detach().double().cpu().requires_grad_(True), weight.detach().double().cpu().requires_grad_(True)
    G, U, D = (torch.from_numpy(np.stack([_values(q, s) for q, s in zip(*f)])) for f in (gate, up, down))
    y = torch.zeros(x.shape[0], D.shape[1], dtype=torch.float64)
    for t, row in enumerate(expert.cpu().tolist()):
        for j, e in enumerate(row):
            if 0 <= e < G.shape[0]:
                h = torch.nn.functional.silu(G[e] @ x[t]) * (U[e] @ x[t])
                y[t] = y[t] + w[t, j] * (D[e] @ h)
    y.backward(dy.double().cpu())
    return y.detach().numpy(), x.grad.numpy(), w.grad.numpy()


@pytest.mark.parametrize("padded", [False, True])
@pytest.mark.parametrize("T,k,E,inp,hid", [(1, 2, 4, 128, 160), (4, 3, 8, 288, 128), (60, 2, 3, 160, 272), (300, 4, 6, 256, 144)])
def test_experts_forward_and_backward(T, k, E, inp, hid, padded):
    hid = -(-hid // 32) * 32
    x, expert, weight, *W = _experts(T, k, E, inp, hid, T + k, padded)
    x.requires_grad_(True)
    weight.requires_grad_(True)
    y = _mlp(x, expert, weight, *W)
    dy = _rnd(1)(T, inp).to(BF)
    y.backward(dy)
    assert_no_device_error()
    ref = _mlp_reference(x, expert, weight, *W, dy)
    # five bf16 roundings in a row on the way to y, eight on the way to dx
    for name, got, want, tol in zip(("y", "dx", "dw"), (y, x.grad, weight.grad), ref, (0.012, 0.02, 0.015)):
        _near(name, got, want, tol)
    if padded and T >= 4:
        assert not y[T - T // 4:].any() and not x.grad[T - T // 4:].any() and not weight.grad[T - T // 4:].any()


def test_one_product_of_experts_and_its_tail():
    x, expert, weight, gate, *_ = _experts(50, 3, 5, 256, 160, 3, padded=True)
    y = ops.experts_q4(x, expert, weight.to(BF), *gate)
    _, inverse, offsets = ops.expert_sort(expert, 5)
    ys = ops.matmul_q4(ops.expert_send(x, inverse, offsets), *gate, offsets)
    assert torch.equal(y, ops.expert_return(ys, inverse, offsets, weight.to(BF).float()))
    n = int(offsets[-1])
    assert n < 150 and not ys[n:].any()               # rows that no expert has
    assert torch.equal(expert.int(), expert.int()) and all(
        torch.equal(a, b) for a, b in zip(ops.expert_sort(expert, 5), ops.expert_sort(expert.int(), 5)))


def test_clear_takes_rows_on_both_sides():
    for dtype, cols in ((BF, 24), (torch.float32, 7), (BF, 5)):
        x = torch.ones(10, cols, device=DEV, dtype=dtype)
        dora.dora_expert_clear(x, torch.tensor([2, 3, 7], dtype=I32, device=DEV))
        assert x[:, 0].tolist() == [0, 0, 1, 1, 1, 1, 1, 0, 0, 0] and torch.equal(x.amin(1), x.amax(1))
        dora.dora_expert_clear(x, torch.tensor([-4, 99], dtype=I32, device=DEV))
        assert x[:, 0].tolist() == [0, 0, 1, 1, 1, 1, 1, 0, 0, 0]


@pytest.mark.parametrize("T", [5, 40, 200])
def test_transposed_product_is_the_gradient(T):
    """<x W^T, dy> = <x, dy W>, and a difference of the product in a direction of x."""
    rnd = _rnd(T)
    wq, ws = ops.q4_store(rnd(272, 544))
    x, dx = (torch.randint(-4, 5, (T, 544), generator=torch.Generator(device=DEV).manual_seed(T + i), device=DEV).to(BF) for i in range(2))
    dy = rnd(T, 272).to(BF)
    x.requires_grad_(True)
    y = ops.matmul_q4(x, wq, ws)
    y.backward(dy)
    W = _values(wq, ws)
    # small whole numbers: x + dx and x - dx are exact, so the difference is the product itself
    diff = (to_f64(ops.matmul_q4((x + dx).detach(), wq, ws)) - to_f64(ops.matmul_q4((x - dx).detach(), wq, ws))) / 2
    left, right = (diff * to_f64(dy)).sum(), (to_f64(dx) * to_f64(x.grad)).sum()
    scale = (np.abs(to_f64(dx)) @ np.abs(W).T * np.abs(to_f64(dy))).sum()
    size = (np.abs(to_f64((x + dx).detach())) @ np.abs(W).T * np.abs(to_f64(dy))).sum()
    # every result of either side is off by half a bf16 step and the fp32 sum
    assert abs(left - right) <= 2.0 ** -8 * (scale + 2 * size)


def test_opcheck():
    x, expert, weight, gate, *_ = _experts(12, 2, 3, 128, 160, 4)
    _, inverse, offsets = ops.expert_sort(expert, 3)
    xs = ops.expert_send(x, inverse, offsets)
    q, s = ops.q4_store(_rnd(0)(48, 64))
    tests = ("test_schema", "test_autograd_registration", "test_faketensor")
    check = lambda op, *a: torch.library.opcheck(op, a, test_utils=tests)  # noqa: E731
    check(torch.ops.dora.q4_store.default, _rnd(1)(8, 64))
    check(torch.ops.dora.q4_load.default, q, s, BF)
    check(torch.ops.dora.matmul_q4.default, _rnd(2)(7, 64).to(BF).requires_grad_(True), q, s, None)
    check(torch.ops.dora.matmul_q4.default, xs.detach().requires_grad_(True), *gate, offsets)
    check(torch.ops.dora.matmul_q4_t.default, _rnd(3)(7, 48).to(BF), q, s, None)
    check(torch.ops.dora.expert_sort.default, expert, 3)
    check(torch.ops.dora.expert_send.default, x.detach().requires_grad_(True), inverse, offsets)
    check(torch.ops.dora.expert_return.default, xs.detach().requires_grad_(True), inverse, offsets, weight.detach().requires_grad_(True))
    check(torch.ops.dora.expert_return.default, xs.detach().requires_grad_(True), inverse, offsets, None)
    check(torch.ops.dora.expert_return_bwd.default, x, xs, inverse, offsets, weight)


def test_experts_compile():
    x, expert, weight, *W = _experts(40, 2, 3, 160, 192, 9, padded=True)
    one = lambda a, e, w, gate, *_: ops.experts_q4(a, e, w, *gate)  # noqa: E731
    for step, dy in ((_mlp, _rnd(2)(40, 160).to(BF)), (one, _rnd(2)(40, 192).to(BF))):
        grads = []
        for f in (step, torch.compile(step, fullgraph=True, backend="aot_eager")):
            a, b = x.clone().requires_grad_(True), weight.clone().requires_grad_(True)
            y = f(a, expert, b, *W)
            y.backward(dy)
            grads.append((y.detach(), b.grad, a.grad))
        # (a traced silu's own gradient is another formula's in bf16: through it dx is
        # equal only up to that)
        for p, q in list(zip(*grads))[: 2 if step is _mlp else 3]:
            assert torch.equal(p, q)


# ---- graphs, streams --------------------------------------------------------
@pytest.mark.parametrize("T", [1, 8, 40, 200])
def test_graph_replay_takes_new_inputs(T):
    """A whole pass through the experts in a CUDA graph, replayed with other tokens, other
    experts and other loads."""
    x, expert, weight, *W = _experts(T, 2, 6, 160, 256, T)
    _mlp(x, expert, weight, *W)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = _mlp(x, expert, weight, *W)
    for seed in (50, 51, 52):
        nx, ne, nw, *_ = _experts(T, 2, 6, 160, 256, seed, padded=seed == 51)
        x.copy_(nx)
        expert.copy_(ne)
        weight.copy_(nw)
        graph.replay()
        want = _mlp(nx, ne, nw, *W)
        torch.cuda.synchronize()
        assert torch.equal(y, want)
    assert_no_device_error()


def test_forward_and_backward_in_one_graph():
    x, expert, weight, *W = _experts(100, 2, 4, 160, 256, 1)
    dy = _rnd(3)(100, 160).to(BF)

    def step(a, w):
        y = _mlp(a, expert, w, *W)
        return (y, *torch.autograd.grad(y, (a, w), dy))
    want = [v.clone() for v in step(x.clone().requires_grad_(True), weight.clone().requires_grad_(True))]
    a, w = x.clone().requires_grad_(True), weight.clone().requires_grad_(True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(a, w)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(a, w)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p.detach(), q.detach()) for p, q in zip(got, want))


@pytest.mark.parametrize("t", [False, True], ids=["xWt", "dyW"])
def test_calls_on_several_streams_at_once(t):
    """Calls of different sizes in flight together, each with a workspace of its own."""
    rnd = _rnd(11)
    out, inp = 1040, 1120
    wq, ws = ops.q4_store(rnd(out, inp))
    sizes = [1, 8, 20, 100, 150, 700]
    xs = [rnd(T, out if t else inp).to(BF) for T in sizes]
    f = ops.matmul_q4_t if t else ops.matmul_q4
    want = [f(x, wq, ws) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sizes]
    for _ in range(5):
        got = []
        for x, st in zip(xs, streams):
            with torch.cuda.stream(st):
                got.append(f(x, wq, ws))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert_no_device_error()


def test_stream_argument():
    rnd = _rnd(12)
    wq, ws = ops.q4_store(rnd(272, 288))
    x = rnd(5, 288).to(BF)
    want = ops.matmul_q4(x, wq, ws)
    torch.cuda.synchronize()
    st, y = torch.cuda.Stream(), torch.empty(5, 272, dtype=BF, device=DEV)
    dora.dora_matmul_q4(x, wq, ws, y, stream=st)
    st.synchronize()
    assert torch.equal(y, want)


def test_calls_back_to_back_read_what_the_one_before_wrote():
    """The products' launches overlap the end of the launch before them: a chain in which
    each reads the result of the last, weight included, many times over."""
    rnd = _rnd(13)
    W = rnd(256, 256) / 16
    for T in (1, 8, 9, 64, 150, 300):
        x = rnd(T, 256).to(BF)
        want = None
        for _ in range(20):
            y = x
            for i in range(6):
                q, s = ops.q4_store(W * (1 + i))          # the weight itself is new at each step
                y = ops.matmul_q4(y, q, s)
                y = ops.matmul_q4_t(y, q, s)
            if want is None:
                torch.cuda.synchronize()
                want = x
                for i in range(6):
                    q, s = ops.q4_store(W * (1 + i))
                    torch.cuda.synchronize()
                    want = ops.matmul_q4(want, q, s)
                    torch.cuda.synchronize()
                    want = ops.matmul_q4_t(want, q, s)
                    torch.cuda.synchronize()
            assert torch.equal(y, want)


# ---- the failure path -------------------------------------------------------
@pytest.mark.parametrize("t", [False, True], ids=["xWt", "dyW"])
@pytest.mark.parametrize("T,inp", [(1, 512), (1, 544), (20, 512), (20, 544), (60, 512), (120, 512), (120, 544), (300, 512), (700, 4096)])
def test_withheld_loads_end_in_an_error(T, inp, t):
    rnd = _rnd(T)
    wq, ws = ops.q4_store(rnd(400, inp))
    x = rnd(T, 400 if t else inp).to(BF)
    f = ops.matmul_q4_t if t else ops.matmul_q4
    good = f(x, wq, ws)
    assert_no_device_error()
    dora.dora_test_stall_loads(True, 20_000_000)      # 20 ms
    try:
        f(x, wq, ws)
        code = dora.dora_device_error()               # synchronises
    finally:
        dora.dora_test_stall_loads(False)
    assert code != 0
    again = f(x, wq, ws)
    assert_no_device_error()
    assert torch.equal(again, good)
