"""What the 4-bit operators and the experts' calls refuse, on the CPU: the binding by
shapes and types, the C ABI by its status, before anything is launched."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import parameter_efficient_fine_gb300 as dora
from parameter_efficient_fine_gb300 import build as dbuild
from parameter_efficient_fine_gb300 import ops

FAKE = 1 << 20      # a 256-byte aligned non-null address: never dereferenced on these paths
OK, NULL, SHAPE, ALIGN, DTYPE, WORKSPACE = 0, 1, 2, 3, 4, 5
BF, F32, U8, I32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32


@pytest.fixture(scope="module")
def lib():
    dbuild.build()
    return dora.load_library()


def _empty(dtype, *shape):
    return torch.empty(*shape, dtype=dtype)


# ---- binding ----------------------------------------------------------------
@pytest.mark.parametrize("x,q,scale", [
    ((BF, 4, 48), (U8, 4, 24), (U8, 4, 1)),            # no whole groups
    ((BF, 4, 64), (U8, 4, 64), (U8, 4, 2)),            # a byte an element
    ((BF, 4, 64), (U8, 4, 32), (U8, 4, 1)),
    ((BF, 4, 64), (U8, 8, 32), (U8, 8, 2)),
    ((BF, 2, 4, 64), (U8, 8, 32), (U8, 8, 2)),         # a stack's form is a stack
    ((BF, 64), (U8, 32), (U8, 2)),
])
def test_forms_of_other_shapes_are_refused(x, q, scale):
    x, q, scale = _empty(*x), _empty(*q), _empty(*scale)
    with pytest.raises(ValueError, match="4-bit form|a matrix"):
        dora.dora_q4_store(x, q, scale)
    with pytest.raises(ValueError, match="4-bit form|a matrix"):
        dora.dora_q4_load(q, scale, x)


def test_types_are_refused():
    with pytest.raises(TypeError, match="bytes"):
        dora.dora_q4_store(_empty(BF, 4, 64), _empty(I32, 4, 32), _empty(U8, 4, 2))
    with pytest.raises(TypeError, match="dtype"):
        dora.dora_q4_store(_empty(torch.float16, 4, 64), _empty(U8, 4, 32), _empty(U8, 4, 2))
    with pytest.raises(TypeError, match="int32 or int64"):
        dora.dora_expert_sort(_empty(torch.int16, 4, 2), 3, _empty(I32, 8), _empty(I32, 4, 2), _empty(I32, 4))


def test_host_tensors_are_refused():
    with pytest.raises(ValueError, match="CUDA tensors"):
        dora.dora_q4_store(_empty(BF, 4, 64), _empty(U8, 4, 32), _empty(U8, 4, 2))
    with pytest.raises(ValueError, match="CUDA tensors"):
        dora.dora_expert_sort(_empty(I32, 4, 2), 3, _empty(I32, 8), _empty(I32, 4, 2), _empty(I32, 4))


GOOD = dict(x=(BF, 5, 64), wq=(U8, 48, 32), wscale=(U8, 48, 2), y=(BF, 5, 48), offsets=None)
STACK = dict(GOOD, wq=(U8, 3, 48, 32), wscale=(U8, 3, 48, 2), offsets=(I32, 4))


@pytest.mark.parametrize("base,change", [
    (GOOD, dict(x=(F32, 5, 64))), (GOOD, dict(x=(BF, 5, 32))), (GOOD, dict(y=(BF, 4, 48))), (GOOD, dict(y=(F32, 5, 48))),
    (GOOD, dict(wscale=(U8, 48, 1))), (GOOD, dict(wq=(BF, 48, 32))), (GOOD, dict(wq=(U8, 48, 24))),
    (GOOD, dict(wq=(U8, 3, 48, 32))), (GOOD, dict(offsets=(I32, 2))), (STACK, dict(offsets=None)),
    (STACK, dict(offsets=(I32, 3))), (STACK, dict(offsets=(torch.int64, 4))), (STACK, dict(wscale=(U8, 48, 2))),
])
def test_products_of_other_shapes_are_refused(base, change):
    d = {k: v and _empty(*v) for k, v in dict(base, **change).items()}
    with pytest.raises((TypeError, ValueError), match="dora_matmul_q4"):
        dora.dora_matmul_q4(d["x"], d["wq"], d["wscale"], d["y"], d["offsets"])
    with pytest.raises((TypeError, ValueError), match="dora_matmul_q4_t"):
        dora.dora_matmul_q4_t(d["y"], d["wq"], d["wscale"], d["x"], d["offsets"])


ROUTE = dict(x=(BF, 4, 24), xs=(BF, 8, 24), inverse=(I32, 4, 2), offsets=(I32, 4), weight=(F32, 4, 2))


@pytest.mark.parametrize("change", [
    dict(xs=(BF, 7, 24)), dict(xs=(F32, 8, 24)), dict(xs=(BF, 8, 16)), dict(x=(BF, 5, 24)), dict(inverse=(torch.int64, 4, 2)),
    dict(offsets=(I32, 1)), dict(offsets=(I32, 4098)), dict(offsets=(torch.int64, 4)), dict(offsets=(I32, 2, 2)),
])
def test_routes_of_other_shapes_are_refused(change):
    d = {k: _empty(*v) for k, v in dict(ROUTE, **change).items()}
    with pytest.raises((TypeError, ValueError), match="dora_expert_send"):
        dora.dora_expert_send(d["x"], d["inverse"], d["offsets"], d["xs"])
    with pytest.raises((TypeError, ValueError), match="dora_expert_return"):
        dora.dora_expert_return(d["xs"], d["inverse"], d["offsets"], d["weight"], d["x"])
    with pytest.raises((TypeError, ValueError), match="dora_expert_return_bwd"):
        dora.dora_expert_return_bwd(d["x"], d["xs"], d["inverse"], d["offsets"], d["weight"], d["xs"], d["weight"])


def test_weights_of_another_shape_or_type_are_refused():
    d = {k: _empty(*v) for k, v in ROUTE.items()}
    for w in (_empty(F32, 4, 3), _empty(BF, 4, 2)):
        with pytest.raises(ValueError, match="dora_expert_return"):
            dora.dora_expert_return(d["xs"], d["inverse"], d["offsets"], w, d["x"])
        with pytest.raises(ValueError, match="dora_expert_return_bwd"):
            dora.dora_expert_return_bwd(d["x"], d["xs"], d["inverse"], d["offsets"], w, d["xs"], d["weight"])
    with pytest.raises(ValueError, match="experts"):
        dora.dora_expert_sort(_empty(I32, 4, 2), 0, _empty(I32, 8), _empty(I32, 4, 2), _empty(I32, 1))


# ---- C ABI ------------------------------------------------------------------
def test_store_and_load_statuses(lib):
    for f, args in ((lib.dora_q4_store, lambda a, x, r, c, q, s: (a, x, r, c, q, s, None)),
                    (lib.dora_q4_load, lambda a, x, r, c, q, s: (a, q, s, r, c, x, None))):
        assert f(*args(7, FAKE, 4, 64, FAKE, FAKE)) == DTYPE
        for r, c in ((-1, 64), (4, -32), (4, 48), (1 << 31, 32)):
            assert f(*args(1, FAKE, r, c, FAKE, FAKE)) == SHAPE
        assert f(*args(1, FAKE, 0, 64, FAKE, FAKE)) == OK and f(*args(1, None, 4, 0, None, None)) == OK
        for x, q, s in ((None, FAKE, FAKE), (FAKE, None, FAKE), (FAKE, FAKE, None)):
            assert f(*args(1, x, 4, 64, q, s)) == NULL
        assert f(*args(1, FAKE + 2, 4, 64, FAKE, FAKE)) == ALIGN and f(*args(1, FAKE, 4, 64, FAKE + 4, FAKE)) == ALIGN


@pytest.mark.parametrize("t", [False, True])
def test_product_statuses(lib, t):
    f = lib.dora_matmul_q4_t if t else lib.dora_matmul_q4

    def call(x=FAKE, off=None, wq=FAKE, ws=FAKE, T=5, out=48, inp=64, E=1, y=FAKE, wk=None, n=0):
        return f(x, off, wq, ws, T, out, inp, E, y, wk, n, None)

    for bad in (dict(T=-1), dict(out=-16), dict(inp=-32), dict(inp=48), dict(E=0), dict(E=4097, off=FAKE), dict(T=1 << 31),
                dict(out=0) if t else dict(inp=0)):
        assert call(**bad) == SHAPE, bad
    for bad in (dict(x=None), dict(wq=None), dict(ws=None), dict(y=None), dict(E=3)):
        assert call(**bad) == NULL, bad
    for bad in (dict(x=FAKE + 2), dict(wq=FAKE + 8), dict(ws=FAKE + 4), dict(y=FAKE + 8), dict(off=FAKE + 2, E=3), dict(out=40)):
        assert call(**bad) == ALIGN, bad
    assert call(T=0) == OK and call(**(dict(inp=0) if t else dict(out=0))) == OK
    big = dict(T=200, out=8192, inp=8192)
    size = (dora.dora_matmul_q4_t_workspace if t else dora.dora_matmul_q4_workspace)(200, 8192, 8192, 1)
    assert size > 0
    for wk, n in ((None, 0), (FAKE, size - 1), (FAKE + 128, size)):
        assert call(**big, wk=wk, n=n) == WORKSPACE


def test_workspaces():
    w, wt = dora.dora_matmul_q4_workspace, dora.dora_matmul_q4_t_workspace
    assert w(1, 8192, 8192) == w(8, 8192, 8192) == 0 and w(15360, 8192, 8192) == wt(15360, 8192, 8192) == 0
    assert w(9, 64, 128) == 2 * 9 * 128 + 8 * 9                # pieces of x and their scale words
    # experts: tiles for twice the mean
    assert w(32, 64, 128, 8) == 0 and w(40, 64, 128, 8) == w(33, 64, 128, 8) // 33 * 40 == 2 * 40 * 128 + 8 * 40
    for bad in ((0, 64, 128, 1), (9, 0, 128, 1), (9, 64, 0, 1), (9, 64, 128, 0), (9, 64, 128, 5000)):
        assert w(*bad) == wt(*bad) == 0
    # never more than eight parts of the result
    for T in (130, 200, 1000, 5000):
        for out, inp in ((256, 14336), (8192, 8192), (1024, 1024)):
            assert w(T, out, inp) <= 8 * T * out * 4 and wt(T, out, inp) <= 8 * T * inp * 4


def test_route_statuses(lib):
    sort = lambda ib=4, e=FAKE, T=4, k=2, E=3, o=FAKE, i=FAKE, f=FAKE: lib.dora_expert_sort(ib, e, T, k, E, o, i, f, None)  # noqa: E731
    assert sort(ib=2) == DTYPE
    for bad in (dict(T=-1), dict(k=0), dict(E=0), dict(E=4097), dict(T=1 << 30, k=2)):
        assert sort(**bad) == SHAPE, bad
    for bad in (dict(e=None), dict(o=None), dict(i=None), dict(f=None)):
        assert sort(**bad) == NULL, bad
    assert sort(e=FAKE + 2) == ALIGN and sort(ib=8, e=FAKE + 4) == ALIGN and sort(f=FAKE + 1) == ALIGN

    def rest(act=1, x=FAKE, xs=FAKE, i=FAKE, f=FAKE, w=FAKE, T=4, k=2, cols=24, E=3):
        return (lib.dora_expert_send(act, x, i, f, T, k, cols, E, xs, None),
                lib.dora_expert_return(act, xs, i, f, w, T, k, cols, E, x, None),
                lib.dora_expert_return_bwd(act, x, xs, i, f, w, T, k, cols, E, xs, w, None))
    assert set(rest(act=5)) == {DTYPE}
    for bad in (dict(T=-1), dict(k=0), dict(cols=-1), dict(E=0), dict(T=1 << 30)):
        assert set(rest(**bad)) == {SHAPE}, bad
    assert set(rest(T=0)) == {OK}
    for bad in (dict(x=None), dict(xs=None), dict(i=None), dict(f=None)):
        assert set(rest(**bad)) == {NULL}, bad
    assert rest(w=None)[2] == NULL
    for bad in (dict(x=FAKE + 1), dict(xs=FAKE + 1), dict(i=FAKE + 2), dict(f=FAKE + 2)):
        assert set(rest(**bad)) == {ALIGN}, bad
    clear = lambda act=1, x=FAKE, f=FAKE, r=4, c=8, E=3: lib.dora_expert_clear(act, x, f, r, c, E, None)  # noqa: E731
    assert clear(act=9) == DTYPE and clear(r=-1) == SHAPE and clear(E=0) == SHAPE and clear(r=0) == OK
    assert clear(x=None) == NULL and clear(f=None) == NULL and clear(x=FAKE + 1) == ALIGN


# ---- ops while traced -------------------------------------------------------
def _fake(dtype, *shape):
    return torch.empty(*shape, device="cuda", dtype=dtype)


LAYER = dict(x=(BF, 6, 64), wq=(U8, 144, 32), wscale=(U8, 144, 2), A=(F32, 24, 64), B=(F32, 144, 24), m=(F32, 144),
             g=(F32, 144), norm=(F32, 144))


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("name,value", [
    ("x", (F32, 6, 64)), ("x", (BF, 6, 32)), ("x", (BF, 384)), ("wq", (F32, 144, 32)), ("wq", (U8, 136, 32)), ("wq", (U8, 144, 24)),
    ("wscale", (U8, 144, 1)), ("A", (F32, 24, 32)), ("B", (F32, 144, 16)), ("g", (F32, 143)), ("g", (BF, 144)),
])
def test_layer_arguments_are_refused_while_traced(name, value, grad):
    with FakeTensorMode():
        d = {k: _fake(*v) for k, v in dict(LAYER, **{name: value}).items()}
        d["B"].requires_grad_(grad)
        with pytest.raises((TypeError, ValueError), match="linear_q4"):
            ops.dora_linear_q4(**d, s=2.0)


def test_layer_shapes_while_traced():
    with FakeTensorMode():
        d = {k: _fake(*v) for k, v in LAYER.items()}
        assert ops.dora_linear_q4(**d, s=2.0).shape == (6, 144)
        d["A"].requires_grad_(True)
        assert ops.dora_linear_q4(**d, s=2.0).shape == (6, 144)
        d["A"] = _fake(F32, 12, 64).requires_grad_(True)
        d["B"] = _fake(F32, 144, 12)
        with pytest.raises(ValueError, match="rank"):
            ops.dora_linear_q4(**d, s=2.0)


def test_experts_while_traced():
    with FakeTensorMode():
        x, w = _fake(BF, 6, 64), _fake(F32, 6, 2)
        e, wq, ws = _fake(torch.int64, 6, 2), _fake(U8, 3, 144, 32), _fake(U8, 3, 144, 2)
        y = ops.experts_q4(x, e, w, wq, ws)
        assert y.shape == (6, 144) and y.dtype == BF
        for bad in (dict(wq=wq[0]), dict(weight=_fake(F32, 6, 3)), dict(expert=_fake(torch.int64, 6)), dict(x=_fake(BF, 5, 64))):
            with pytest.raises(ValueError, match="experts_q4"):
                ops.experts_q4(**dict(dict(x=x, expert=e, weight=w, wq=wq, wscale=ws), **bad))
        order, inverse, offsets = ops.expert_sort(e, 3)
        assert (order.shape, inverse.shape, offsets.shape) == ((12,), (6, 2), (4,)) and order.dtype == I32
        q, s = ops.q4_store(_fake(F32, 3, 144, 64))
        assert q.shape == (3, 144, 32) and s.shape == (3, 144, 2) and ops.q4_load(q, s, BF).shape == (3, 144, 64)
