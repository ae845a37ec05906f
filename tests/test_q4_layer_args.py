"""What the layer on a 4-bit weight and the operators under it refuse is refused alike with
and without gradients, and while a model is traced; on the CPU."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

from parameter_efficient_fine_gb300 import ops

BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8
LAYER = dict(x=(BF, 6, 64), wq=(U8, 144, 32), wscale=(U8, 144, 2), A=(F32, 24, 64), B=(F32, 144, 24), m=(F32, 144),
             g=(F32, 144), norm=(F32, 144))


def _fake(dtype, *shape):
    return torch.empty(*shape, device="cuda", dtype=dtype)


@pytest.mark.parametrize("grad", [None, "x", "B", "m"])
@pytest.mark.parametrize("name,value", [("m", (F32, 143)), ("m", (F32, 144, 1)), ("m", (F32, 1)), ("norm", (F32, 143)),
                                        ("norm", (BF, 144)), ("norm", (F32, 144, 1))])
def test_m_and_norm_are_refused_with_and_without_gradients(name, value, grad):
    with FakeTensorMode():
        d = {k: _fake(*v) for k, v in dict(LAYER, **{name: value}).items()}
        if grad:
            d[grad].requires_grad_(True)
        with pytest.raises(ValueError, match=f"linear_q4: {name} is"):
            ops.dora_linear_q4(**d, s=2.0)


# ---- the operators while traced: what the eager call refuses, by the same checks ----
I32, I64 = torch.int32, torch.int64
PLAIN = dict(x=(BF, 5, 64), wq=(U8, 48, 32), wscale=(U8, 48, 2), offsets=None)
STACK = dict(x=(BF, 5, 64), wq=(U8, 3, 48, 32), wscale=(U8, 3, 48, 2), offsets=(I32, 4))


def _tensors(base, change):
    return {k: v and _fake(*v) for k, v in dict(base, **change).items()}


@pytest.mark.parametrize("base,change", [
    (PLAIN, dict(x=(F32, 5, 64))), (PLAIN, dict(x=(BF, 5, 32))), (PLAIN, dict(x=(BF, 320))), (PLAIN, dict(wscale=(U8, 48, 1))),
    (PLAIN, dict(wq=(BF, 48, 32))), (PLAIN, dict(wq=(U8, 48, 24))), (PLAIN, dict(wq=(U8, 3, 48, 32))), (PLAIN, dict(wq=(U8, 32))),
    (PLAIN, dict(offsets=(I32, 2))), (STACK, dict(offsets=None)), (STACK, dict(offsets=(I32, 3))), (STACK, dict(offsets=(I64, 4))),
    (STACK, dict(wscale=(U8, 48, 2))), (PLAIN, dict(wscale=(F32, 48, 2))),
])
def test_products_are_refused_while_traced(base, change):
    with FakeTensorMode():
        d = _tensors(base, change)
        with pytest.raises((TypeError, ValueError), match="matmul_q4"):
            ops.matmul_q4(d["x"], d["wq"], d["wscale"], d["offsets"])
    if "x" in change and change["x"][1:] != (5, 64):
        change = dict(change, x=(change["x"][0], *(48 if n == 64 else n for n in change["x"][1:])))
    base = dict(base, x=(BF, 5, 48))
    if change.get("x") == (F32, 5, 64):
        change = dict(x=(F32, 5, 48))
    with FakeTensorMode():
        d = _tensors(base, change)
        with pytest.raises((TypeError, ValueError), match="matmul_q4_t"):
            ops.matmul_q4_t(d["x"], d["wq"], d["wscale"], d["offsets"])


def test_what_the_library_refuses_is_refused_while_traced():
    with FakeTensorMode():
        wq, ws = _fake(U8, 40, 32), _fake(U8, 40, 2)
        for call in (lambda: ops.matmul_q4(_fake(BF, 5, 64), wq, ws), lambda: ops.matmul_q4_t(_fake(BF, 5, 40), wq, ws)):
            with pytest.raises(ValueError, match="matmul_q4.*multiple of 16"):
                call()
        d = _tensors(STACK, dict(wq=(U8, 4097, 48, 32), wscale=(U8, 4097, 48, 2), offsets=(I32, 4098)))
        with pytest.raises(ValueError, match="matmul_q4.*experts"):
            ops.matmul_q4(**d)


def test_products_while_traced():
    with FakeTensorMode():
        for base in (PLAIN, STACK):
            d = _tensors(base, {})
            assert ops.matmul_q4(**d).shape == (5, 48)
            d["x"] = _fake(BF, 5, 48)
            y = ops.matmul_q4_t(d["x"], d["wq"], d["wscale"], d["offsets"])
            assert y.shape == (5, 64) and y.dtype == BF


@pytest.mark.parametrize("q,scale,dtype", [((U8, 4, 32), (U8, 4, 1), BF), ((BF, 4, 32), (U8, 4, 2), BF), ((U8, 4, 24), (U8, 4, 1), BF),
                                           ((U8, 32), (U8, 2), BF), ((U8, 4, 32), (U8, 4, 2), torch.float16)])
def test_forms_are_refused_while_traced(q, scale, dtype):
    with FakeTensorMode(), pytest.raises((TypeError, ValueError), match="q4_load|dtype"):
        ops.q4_load(_fake(*q), _fake(*scale), dtype)


@pytest.mark.parametrize("x", [(torch.float16, 4, 64), (U8, 4, 64)])
def test_types_that_have_no_form_are_refused_while_traced(x):
    with FakeTensorMode(), pytest.raises(TypeError, match="dtype"):
        ops.q4_store(_fake(*x))


@pytest.mark.parametrize("expert,experts", [((torch.int16, 4, 2), 3), ((I32, 4, 2), 0), ((I32, 4, 2), 4097), ((I32, 8), 3)])
def test_sorts_are_refused_while_traced(expert, experts):
    with FakeTensorMode(), pytest.raises((TypeError, ValueError), match="expert_sort"):
        ops.expert_sort(_fake(*expert), experts)


ROUTE = dict(x=(BF, 4, 24), xs=(BF, 8, 24), inverse=(I32, 4, 2), offsets=(I32, 4), weight=(F32, 4, 2))


@pytest.mark.parametrize("change", [dict(x=(BF, 5, 24), xs=(BF, 7, 24)), dict(inverse=(I64, 4, 2)), dict(offsets=(I32, 1)), dict(offsets=(I64, 4)),
                                    dict(offsets=(I32, 2, 2)), dict(inverse=(I32, 8)), dict(x=(torch.float16, 4, 24), xs=(torch.float16, 8, 24))])
def test_routes_are_refused_while_traced(change):
    with FakeTensorMode():
        d = _tensors(ROUTE, change)
        for match, call in (("expert_send", lambda: ops.expert_send(d["x"], d["inverse"], d["offsets"])),
                            ("expert_return", lambda: ops.expert_return(d["xs"], d["inverse"], d["offsets"], d["weight"])),
                            ("expert_return_bwd", lambda: ops.expert_return_bwd(d["x"], d["xs"], d["inverse"], d["offsets"], d["weight"]))):
            with pytest.raises((TypeError, ValueError), match=match + "|dtype"):
                call()


@pytest.mark.parametrize("weight", [(F32, 4, 3), (BF, 4, 2), (F32, 8)])
def test_weights_are_refused_while_traced(weight):
    with FakeTensorMode():
        d = _tensors(ROUTE, dict(weight=weight))
        with pytest.raises(ValueError, match="expert_return"):
            ops.expert_return(d["xs"], d["inverse"], d["offsets"], d["weight"])
        with pytest.raises(ValueError, match="expert_return_bwd"):
            ops.expert_return_bwd(d["x"], d["xs"], d["inverse"], d["offsets"], d["weight"])
