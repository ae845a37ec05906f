"""What the layer on an 8-bit weight does not take is refused by the call
itself, eagerly and while it is traced, not later in its backward."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

from parameter_efficient_fine_gb300 import ops

T, OUT, IN, R = 6, 144, 272, 24


def _args(make, r=R, **change):
    """The layer's arguments; `change` gives one of them other sizes or another type."""
    bf, f32, u8 = torch.bfloat16, torch.float32, torch.uint8
    d = dict(x=(bf, T, IN), wq=(u8, OUT, IN), wscale=(u8, 2, 3), A=(f32, r, IN), B=(f32, OUT, r), m=(f32, OUT),
             g=(f32, OUT), norm=(f32, OUT))
    d.update(change)
    return dict({k: make(v[0], *v[1:]) for k, v in d.items()}, s=2.0)


def _fake(dtype, *shape):
    return torch.empty(*shape, device="cuda", dtype=dtype)


REFUSED = [
    ("x", (torch.float32, T, IN)), ("x", (torch.float16, T, IN)), ("x", (torch.bfloat16, T, IN - 16)),
    ("x", (torch.bfloat16, T * IN)), ("wq", (torch.float32, OUT, IN)), ("wq", (torch.uint8, OUT - 8, IN)),
    ("wscale", (torch.uint8, 2, 2)), ("wscale", (torch.uint8, OUT, 3)), ("A", (torch.float32, R + 8, IN)),
    ("A", (torch.float32, R, IN - 16)), ("B", (torch.float32, OUT + 16, R)), ("g", (torch.float32, OUT - 1)),
    ("g", (torch.bfloat16, OUT)),
]


@pytest.mark.parametrize("name,value", REFUSED)
def test_wrong_arguments_are_refused_while_traced(name, value):
    with FakeTensorMode():
        with pytest.raises((TypeError, ValueError), match="linear_q8"):
            ops.dora_linear_q8(**_args(_fake, **{name: value}))


def test_features_that_are_no_multiple_of_16_are_refused_while_traced():
    with FakeTensorMode():
        for change in (dict(x=(torch.bfloat16, T, 264), wq=(torch.uint8, OUT, 264), A=(torch.float32, R, 264)),
                       dict(wq=(torch.uint8, 136, IN), B=(torch.float32, 136, R), m=(torch.float32, 136),
                            g=(torch.float32, 136), norm=(torch.float32, 136))):
            with pytest.raises(ValueError, match="linear_q8"):
                ops.dora_linear_q8(**_args(_fake, **change))


@pytest.mark.parametrize("r", [4, 12, 1032])
def test_a_rank_without_a_gradient_of_A_is_refused_by_the_forward(r):
    with FakeTensorMode():
        d = _args(_fake, r=r)
        assert ops.dora_linear_q8(**d).shape == (T, OUT)         # its output needs no such rank
        d["x"].requires_grad_(True)
        ops.dora_linear_q8(**d)                                  # nor does the gradient of x
        d["A"].requires_grad_(True)
        with torch.no_grad():
            ops.dora_linear_q8(**d)
        with pytest.raises(ValueError, match="rank"):
            ops.dora_linear_q8(**d)


@pytest.mark.parametrize("name,value", [("m", (torch.float32, OUT, 1)), ("norm", (torch.bfloat16, OUT)),
                                        ("norm", (torch.float32, OUT - 16))])
def test_what_only_the_backward_reads_is_checked_by_the_forward(name, value):
    with FakeTensorMode():
        d = _args(_fake, **{name: value})
        ops.dora_linear_q8(**d)
        d["m"].requires_grad_(True)
        with pytest.raises(ValueError, match="linear_q8"):
            ops.dora_linear_q8(**d)


@pytest.mark.gpu
@pytest.mark.parametrize("name,value", REFUSED)
def test_wrong_arguments_are_refused(name, value):
    make = lambda dt, *s: torch.ones(*s, dtype=dt, device="cuda")  # noqa: E731
    with pytest.raises((TypeError, ValueError), match="linear_q8"):
        ops.dora_linear_q8(**_args(make, **{name: value}))


@pytest.mark.gpu
@pytest.mark.parametrize("r", [4, 12])
def test_any_rank_where_A_needs_no_gradient(r):
    gen = torch.Generator(device="cuda").manual_seed(r)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    wq, wscale = ops.q8_store(rnd(OUT, IN) / 16, 128)
    d = dict(x=rnd(T, IN).bfloat16().requires_grad_(True), wq=wq, wscale=wscale, A=rnd(r, IN) / 16, B=rnd(OUT, r),
             m=rnd(OUT), g=rnd(OUT), norm=rnd(OUT).abs() + 1, s=2.0)
    dy = rnd(T, OUT).bfloat16()
    y = ops.dora_linear_q8(**d)
    y.backward(dy)
    # the same layer with zero rows added to A and columns to B, to a rank that a gradient of A could take
    z = dict(d, x=d["x"].detach().clone().requires_grad_(True), A=torch.zeros(16, IN, device="cuda"),
             B=torch.zeros(OUT, 16, device="cuda"))
    z["A"][:r], z["B"][:, :r] = d["A"], d["B"]
    w = ops.dora_linear_q8(**z)
    w.backward(dy)
    for a, b in ((y, w), (d["x"].grad, z["x"].grad)):           # bf16 products over other lengths: a rounding apart
        torch.testing.assert_close(a, b, rtol=2.0 ** -5, atol=2.0 ** -5 * float(b.detach().float().abs().max()))
    z["A"].requires_grad_(True)
    ops.dora_linear_q8(**z).backward(dy)
    d["A"].requires_grad_(True)
    with pytest.raises(ValueError, match="rank"):
        ops.dora_linear_q8(**d)
