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
