"""The binding's refusals for the 8-bit calls that the C entry points cannot
make themselves (CPU only: no compute call is made)."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import parameter_efficient_fine_gb300 as dora
from parameter_efficient_fine_gb300 import ops

U8 = torch.uint8


@pytest.mark.parametrize("block_rows", [0, -1, 2, 64, 1 << 32, (1 << 32) + 1, (1 << 32) + 128])
def test_a_block_of_other_rows_is_refused(block_rows):
    """Past 32 bits too: the C argument is an int, and (1 << 32) + 1 would arrive as 1
    with a scale of any size."""
    x = torch.zeros(300, 256)
    q, sc = torch.zeros(300, 256, dtype=U8), torch.zeros(1, 1, dtype=U8)
    with pytest.raises(ValueError, match="rows a scale"):
        dora.dora_q8_store(x, block_rows, q, sc, stream=0)
    with pytest.raises(ValueError, match="rows a scale"):
        dora.dora_q8_load(q, sc, block_rows, x, stream=0)
    with FakeTensorMode(), pytest.raises(ValueError, match="rows a scale"):
        ops.q8_store(torch.empty(300, 256, device="cuda"), block_rows)


def test_a_workspace_that_is_no_memory_of_its_size_is_refused():
    """An expanded tensor counts more elements than it has memory."""
    bf = torch.bfloat16
    q, sc, dy, g = torch.zeros(64, 256, dtype=U8), torch.zeros(64, 2, dtype=U8), torch.zeros(64, 256, dtype=bf), torch.ones(256)
    ws = torch.zeros(1, dtype=U8).expand(1 << 30)
    with pytest.raises(ValueError, match="contiguous"):
        dora.dora_compose_bwd_q8(dy, q, sc, g, g, 1.0, dy.clone(), dy.clone(), g.clone(), ws, stream=0)
    with pytest.raises(ValueError, match="contiguous"):
        dora.dora_lora_grad_q8(torch.zeros(64, 8, dtype=bf), q, sc, torch.zeros(8, 256), ws, stream=0)


class On:
    """A tensor that says it lies on a device; its address is never read."""

    def __init__(self, device, dtype, *shape):
        self.t, self.index, self.is_cuda = torch.empty(*shape, dtype=dtype, device="meta"), device, True

    def __getattr__(self, name):
        return getattr(self.t, name)

    def get_device(self):
        return self.index

    def data_ptr(self):
        return 1 << 20


CALLS = {   # the tensors of each call, and the rest of its arguments in their places
    "dora_q8_store": lambda t, u8, bf, f32: (t(bf, 4, 256), 1, t(u8, 4, 256), t(u8, 4, 2)),
    "dora_q8_load": lambda t, u8, bf, f32: (t(u8, 4, 256), t(u8, 4, 2), 1, t(bf, 4, 256)),
    "dora_compose_fwd_q8": lambda t, u8, bf, f32: (t(bf, 4, 256), t(bf, 4, 256), t(f32, 256), 1.0, t(bf, 4, 256),
                                                   t(u8, 4, 256), t(u8, 4, 2)),
    "dora_compose_bwd_q8": lambda t, u8, bf, f32: (t(bf, 4, 256), t(u8, 4, 256), t(u8, 4, 2), t(f32, 256), t(f32, 256),
                                                   1.0, t(bf, 4, 256), t(bf, 4, 256), t(f32, 256), t(u8, 4096)),
    "dora_lora_grad_q8": lambda t, u8, bf, f32: (t(bf, 4, 8), t(u8, 4, 256), t(u8, 4, 2), t(f32, 8, 256), t(u8, 4096)),
    "dora_matmul_q8": lambda t, u8, bf, f32: (t(u8, 4, 256), t(u8, 4, 2), t(u8, 128, 256), t(u8, 1, 2), t(bf, 4, 128)),
    "dora_matmul_q8_t": lambda t, u8, bf, f32: (t(u8, 4, 128), t(u8, 4, 1), t(u8, 128, 256), t(u8, 1, 2), t(bf, 4, 256)),
}


@pytest.mark.parametrize("name", CALLS)
def test_tensors_of_another_device_are_refused(name, monkeypatch):
    """The kernels run on the current device; another one's memory is not theirs to touch."""
    reached = []

    class Library:
        def __getattr__(self, entry):
            return lambda *a: reached.append(entry) or 0
    monkeypatch.setattr(dora, "load_library", Library)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)

    def call(odd, device):
        """The call with tensor number `odd` (all where None) on `device`, the others on cuda:0."""
        seen = iter(range(100))
        args = CALLS[name](lambda dt, *s: On(device if odd in (None, next(seen)) else 0, dt, *s), U8, torch.bfloat16,
                           torch.float32)
        getattr(dora, name)(*args, stream=0)
        return sum(isinstance(a, On) for a in args)

    n = call(None, 0)
    assert reached == [name] and n >= 3
    for odd in (None, *range(n)):
        with pytest.raises(ValueError, match="cuda:1"):
            call(odd, 1)
    assert reached == [name]
