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
