"""The failure path of the 8-bit kernels that tests/test_gpu_q8_layer.py leaves
out: dy W on both of its kernels, and the gradient of A with a tile wide enough
that conversion warps wait for dxa.  With their loads withheld, the kernels'
waits give up after a short limit set here, record a code and leave the
context usable: the next call gives the bits of the one before."""
import pytest
import torch

import parameter_efficient_fine_gb300 as dora
from parameter_efficient_fine_gb300 import ops

from gpu_util import DEV, assert_no_device_error

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("call,T", [("matmul_q8_t", 1), ("matmul_q8_t", 20), ("matmul_q8_t", 128), ("matmul_q8_t", 300),
                                    ("matmul_q8_t", 2000), ("grad", 100), ("grad", 900)])
def test_withheld_loads_end_in_an_error(call, T):
    gen = torch.Generator(device=DEV).manual_seed(T)
    rnd = lambda *s: torch.randn(*s, generator=gen, device=DEV)  # noqa: E731
    if call == "grad":
        q, sc = ops.q8_store(rnd(T, 1040), 1)
        dxa, res = rnd(T, 160).bfloat16(), torch.empty(160, 1040, device=DEV)
        ws = torch.empty(dora.dora_lora_grad_q8_workspace(T, 1040, 160), dtype=torch.uint8, device=DEV)
        run = lambda: dora.dora_lora_grad_q8(dxa, q, sc, res, ws)  # noqa: E731
    else:
        q, sc = ops.q8_store(rnd(T, 528), 1)
        wq, wsc = ops.q8_store(rnd(528, 2576), 128)
        res = torch.empty(T, 2576, device=DEV, dtype=torch.bfloat16)
        run = lambda: dora.dora_matmul_q8_t(q, sc, wq, wsc, res)  # noqa: E731
    run()
    good = res.clone()
    assert_no_device_error()
    dora.dora_test_stall_loads(True, 20_000_000)      # 20 ms
    try:
        run()
        code = dora.dora_device_error()               # synchronises
    finally:
        dora.dora_test_stall_loads(False)
    assert code != 0
    run()
    assert_no_device_error()
    assert torch.equal(res, good)
