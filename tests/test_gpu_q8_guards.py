"""Out-of-bounds write checks of the 8-bit store, load and compose at odd sizes
and odd addresses: each output is the middle of an allocation filled with a
sentinel, and may begin `by` elements past an aligned address, so the kernels
for ragged rows write next to sentinels on both sides.  The results have to be
those of ordinary buffers."""
import pytest
import torch

import parameter_efficient_fine_gb300 as dora

from gpu_util import DEV, assert_no_device_error
from test_gpu_guards import Guarded

pytestmark = pytest.mark.gpu

U8 = torch.uint8
SIZES = [(1, 1), (33, 1003), (130, 17), (257, 136), (300, 520), (9, 2048)]
DTYPES = [torch.bfloat16, torch.float32]


def guarded(dtype, *shape, by=0):
    """(buffer, view) of a guarded matrix that begins `by` elements past an aligned address."""
    size = torch.empty(0, dtype=dtype).element_size()
    n = size
    for d in shape:
        n *= d
    buf = Guarded(n + by * size)
    buf.lo, buf.nbytes = buf.lo + by * size, n
    buf.inner = buf.raw[buf.lo:buf.lo + n]
    return buf, buf.view(dtype, shape)


def run(make, T, out, dtype, by, block_rows):
    """Every output of a store, a load and a compose step, in buffers from `make`."""
    gen = torch.Generator(device=DEV).manual_seed(T + out)
    base, lora, dy = (torch.randn(T, out, generator=gen, device=DEV).to(dtype) for _ in range(3))
    g, n = (torch.rand(out, generator=gen, device=DEV) + 0.5 for _ in range(2))
    nsc = -(-out // 128)
    names = {"q": (U8, T, out), "scale": (U8, -(-T // block_rows), nsc), "x": (dtype, T, out), "y": (dtype, T, out),
             "vq": (U8, T, out), "vscale": (U8, T, nsc), "d_base": (dtype, T, out), "d_lora": (dtype, T, out),
             "d_mag": (torch.float32, out)}
    b = {k: make(*v, by=by + i % 2) for i, (k, v) in enumerate(names.items())}
    size = dora.dora_compose_bwd_q8_workspace(T, out)
    b["workspace"] = make(U8, size)
    v8 = torch.empty(T, out, device=DEV)
    v = {k: view for k, (_, view) in b.items()}
    dora.dora_q8_store(base, block_rows, v["q"], v["scale"])
    dora.dora_q8_load(v["q"], v["scale"], block_rows, v["x"])
    dora.dora_compose_fwd_q8(base, lora, g, 0.75, v["y"], v["vq"], v["vscale"])
    dora.dora_compose_bwd_q8(dy, v["vq"], v["vscale"], g, n, 0.75, v["d_base"], v["d_lora"], v["d_mag"], v["workspace"])
    dora.dora_q8_load(v["vq"], v["vscale"], 1, v8)
    assert_no_device_error()
    return b, (dy.double().abs() * v8.double().abs()).sum(0) / n.double()


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("by", [0, 1, 3])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,out", SIZES)
def test_writes_stay_in_bounds_at_any_address(T, out, dtype, by, block_rows):
    got, size = run(guarded, T, out, dtype, by, block_rows)
    ref, _ = run(lambda dt, *shape, by=0: (None, torch.full(shape, 0x5a, dtype=dt, device=DEV)), T, out, dtype, 0,
                 block_rows)
    for k, (buf, view) in got.items():
        buf.check(k)
        if k == "d_mag":      # an aligned and a ragged call sum the tokens in another order: T + 16 fp32 additions each
            err = (view.double() - ref[k][1].double()).abs()
            assert (err <= 2 * 2.0 ** -24 * (T + 16) * size).all()
        elif k != "workspace":
            assert torch.equal(view, ref[k][1]), k
