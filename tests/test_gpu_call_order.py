"""A result is a function of the call alone: d_mag's bits do not depend on which
calls ran before in the process.

The grid of the compose backward, and with it the order of d_mag's sum, comes
from how many blocks of the kernel an SM holds.  That number belongs to one
kernel: the form for whole 16-byte pieces and the one for ragged rows hold
different numbers, and neither may plan with the other's.  Each order of calls
runs in a process of its own, as the numbers are looked up once per process.
"""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# prints a digest of d_mag for each width, in the order of the widths given
CHILD = """
import hashlib, sys, torch
import parameter_efficient_fine_gb300 as dora
T, act = 4000, getattr(torch, sys.argv[1])
for out in map(int, sys.argv[2:]):
    gen = torch.Generator(device="cuda").manual_seed(out)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    dy, base, lora = (rnd(T, out).to(act) for _ in range(3))
    g, n = rnd(out), rnd(out).abs() + 0.5
    q, sc = torch.empty(T, out, dtype=torch.uint8, device="cuda"), torch.empty(T, -(-out // 128), dtype=torch.uint8, device="cuda")
    y, db, dl, dm = torch.empty_like(dy), torch.empty_like(dy), torch.empty_like(dy), torch.empty(3, out, device="cuda")
    dora.dora_compose_fwd_q8(base, lora, g, 0.5, y, q, sc)
    ws = torch.empty(dora.dora_compose_bwd_workspace(T, out), dtype=torch.uint8, device="cuda")
    dora.dora_compose_bwd(dy, base, lora, g, n, 0.5, db, dl, dm[0], ws)
    dora.dora_compose_bwd_noalloc(dy, base, lora, g, n, 0.5, db, dl, dm[1])
    ws = torch.empty(dora.dora_compose_bwd_q8_workspace(T, out), dtype=torch.uint8, device="cuda")
    dora.dora_compose_bwd_q8(dy, q, sc, g, n, 0.5, db, dl, dm[2], ws)
    assert torch.equal(dm[0], dm[1])
    print(out, *(hashlib.sha256(v.cpu().numpy().tobytes()).hexdigest() for v in dm))
"""


def _digests(act, *widths):
    res = subprocess.run([sys.executable, "-c", CHILD, act, *map(str, widths)], cwd=ROOT, capture_output=True, text=True,
                         timeout=300)
    assert res.returncode == 0, res.stderr
    return sorted(res.stdout.splitlines())


@pytest.mark.parametrize("act", ["bfloat16", "float32"])
def test_d_mag_does_not_depend_on_the_calls_before(act):
    aligned, ragged = 1024, 1001
    first = _digests(act, aligned, ragged)
    assert len(first) == 2 and first == _digests(act, ragged, aligned)
