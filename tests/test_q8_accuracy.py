"""How far the 8-bit products may be from their definition: the norm of a row's error.

An element-wise worst-case bound over K additions is tens of times a result's
rounding at K = 8192 and so passes sums that are held in too few bits.  The norm
does not: y is an fp32 sum rounded once to bf16 (8 significant bits).  The
rounding error of a value in [2^e, 2^(e+1)) is uniform in +-2^(e-8), which is
2^(e-8) / sqrt(3) in the root of the mean square, and over mantissas that are
spread evenly 2^e is 0.65 of the value's: 0.38 2^-8 of a row's norm, with 0.55
2^-8 = 1.1 2^-9 as the bound.  The sum itself adds far less: K / 32 matrix
instructions that each drop at most 2^-23 of the running sum, which for random
terms is no larger than some times the result, 2^-14 at K = 14336.

A sum held in 14 bits is seen: 256 steps that each drop half of 2^-13 of it on
the mean are about 2^-6.
"""
import numpy as np
import pytest
import torch

BOUND = 1.1 * 2.0 ** -9


def row_errors(got, ref):
    """Norm of the error over the norm of the value, row by row."""
    return np.linalg.norm(got - ref, axis=1) / np.linalg.norm(ref, axis=1)


def _truncate(v, bits):
    """v with its lower significant bits dropped, toward zero."""
    m, e = np.frexp(v)
    return np.ldexp(np.trunc(np.ldexp(m, bits)), e - bits)


def _bf16(v):
    return torch.from_numpy(v).float().bfloat16().double().numpy()


@pytest.mark.parametrize("bits,passes", [(24, True), (22, True), (14, False)])
def test_the_bound_sees_a_sum_held_in_few_bits(bits, passes):
    rng = np.random.default_rng(bits)
    K = 8192
    x, w = rng.standard_normal((4, K)), rng.standard_normal((512, K))
    acc = np.zeros((4, 512))
    for k in range(0, K, 32):
        acc = _truncate(acc + x[:, k:k + 32] @ w[:, k:k + 32].T, bits)
    assert bool((row_errors(_bf16(acc), x @ w.T) <= BOUND).all()) == passes


@pytest.mark.gpu
@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("T,feat,k", [(1, 1024, 8192), (37, 512, 14336), (128, 1040, 4096), (129, 784, 8192),
                                      (300, 2064, 2064), (2000, 1024, 14336)])
def test_products(T, feat, k, trans):
    import parameter_efficient_fine_gb300 as dora
    from gpu_util import DEV, assert_no_device_error
    from parameter_efficient_fine_gb300 import ops
    gen = torch.Generator(device=DEV).manual_seed(T + feat + k)
    q, sc = ops.q8_store(torch.randn(T, k, generator=gen, device=DEV), 1)
    wq, wsc = ops.q8_store(torch.randn(*((k, feat) if trans else (feat, k)), generator=gen, device=DEV), 128)
    y = torch.empty(T, feat, dtype=torch.bfloat16, device=DEV)
    (dora.dora_matmul_q8_t if trans else dora.dora_matmul_q8)(q, sc, wq, wsc, y)
    x, w = (ops.q8_load(*form, torch.float32).double() for form in ((q, sc, 1), (wq, wsc, 128)))
    assert_no_device_error()
    ref = x @ (w if trans else w.t())
    assert (row_errors(y.double().cpu().numpy(), ref.cpu().numpy()) <= BOUND).all()
