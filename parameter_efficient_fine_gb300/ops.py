"""torch.library registration of the DoRA hot path (integration only).

The custom ops; each allocates its outputs (and the library's workspace)
with torch and calls the C entry points of the same names on the current CUDA
stream.  No arithmetic happens here but the low-rank products of linear_q8 and
linear_q4 and of their backward, which are torch's:

  torch.ops.dora.norm_factored(W0, A, B, m, s) -> (norm, g)
  torch.ops.dora.row_sumsq(W0) -> n0sq                       (bf16 W0: ||W0_i||^2, once)
  torch.ops.dora.norm_factored_bf16(W0, A, B, m, n0sq, s) -> (norm, g)   (bf16 W0, A, B)
  torch.ops.dora.compose(base, lora, m, g, norm, s) -> y
  torch.ops.dora.compose_bwd(dy, base, lora, g, norm, s) -> (d_base, d_lora, d_mag)
  torch.ops.dora.norm_factored_bwd(W0, A, B, norm, g, d_mag, s) -> (dA, dB)   (through the norm)
  torch.ops.dora.module(base, lora, W0, A, B, m, s) -> (y, norm, g)           (norm not detached)
  torch.ops.dora.q8_store(x, block_rows) -> (q, scale)         (x in 8 bits: E4M3, a scale per 128)
  torch.ops.dora.q8_load(q, scale, block_rows, dtype) -> x
  torch.ops.dora.compose_q8(base, lora, m, g, norm, s) -> (y, vq, vscale)     (v = base + s lora in 8 bits)
  torch.ops.dora.compose_bwd_q8(dy, vq, vscale, g, norm, s) -> (d_base, d_lora, d_mag)
  torch.ops.dora.matmul_q8(xq, xscale, wq, wscale) -> y        (x W^T, both in 8 bits)
  torch.ops.dora.matmul_q8_t(dyq, dyscale, wq, wscale) -> dx   (dy W)
  torch.ops.dora.lora_grad_q8(dxa, xq, xscale) -> dA           (dxa^T x)
  torch.ops.dora.linear_q8(x, wq, wscale, A, B, m, g, norm, s) -> (y, ...)    (the layer on those)
  torch.ops.dora.q4_store(x) -> (q, scale)                     (x in 4 bits: E2M1, a scale per 32)
  torch.ops.dora.q4_load(q, scale, dtype) -> x
  torch.ops.dora.matmul_q4(x, wq, wscale, offsets) -> y        (x W^T, W in 4 bits, or by expert)
  torch.ops.dora.matmul_q4_t(dy, wq, wscale, offsets) -> dx    (dy W)
  torch.ops.dora.linear_q4(x, wq, wscale, A, B, m, g, norm, s) -> (y, ...)    (the layer on those)
  torch.ops.dora.expert_sort(expert, experts) -> (order, inverse, offsets)
  torch.ops.dora.expert_send(x, inverse, offsets) -> xs        (tokens' rows by expert)
  torch.ops.dora.expert_return(ys, inverse, offsets, weight) -> y             (their weighted sums)
  torch.ops.dora.expert_return_bwd(dy, ys, inverse, offsets, weight) -> (d_ys, d_weight)

``compose`` is differentiable in base, lora and m.  It takes m beside g (the
norm op's output g = m / norm) so that autograd can deliver dL/dm: with the
row norm treated as a constant in the backward (the method's page,
"人工智能训练新突破：Anthropic团队破解大模型微调内存瓶颈难题", says nothing about a
gradient through the norm; this is the reading the library follows),
dL/dm_j = sum_t dy_tj (base_tj + s lora_tj) / norm_j, which is exactly the
library's d_mag, and dL/dbase = g dy, dL/dlora = s g dy are its d_base and
d_lora.  The backward is therefore one call of dora_compose_bwd.

``module`` is the variant with the norm NOT detached: differentiable in base,
lora, A, B and m.  Its backward is one dora_compose_bwd call followed, when A
or B needs a gradient, by one dora_norm_factored_bwd call on the d_mag it
returned (dL/dn = -g d_mag); its norm and g outputs are not differentiable.

``compose_q8`` is ``compose`` that keeps one byte an element for its backward
(v in 8 bits) instead of base and lora.  ``linear_q8`` is the whole layer on a
frozen weight in 8 bits: x goes into 8 bits once, feeds the base product from
there and stays there for the gradient of A; what it holds from forward to
backward is x and v in 8 bits and xa.  It is differentiable in x, A, B and m;
rounding to 8 bits passes gradients through unchanged, and dy g (the gradient
of base) is itself rounded to 8 bits for dx.

``matmul_q4`` is differentiable in x (its gradient is matmul_q4_t),
``expert_send`` in x and ``expert_return`` in ys and weight.  Rows of their
outputs that no expert has are 0.  ``linear_q4`` is ``linear_q8`` on a frozen
weight in 4 bits: its products take x and dy g as they are, in bfloat16; x and
v are kept in 8 bits as there.

Inputs must be contiguous, row-major and on one CUDA device (the C ABI's
layout); m, n0sq, norm and g are float32, the weights float32 (bfloat16 for
the _bf16 norm and row_sumsq), activations float32 or bfloat16.
"""
from __future__ import annotations

from typing import Optional

import torch
from torch import Tensor

from . import (_act, _expert_sort_sizes, _matmul_q4_sizes, _q4, _routed, _same, dora_compose_bwd, dora_compose_bwd_q8,
               dora_compose_bwd_q8_workspace, dora_compose_bwd_workspace, dora_compose_fwd, dora_compose_fwd_q8,
               dora_expert_clear, dora_expert_return, dora_expert_return_bwd, dora_expert_send, dora_expert_sort,
               dora_lora_grad_q8, dora_lora_grad_q8_workspace, dora_matmul_q4, dora_matmul_q4_t,
               dora_matmul_q4_t_workspace, dora_matmul_q4_workspace, dora_matmul_q8, dora_matmul_q8_t,
               dora_norm_factored, dora_norm_factored_bf16, dora_norm_factored_bf16_workspace, dora_norm_factored_bwd,
               dora_norm_factored_bwd_workspace, dora_norm_factored_workspace, dora_q4_load, dora_q4_store,
               dora_q8_load, dora_q8_store, dora_row_sumsq_bf16)

__all__ = ["norm_factored", "row_sumsq", "norm_factored_bf16", "compose", "compose_bwd", "norm_factored_bwd",
           "module", "dora_module", "q8_store", "q8_load", "compose_q8", "compose_bwd_q8", "matmul_q8", "matmul_q8_t",
           "lora_grad_q8", "linear_q8", "dora_linear_q8", "q4_store", "q4_load", "matmul_q4", "matmul_q4_t", "linear_q4",
           "dora_linear_q4", "expert_sort", "expert_send", "expert_return", "expert_return_bwd", "experts_q4"]


def _contig(name: str, *ts: Tensor) -> None:
    for t in ts:
        if not t.is_contiguous():
            raise ValueError(f"dora::{name}: inputs must be contiguous (row-major)")


@torch.library.custom_op("dora::norm_factored", mutates_args=(), device_types="cuda")
def norm_factored(W0: Tensor, A: Tensor, B: Tensor, m: Tensor, s: float) -> tuple[Tensor, Tensor]:
    """n_i = ||W0_i + s (B A)_i|| (factored: base + cross + Gram terms) and g = m / n."""
    _contig("norm_factored", W0, A, B, m)
    out, inp = W0.shape
    r = A.shape[0]
    norm = torch.empty(out, device=W0.device, dtype=torch.float32)
    g = torch.empty_like(norm)
    ws = torch.empty(max(dora_norm_factored_workspace(out, inp, r), 1), dtype=torch.uint8, device=W0.device)
    dora_norm_factored(W0, A, B, m, s, norm, g, ws)
    return norm, g


@norm_factored.register_fake
def _norm_factored_fake(W0, A, B, m, s):
    out = W0.shape[0]
    return W0.new_empty(out, dtype=torch.float32), W0.new_empty(out, dtype=torch.float32)


@torch.library.custom_op("dora::row_sumsq", mutates_args=(), device_types="cuda")
def row_sumsq(W0: Tensor) -> Tensor:
    """||W0_i||^2 of a bfloat16 W0 in fp32 (fixed summation order)."""
    _contig("row_sumsq", W0)
    n0sq = torch.empty(W0.shape[0], device=W0.device, dtype=torch.float32)
    dora_row_sumsq_bf16(W0, n0sq)
    return n0sq


@row_sumsq.register_fake
def _row_sumsq_fake(W0):
    return W0.new_empty(W0.shape[0], dtype=torch.float32)


@torch.library.custom_op("dora::norm_factored_bf16", mutates_args=(), device_types="cuda")
def norm_factored_bf16(W0: Tensor, A: Tensor, B: Tensor, m: Tensor, n0sq: Tensor, s: float) -> tuple[Tensor, Tensor]:
    """The factored norm for bfloat16 W0, A, B with ||W0_i||^2 given (n0sq)."""
    _contig("norm_factored_bf16", W0, A, B, m, n0sq)
    out, inp = W0.shape
    r = A.shape[0]
    norm = torch.empty(out, device=W0.device, dtype=torch.float32)
    g = torch.empty_like(norm)
    ws = torch.empty(max(dora_norm_factored_bf16_workspace(out, inp, r), 1), dtype=torch.uint8, device=W0.device)
    dora_norm_factored_bf16(W0, A, B, m, n0sq, s, norm, g, ws)
    return norm, g


@norm_factored_bf16.register_fake
def _norm_factored_bf16_fake(W0, A, B, m, n0sq, s):
    out = W0.shape[0]
    return W0.new_empty(out, dtype=torch.float32), W0.new_empty(out, dtype=torch.float32)


@torch.library.custom_op("dora::compose_bwd", mutates_args=(), device_types="cuda")
def compose_bwd(dy: Tensor, base: Tensor, lora: Tensor, g: Tensor, norm: Tensor,
                s: float) -> tuple[Tensor, Tensor, Tensor]:
    """d_base = g dy, d_lora = s g dy, d_mag = sum_t dy (base + s lora) / norm."""
    _contig("compose_bwd", dy, base, lora, g, norm)
    T, out = dy.shape
    d_base = torch.empty_like(dy)
    d_lora = torch.empty_like(dy)
    d_mag = torch.empty(out, device=dy.device, dtype=torch.float32)
    ws = torch.empty(max(dora_compose_bwd_workspace(T, out), 1), dtype=torch.uint8, device=dy.device)
    dora_compose_bwd(dy, base, lora, g, norm, s, d_base, d_lora, d_mag, ws)
    return d_base, d_lora, d_mag


@compose_bwd.register_fake
def _compose_bwd_fake(dy, base, lora, g, norm, s):
    return torch.empty_like(dy), torch.empty_like(dy), dy.new_empty(dy.shape[1], dtype=torch.float32)


@torch.library.custom_op("dora::compose", mutates_args=(), device_types="cuda")
def compose(base: Tensor, lora: Tensor, m: Tensor, g: Tensor, norm: Tensor, s: float) -> Tensor:
    """y = base + (g - 1) base + g s lora (fp32 inside, one rounding to the activation dtype)."""
    _contig("compose", base, lora, g)
    y = torch.empty_like(base)
    dora_compose_fwd(base, lora, g, s, y)
    return y


@compose.register_fake
def _compose_fake(base, lora, m, g, norm, s):
    return torch.empty_like(base)


def _compose_setup(ctx, inputs, output):
    base, lora, m, g, norm, s = inputs
    ctx.save_for_backward(base, lora, g, norm)
    ctx.s = s


def _compose_backward(ctx, dy):
    base, lora, g, norm = ctx.saved_tensors
    d_base, d_lora, d_mag = compose_bwd(dy.contiguous(), base, lora, g, norm, ctx.s)
    return d_base, d_lora, d_mag, None, None, None


compose.register_autograd(_compose_backward, setup_context=_compose_setup)


@torch.library.custom_op("dora::norm_factored_bwd", mutates_args=(), device_types="cuda")
def norm_factored_bwd(W0: Tensor, A: Tensor, B: Tensor, norm: Tensor, g: Tensor, d_mag: Tensor,
                      s: float) -> tuple[Tensor, Tensor]:
    """dA, dB through the row norm for dL/dn = -g d_mag (d_mag as compose_bwd returns it)."""
    _contig("norm_factored_bwd", W0, A, B, norm, g, d_mag)
    out, inp = W0.shape
    r = A.shape[0]
    dA = torch.empty(r, inp, device=W0.device, dtype=torch.float32)
    dB = torch.empty(out, r, device=W0.device, dtype=torch.float32)
    ws = torch.empty(max(dora_norm_factored_bwd_workspace(out, inp, r), 1), dtype=torch.uint8, device=W0.device)
    dora_norm_factored_bwd(W0, A, B, norm, g, d_mag, s, dA, dB, ws)
    return dA, dB


@norm_factored_bwd.register_fake
def _norm_factored_bwd_fake(W0, A, B, norm, g, d_mag, s):
    return torch.empty_like(A, dtype=torch.float32), torch.empty_like(B, dtype=torch.float32)


@torch.library.custom_op("dora::module", mutates_args=(), device_types="cuda")
def module(base: Tensor, lora: Tensor, W0: Tensor, A: Tensor, B: Tensor, m: Tensor,
           s: float) -> tuple[Tensor, Tensor, Tensor]:
    """y = g (base + s lora) with n and g from the factored norm; returns (y, norm, g)."""
    _contig("module", base, lora, W0, A, B, m)
    out, inp = W0.shape
    r = A.shape[0]
    norm = torch.empty(out, device=W0.device, dtype=torch.float32)
    g = torch.empty_like(norm)
    ws = torch.empty(max(dora_norm_factored_workspace(out, inp, r), 1), dtype=torch.uint8, device=W0.device)
    dora_norm_factored(W0, A, B, m, s, norm, g, ws)
    y = torch.empty_like(base)
    dora_compose_fwd(base, lora, g, s, y)
    return y, norm, g


@module.register_fake
def _module_fake(base, lora, W0, A, B, m, s):
    out = W0.shape[0]
    return torch.empty_like(base), W0.new_empty(out, dtype=torch.float32), W0.new_empty(out, dtype=torch.float32)


def _module_setup(ctx, inputs, output):
    base, lora, W0, A, B, m, s = inputs
    _, norm, g = output
    ctx.save_for_backward(base, lora, W0, A, B, norm, g)
    ctx.s = s
    ctx.mark_non_differentiable(norm, g)


def _module_backward(ctx, dy, d_norm_out, d_g_out):
    base, lora, W0, A, B, norm, g = ctx.saved_tensors
    d_base, d_lora, d_mag = compose_bwd(dy.contiguous(), base, lora, g, norm, ctx.s)
    dA = dB = None
    if ctx.needs_input_grad[3] or ctx.needs_input_grad[4]:
        dA, dB = norm_factored_bwd(W0, A, B, norm, g, d_mag, ctx.s)
    return d_base, d_lora, None, dA, dB, d_mag, None


module.register_autograd(_module_backward, setup_context=_module_setup)


def dora_module(base: Tensor, lora: Tensor, W0: Tensor, A: Tensor, B: Tensor, m: Tensor, s: float,
                detach_norm: bool = True) -> Tensor:
    """One DoRA module's output from its two matmul results.

    detach_norm=True (the page's backward): the factored norm carries no
    gradient; the fused compose is differentiable in base, lora and m.
    detach_norm=False: the gradient also flows through the norm into A and B
    (dora::module)."""
    if not detach_norm:
        return module(base, lora, W0.detach(), A, B, m, s)[0]
    norm, g = norm_factored(W0.detach(), A.detach(), B.detach(), m.detach(), s)
    return compose(base, lora, m, g, norm, s)


# ---------------------------------------------------------------------------
# 8 bits: E4M3 with a power-of-two scale per 128 columns (include/dora.h)
# ---------------------------------------------------------------------------
def _scale_shape(rows: int, cols: int, block_rows: int) -> tuple[int, int]:
    if block_rows != 1 and block_rows != 128:
        raise ValueError(f"dora: an 8-bit form has 1 or 128 rows a scale, got {block_rows}")
    return -(-rows // block_rows), -(-cols // 128)


def _workspace(nbytes: int, like: Tensor) -> Tensor:
    return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=like.device)


@torch.library.custom_op("dora::q8_store", mutates_args=(), device_types="cuda")
def q8_store(x: Tensor, block_rows: int) -> tuple[Tensor, Tensor]:
    """x [rows, cols] in 8 bits: (q, scale), a scale per block_rows (1 or 128) x 128 elements."""
    _contig("q8_store", x)
    q = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    scale = torch.empty(_scale_shape(*x.shape, block_rows), dtype=torch.uint8, device=x.device)
    dora_q8_store(x, block_rows, q, scale)
    return q, scale


@q8_store.register_fake
def _q8_store_fake(x, block_rows):
    return x.new_empty(x.shape, dtype=torch.uint8), x.new_empty(_scale_shape(*x.shape, block_rows), dtype=torch.uint8)


@torch.library.custom_op("dora::q8_load", mutates_args=(), device_types="cuda")
def q8_load(q: Tensor, scale: Tensor, block_rows: int, dtype: torch.dtype) -> Tensor:
    """The values of an 8-bit form, float32 or bfloat16."""
    _contig("q8_load", q, scale)
    x = torch.empty(q.shape, dtype=dtype, device=q.device)
    dora_q8_load(q, scale, block_rows, x)
    return x


@q8_load.register_fake
def _q8_load_fake(q, scale, block_rows, dtype):
    return q.new_empty(q.shape, dtype=dtype)


@torch.library.custom_op("dora::compose_bwd_q8", mutates_args=(), device_types="cuda")
def compose_bwd_q8(dy: Tensor, vq: Tensor, vscale: Tensor, g: Tensor, norm: Tensor,
                   s: float) -> tuple[Tensor, Tensor, Tensor]:
    """d_base = g dy, d_lora = s g dy, d_mag = sum_t dy v / norm from the 8-bit v."""
    _contig("compose_bwd_q8", dy, vq, vscale, g, norm)
    d_base = torch.empty_like(dy)
    d_lora = torch.empty_like(dy)
    d_mag = torch.empty(dy.shape[1], device=dy.device, dtype=torch.float32)
    dora_compose_bwd_q8(dy, vq, vscale, g, norm, s, d_base, d_lora, d_mag,
                        _workspace(dora_compose_bwd_q8_workspace(*dy.shape), dy))
    return d_base, d_lora, d_mag


@compose_bwd_q8.register_fake
def _compose_bwd_q8_fake(dy, vq, vscale, g, norm, s):
    return torch.empty_like(dy), torch.empty_like(dy), dy.new_empty(dy.shape[1], dtype=torch.float32)


@torch.library.custom_op("dora::compose_q8", mutates_args=(), device_types="cuda")
def compose_q8(base: Tensor, lora: Tensor, m: Tensor, g: Tensor, norm: Tensor,
               s: float) -> tuple[Tensor, Tensor, Tensor]:
    """compose, with v = base + s lora kept in 8 bits for the backward: (y, vq, vscale)."""
    _contig("compose_q8", base, lora, g)
    y = torch.empty_like(base)
    vq = torch.empty(base.shape, dtype=torch.uint8, device=base.device)
    vscale = torch.empty(_scale_shape(*base.shape, 1), dtype=torch.uint8, device=base.device)
    dora_compose_fwd_q8(base, lora, g, s, y, vq, vscale)
    return y, vq, vscale


@compose_q8.register_fake
def _compose_q8_fake(base, lora, m, g, norm, s):
    return (torch.empty_like(base), base.new_empty(base.shape, dtype=torch.uint8),
            base.new_empty(_scale_shape(*base.shape, 1), dtype=torch.uint8))


def _compose_q8_setup(ctx, inputs, output):
    _, _, _, g, norm, s = inputs
    _, vq, vscale = output
    ctx.save_for_backward(vq, vscale, g, norm)
    ctx.s = s
    ctx.mark_non_differentiable(vq, vscale)


def _compose_q8_backward(ctx, dy, _vq, _vscale):
    vq, vscale, g, norm = ctx.saved_tensors
    d_base, d_lora, d_mag = compose_bwd_q8(dy.contiguous(), vq, vscale, g, norm, ctx.s)
    return d_base, d_lora, d_mag, None, None, None


compose_q8.register_autograd(_compose_q8_backward, setup_context=_compose_q8_setup)


@torch.library.custom_op("dora::matmul_q8", mutates_args=(), device_types="cuda")
def matmul_q8(xq: Tensor, xscale: Tensor, wq: Tensor, wscale: Tensor) -> Tensor:
    """x W^T in bfloat16, x and W in 8 bits (block_rows 1 and 128)."""
    _contig("matmul_q8", xq, xscale, wq, wscale)
    y = torch.empty(xq.shape[0], wq.shape[0], dtype=torch.bfloat16, device=xq.device)
    dora_matmul_q8(xq, xscale, wq, wscale, y)
    return y


@matmul_q8.register_fake
def _matmul_q8_fake(xq, xscale, wq, wscale):
    return xq.new_empty(xq.shape[0], wq.shape[0], dtype=torch.bfloat16)


@torch.library.custom_op("dora::matmul_q8_t", mutates_args=(), device_types="cuda")
def matmul_q8_t(dyq: Tensor, dyscale: Tensor, wq: Tensor, wscale: Tensor) -> Tensor:
    """dy W in bfloat16, dy and the same W in 8 bits."""
    _contig("matmul_q8_t", dyq, dyscale, wq, wscale)
    dx = torch.empty(dyq.shape[0], wq.shape[1], dtype=torch.bfloat16, device=dyq.device)
    dora_matmul_q8_t(dyq, dyscale, wq, wscale, dx)
    return dx


@matmul_q8_t.register_fake
def _matmul_q8_t_fake(dyq, dyscale, wq, wscale):
    return dyq.new_empty(dyq.shape[0], wq.shape[1], dtype=torch.bfloat16)


@torch.library.custom_op("dora::lora_grad_q8", mutates_args=(), device_types="cuda")
def lora_grad_q8(dxa: Tensor, xq: Tensor, xscale: Tensor) -> Tensor:
    """dA = dxa^T x in float32, dxa bfloat16, x in 8 bits."""
    _contig("lora_grad_q8", dxa, xq, xscale)
    (T, r), inp = dxa.shape, xq.shape[1]
    dA = torch.empty(r, inp, dtype=torch.float32, device=dxa.device)
    dora_lora_grad_q8(dxa, xq, xscale, dA, _workspace(dora_lora_grad_q8_workspace(T, inp, r), dxa))
    return dA


@lora_grad_q8.register_fake
def _lora_grad_q8_fake(dxa, xq, xscale):
    return dxa.new_empty(dxa.shape[1], xq.shape[1], dtype=torch.float32)


def _linear_q8_check(x: Tensor, wq: Tensor, wscale: Tensor, A: Tensor, B: Tensor, g: Tensor) -> None:
    """What the layer's forward takes; the same eagerly and while it is traced."""
    if x.dtype != torch.bfloat16:
        raise TypeError(f"dora::linear_q8: x is bfloat16, got {x.dtype}")
    if wq.element_size() != 1 or wscale.element_size() != 1:
        raise TypeError(f"dora::linear_q8: the 8-bit weight is bytes, got {wq.dtype} and {wscale.dtype}")
    if x.dim() != 2 or wq.dim() != 2 or A.dim() != 2:
        raise ValueError(f"dora::linear_q8: x [T, in], wq [out, in] and A [r, in] are matrices, got {tuple(x.shape)}, "
                         f"{tuple(wq.shape)}, {tuple(A.shape)}")
    (out, inp), r = wq.shape, A.shape[0]
    if out % 16 or inp % 16:
        raise ValueError(f"dora::linear_q8: in and out are multiples of 16, got {inp} and {out}")
    for name, t, want in (("x", x, (x.shape[0], inp)), ("wscale", wscale, _scale_shape(out, inp, 128)),
                          ("A", A, (r, inp)), ("B", B, (out, r)), ("g", g, (out,))):
        if t.shape != want:
            raise ValueError(f"dora::linear_q8: {name} is {want} for a weight [{out}, {inp}] and rank {r}, got {tuple(t.shape)}")
    if g.dtype != torch.float32:
        raise ValueError(f"dora::linear_q8: g is float32, got {g.dtype}")


@torch.library.custom_op("dora::linear_q8", mutates_args=(), device_types="cuda")
def linear_q8(x: Tensor, wq: Tensor, wscale: Tensor, A: Tensor, B: Tensor, m: Tensor, g: Tensor, norm: Tensor,
              s: float) -> tuple[Tensor, Tensor, Tensor, Tensor, Tensor, Tensor]:
    """The layer's output y and what its backward needs: (y, xq, xscale, vq, vscale, xa)."""
    _linear_q8_check(x, wq, wscale, A, B, g)
    xq, xscale = q8_store(x, 1)
    # the low-rank products run in x's bfloat16, fp32 A and B rounded to it (2^-8,
    # below what the 8-bit base product next to them carries, 2^-4).  v is kept
    # also where no backward will read it: one form of the call
    xa = x @ A.to(x.dtype).t()
    y, vq, vscale = compose_q8(matmul_q8(xq, xscale, wq, wscale), xa @ B.to(x.dtype).t(), m, g, norm, s)
    return y, xq, xscale, vq, vscale, xa


@linear_q8.register_fake
def _linear_q8_fake(x, wq, wscale, A, B, m, g, norm, s):
    _linear_q8_check(x, wq, wscale, A, B, g)
    T, inp = x.shape
    out = wq.shape[0]
    u8 = torch.uint8
    return (x.new_empty(T, out), x.new_empty(T, inp, dtype=u8), x.new_empty(_scale_shape(T, inp, 1), dtype=u8),
            x.new_empty(T, out, dtype=u8), x.new_empty(_scale_shape(T, out, 1), dtype=u8), x.new_empty(T, A.shape[0]))


def _linear_q8_setup(ctx, inputs, output):
    _, wq, wscale, A, B, m, g, norm, s = inputs
    _, xq, xscale, vq, vscale, xa = output
    # what the backward alone needs is refused by the call that leads to it
    r, (out,) = A.shape[0], g.shape
    if ctx.needs_input_grad[3] and (r % 8 or not 1 <= r <= 1024):
        raise ValueError(f"dora::linear_q8: a gradient of A takes a rank of 8, 16, ... 1024, got {r}")
    if ctx.needs_input_grad[5] and m.shape != (out,):
        raise ValueError(f"dora::linear_q8: m is ({out},), got {tuple(m.shape)}")
    if norm.shape != (out,) or norm.dtype != torch.float32:
        raise ValueError(f"dora::linear_q8: norm is ({out},) of float32, got {tuple(norm.shape)} of {norm.dtype}")
    ctx.save_for_backward(xq, xscale, vq, vscale, xa, wq, wscale, A, B, g, norm)
    ctx.s = s
    ctx.mark_non_differentiable(xq, xscale, vq, vscale, xa)


def _linear_q8_backward(ctx, dy, *_):
    xq, xscale, vq, vscale, xa, wq, wscale, A, B, g, norm = ctx.saved_tensors
    need = ctx.needs_input_grad
    d_base, d_lora, d_mag = compose_bwd_q8(dy.contiguous(), vq, vscale, g, norm, ctx.s)
    dx = dA = dB = None
    # dB and dxa leave their products in bfloat16, as under autocast, and dx is
    # the bfloat16 sum of two such results; dA, from the library's own product,
    # is fp32 until it takes A's type
    if need[4]:
        dB = (d_lora.t() @ xa).to(B.dtype)
    if need[0] or need[3]:
        dxa = d_lora @ B.to(d_lora.dtype)
        if need[3]:
            dA = lora_grad_q8(dxa, xq, xscale).to(A.dtype)
        if need[0]:
            dx = matmul_q8_t(*q8_store(d_base, 1), wq, wscale) + dxa @ A.to(dxa.dtype)
    return dx, None, None, dA, dB, d_mag, None, None, None


linear_q8.register_autograd(_linear_q8_backward, setup_context=_linear_q8_setup)


def dora_linear_q8(x: Tensor, wq: Tensor, wscale: Tensor, A: Tensor, B: Tensor, m: Tensor, g: Tensor, norm: Tensor,
                   s: float) -> Tensor:
    """y = g (x W0^T + s x A^T B^T) for a bfloat16 x and a frozen W0 in 8 bits (q8_store(W0, 128)).

    norm and g = m / norm come from one of the norm ops on the values of the
    8-bit weight (q8_load is exact in bfloat16) and carry no gradient; x, A, B
    and m do.  in and out are multiples of 16; where A takes a gradient, the rank
    is a multiple of 8 up to 1024.  What does not fit is refused by this call."""
    return linear_q8(x, wq, wscale, A, B, m, g, norm, s)[0]


# ---------------------------------------------------------------------------
# 4 bits: E2M1 with a power-of-two scale per 32 columns (include/dora.h)
# ---------------------------------------------------------------------------
def _q4_shapes(x: Tensor) -> tuple[list[int], list[int]]:
    *lead, cols = x.shape
    if not lead or cols % 32:
        raise ValueError(f"dora: a 4-bit form has rows of whole groups of 32 columns, got {tuple(x.shape)}")
    return [*lead, cols // 2], [*lead, cols // 32]


@torch.library.custom_op("dora::q4_store", mutates_args=(), device_types="cuda")
def q4_store(x: Tensor) -> tuple[Tensor, Tensor]:
    """x [..., rows, cols] in 4 bits: (q, scale), a scale per 32 columns of a row."""
    _contig("q4_store", x)
    q, scale = (torch.empty(s, dtype=torch.uint8, device=x.device) for s in _q4_shapes(x))
    dora_q4_store(x, q, scale)
    return q, scale


@q4_store.register_fake
def _q4_store_fake(x):
    _act(x)
    q, scale = _q4_shapes(x)
    return x.new_empty(q, dtype=torch.uint8), x.new_empty(scale, dtype=torch.uint8)


@torch.library.custom_op("dora::q4_load", mutates_args=(), device_types="cuda")
def q4_load(q: Tensor, scale: Tensor, dtype: torch.dtype) -> Tensor:
    """The values of a 4-bit form, float32 or bfloat16."""
    _contig("q4_load", q, scale)
    x = torch.empty((*q.shape[:-1], 2 * q.shape[-1]), dtype=dtype, device=q.device)
    dora_q4_load(q, scale, x)
    return x


@q4_load.register_fake
def _q4_load_fake(q, scale, dtype):
    x = q.new_empty((*q.shape[:-1], 2 * q.shape[-1]), dtype=dtype)
    _q4("dora_q4_load", x.shape, q, scale)
    _act(x)
    return x


@torch.library.custom_op("dora::matmul_q4", mutates_args=(), device_types="cuda")
def matmul_q4(x: Tensor, wq: Tensor, wscale: Tensor, offsets: Optional[Tensor] = None) -> Tensor:
    """x W^T for a bfloat16 x and W in 4 bits; with offsets (expert_sort) W is a stack and
    x's rows are sorted by expert."""
    _contig("matmul_q4", x, wq, wscale)
    T, out, inp, cols, experts = _matmul_q4_sizes("dora_matmul_q4", x, wq, wscale, offsets, True)
    y = torch.empty(T, cols, dtype=torch.bfloat16, device=x.device)
    n = dora_matmul_q4_workspace(T, out, inp, experts)
    dora_matmul_q4(x, wq, wscale, y, offsets, _workspace(n, x) if n else None)
    if offsets is not None:
        dora_expert_clear(y, offsets)
    return y


def _matmul_q4_traced(name, x, wq, wscale, offsets, out_side):
    T, out, _, cols, experts = _matmul_q4_sizes(name, x, wq, wscale, offsets, out_side)
    # what the library itself refuses
    if T and out % 16:
        raise ValueError(f"{name}: out is a multiple of 16, got {out}")
    if not 1 <= experts <= 4096:
        raise ValueError(f"{name}: 1 to 4096 experts, got {experts}")
    return x.new_empty(T, cols, dtype=torch.bfloat16)


@matmul_q4.register_fake
def _matmul_q4_fake(x, wq, wscale, offsets=None):
    return _matmul_q4_traced("dora_matmul_q4", x, wq, wscale, offsets, True)


@torch.library.custom_op("dora::matmul_q4_t", mutates_args=(), device_types="cuda")
def matmul_q4_t(dy: Tensor, wq: Tensor, wscale: Tensor, offsets: Optional[Tensor] = None) -> Tensor:
    """dy W for a bfloat16 dy and the same W."""
    _contig("matmul_q4_t", dy, wq, wscale)
    T, out, inp, cols, experts = _matmul_q4_sizes("dora_matmul_q4_t", dy, wq, wscale, offsets, False)
    dx = torch.empty(T, cols, dtype=torch.bfloat16, device=dy.device)
    n = dora_matmul_q4_t_workspace(T, out, inp, experts)
    dora_matmul_q4_t(dy, wq, wscale, dx, offsets, _workspace(n, dy) if n else None)
    if offsets is not None:
        dora_expert_clear(dx, offsets)
    return dx


@matmul_q4_t.register_fake
def _matmul_q4_t_fake(dy, wq, wscale, offsets=None):
    return _matmul_q4_traced("dora_matmul_q4_t", dy, wq, wscale, offsets, False)


def _matmul_q4_setup(ctx, inputs, output):
    _, wq, wscale, offsets = inputs
    ctx.save_for_backward(wq, wscale, offsets)


def _matmul_q4_backward(ctx, dy):
    return matmul_q4_t(dy.contiguous(), *ctx.saved_tensors), None, None, None


matmul_q4.register_autograd(_matmul_q4_backward, setup_context=_matmul_q4_setup)


def _linear_q4_check(x: Tensor, wq: Tensor, wscale: Tensor, A: Tensor, B: Tensor, m: Tensor,
                     g: Tensor, norm: Tensor) -> None:
    """What the layer's forward takes; the same eagerly and while it is traced."""
    if x.dtype != torch.bfloat16:
        raise TypeError(f"dora::linear_q4: x is bfloat16, got {x.dtype}")
    if wq.element_size() != 1 or wscale.element_size() != 1:
        raise TypeError(f"dora::linear_q4: the 4-bit weight is bytes, got {wq.dtype} and {wscale.dtype}")
    if x.dim() != 2 or wq.dim() != 2 or A.dim() != 2:
        raise ValueError(f"dora::linear_q4: x [T, in], wq [out, in / 2] and A [r, in] are matrices, got {tuple(x.shape)}, "
                         f"{tuple(wq.shape)}, {tuple(A.shape)}")
    out, inp, r = wq.shape[0], 2 * wq.shape[1], A.shape[0]
    if out % 16 or inp % 32:
        raise ValueError(f"dora::linear_q4: in is a multiple of 32 and out of 16, got {inp} and {out}")
    for name, t, want in (("x", x, (x.shape[0], inp)), ("wscale", wscale, (out, inp // 32)), ("A", A, (r, inp)),
                          ("B", B, (out, r)), ("m", m, (out,)), ("g", g, (out,)), ("norm", norm, (out,))):
        if t.shape != want:
            raise ValueError(f"dora::linear_q4: {name} is {want} for a weight [{out}, {inp}] and rank {r}, got {tuple(t.shape)}")
    for name, t in (("g", g), ("norm", norm)):
        if t.dtype != torch.float32:
            raise ValueError(f"dora::linear_q4: {name} is float32, got {t.dtype}")


@torch.library.custom_op("dora::linear_q4", mutates_args=(), device_types="cuda")
def linear_q4(x: Tensor, wq: Tensor, wscale: Tensor, A: Tensor, B: Tensor, m: Tensor, g: Tensor, norm: Tensor,
              s: float) -> tuple[Tensor, Tensor, Tensor, Tensor, Tensor, Tensor]:
    """The layer's output y and what its backward needs: (y, xq, xscale, vq, vscale, xa)."""
    _linear_q4_check(x, wq, wscale, A, B, m, g, norm)
    xq, xscale = q8_store(x, 1)
    xa = x @ A.to(x.dtype).t()
    y, vq, vscale = compose_q8(matmul_q4(x, wq, wscale), xa @ B.to(x.dtype).t(), m, g, norm, s)
    return y, xq, xscale, vq, vscale, xa


@linear_q4.register_fake
def _linear_q4_fake(x, wq, wscale, A, B, m, g, norm, s):
    _linear_q4_check(x, wq, wscale, A, B, m, g, norm)
    T, inp = x.shape
    out = wq.shape[0]
    u8 = torch.uint8
    return (x.new_empty(T, out), x.new_empty(T, inp, dtype=u8), x.new_empty(_scale_shape(T, inp, 1), dtype=u8),
            x.new_empty(T, out, dtype=u8), x.new_empty(_scale_shape(T, out, 1), dtype=u8), x.new_empty(T, A.shape[0]))


def _linear_q4_setup(ctx, inputs, output):
    _, wq, wscale, A, B, _, g, norm, s = inputs
    _, xq, xscale, vq, vscale, xa = output
    # what the backward alone needs is refused by the call that leads to it
    r = A.shape[0]
    if ctx.needs_input_grad[3] and (r % 8 or not 1 <= r <= 1024):
        raise ValueError(f"dora::linear_q4: a gradient of A takes a rank of 8, 16, ... 1024, got {r}")
    ctx.save_for_backward(xq, xscale, vq, vscale, xa, wq, wscale, A, B, g, norm)
    ctx.s = s
    ctx.mark_non_differentiable(xq, xscale, vq, vscale, xa)


def _linear_q4_backward(ctx, dy, *_):
    xq, xscale, vq, vscale, xa, wq, wscale, A, B, g, norm = ctx.saved_tensors
    need = ctx.needs_input_grad
    d_base, d_lora, d_mag = compose_bwd_q8(dy.contiguous(), vq, vscale, g, norm, ctx.s)
    dx = dA = dB = None
    # dB and dxa leave their products in bfloat16, as in linear_q8; dx is the bfloat16
    # sum of two such results
    if need[4]:
        dB = (d_lora.t() @ xa).to(B.dtype)
    if need[0] or need[3]:
        dxa = d_lora @ B.to(d_lora.dtype)
        if need[3]:
            dA = lora_grad_q8(dxa, xq, xscale).to(A.dtype)
        if need[0]:
            dx = matmul_q4_t(d_base, wq, wscale) + dxa @ A.to(dxa.dtype)
    return dx, None, None, dA, dB, d_mag, None, None, None


linear_q4.register_autograd(_linear_q4_backward, setup_context=_linear_q4_setup)


def dora_linear_q4(x: Tensor, wq: Tensor, wscale: Tensor, A: Tensor, B: Tensor, m: Tensor, g: Tensor, norm: Tensor,
                   s: float) -> Tensor:
    """y = g (x W0^T + s x A^T B^T) for a bfloat16 x and a frozen W0 in 4 bits (q4_store(W0)).

    norm and g = m / norm come from one of the norm ops on the values of the 4-bit
    weight (q4_load is exact in bfloat16) and carry no gradient; x, A, B and m do.  in is
    a multiple of 32 and out of 16; where A takes a gradient, the rank is a multiple of 8
    up to 1024.  Where something does, x and v are kept in 8 bits for the backward, which dA
    and d_mag take from them (off by 2.6% of their norm, as in dora_linear_q8).  Where nothing
    takes a gradient, nothing is kept for one: serving a token is the products and a compose."""
    if not (torch.is_grad_enabled() and any(t.requires_grad for t in (x, A, B, m))):
        _linear_q4_check(x, wq, wscale, A, B, m, g, norm)
        lora = (x @ A.to(x.dtype).t()) @ B.to(x.dtype).t()
        return compose(matmul_q4(x, wq, wscale), lora, m, g, norm, s)
    return linear_q4(x, wq, wscale, A, B, m, g, norm, s)[0]


# ---------------------------------------------------------------------------
# tokens sorted by expert and back
# ---------------------------------------------------------------------------
@torch.library.custom_op("dora::expert_sort", mutates_args=(), device_types="cuda")
def expert_sort(expert: Tensor, experts: int) -> tuple[Tensor, Tensor, Tensor]:
    """The entries of expert [T, k] (int32 or int64) sorted by expert, stably: (order
    [T k], inverse [T, k], offsets [experts + 1]), int32.  An entry outside
    [0, experts) goes to no expert, behind all that do."""
    _contig("expert_sort", expert)
    T, k = _expert_sort_sizes(expert, experts)
    i32 = dict(dtype=torch.int32, device=expert.device)
    order, inverse, offsets = torch.empty(T * k, **i32), torch.empty(T, k, **i32), torch.empty(experts + 1, **i32)
    dora_expert_sort(expert, experts, order, inverse, offsets)
    return order, inverse, offsets


@expert_sort.register_fake
def _expert_sort_fake(expert, experts):
    T, k = _expert_sort_sizes(expert, experts)
    i32 = torch.int32
    return expert.new_empty(T * k, dtype=i32), expert.new_empty(T, k, dtype=i32), expert.new_empty(experts + 1, dtype=i32)


@torch.library.custom_op("dora::expert_return", mutates_args=(), device_types="cuda")
def expert_return(ys: Tensor, inverse: Tensor, offsets: Tensor, weight: Optional[Tensor] = None) -> Tensor:
    """y[t] = sum_j weight[t, j] ys[inverse[t, j]] over the entries that have an expert;
    without weights the plain sum."""
    _contig("expert_return", ys, inverse, offsets)
    y = torch.empty(inverse.shape[0], ys.shape[1], dtype=ys.dtype, device=ys.device)
    dora_expert_return(ys, inverse, offsets, None if weight is None else weight.contiguous(), y)
    return y


@expert_return.register_fake
def _expert_return_fake(ys, inverse, offsets, weight=None):
    y = ys.new_empty(inverse.shape[0], *ys.shape[1:])
    T, k, _, _ = _routed("dora_expert_return", y, ys, inverse, offsets)
    if weight is not None:
        _same("dora_expert_return", (T, k), torch.float32, weight)
    _act(ys)
    return y


@torch.library.custom_op("dora::expert_send", mutates_args=(), device_types="cuda")
def expert_send(x: Tensor, inverse: Tensor, offsets: Tensor) -> Tensor:
    """xs[inverse[t, j]] = x[t], the tokens' rows sorted by expert."""
    _contig("expert_send", x, inverse, offsets)
    xs = torch.empty(inverse.numel(), x.shape[1], dtype=x.dtype, device=x.device)
    dora_expert_send(x, inverse, offsets, xs)
    dora_expert_clear(xs, offsets)
    return xs


@expert_send.register_fake
def _expert_send_fake(x, inverse, offsets):
    xs = x.new_empty(inverse.numel(), *x.shape[1:])
    _routed("dora_expert_send", x, xs, inverse, offsets)
    _act(x)
    return xs


def _expert_send_setup(ctx, inputs, output):
    ctx.save_for_backward(inputs[1], inputs[2])


def _expert_send_backward(ctx, d_xs):
    return expert_return(d_xs.contiguous(), *ctx.saved_tensors), None, None


expert_send.register_autograd(_expert_send_backward, setup_context=_expert_send_setup)


@torch.library.custom_op("dora::expert_return_bwd", mutates_args=(), device_types="cuda")
def expert_return_bwd(dy: Tensor, ys: Tensor, inverse: Tensor, offsets: Tensor, weight: Tensor) -> tuple[Tensor, Tensor]:
    """d_ys[inverse[t, j]] = weight[t, j] dy[t], d_weight[t, j] = <dy[t], ys[inverse[t, j]]>."""
    _contig("expert_return_bwd", dy, ys, inverse, offsets, weight)
    d_ys, d_weight = torch.empty_like(ys), torch.empty_like(weight)
    dora_expert_return_bwd(dy, ys, inverse, offsets, weight, d_ys, d_weight)
    dora_expert_clear(d_ys, offsets)
    return d_ys, d_weight


@expert_return_bwd.register_fake
def _expert_return_bwd_fake(dy, ys, inverse, offsets, weight):
    T, k, _, _ = _routed("dora_expert_return_bwd", dy, ys, inverse, offsets)
    _same("dora_expert_return_bwd", (T, k), torch.float32, weight)
    _act(dy)
    return torch.empty_like(ys), torch.empty_like(weight)


def _expert_return_setup(ctx, inputs, output):
    ys, inverse, offsets, weight = inputs
    # without weights the gradient of ys is the sending of dy
    ctx.save_for_backward(None if weight is None else ys, inverse, offsets, weight)


def _expert_return_backward(ctx, dy):
    ys, inverse, offsets, weight = ctx.saved_tensors
    if weight is None:
        return expert_send(dy.contiguous(), inverse, offsets), None, None, None
    d_ys, d_weight = expert_return_bwd(dy.contiguous(), ys, inverse, offsets, weight.contiguous())
    return d_ys, None, None, d_weight


expert_return.register_autograd(_expert_return_backward, setup_context=_expert_return_setup)


def experts_q4(x: Tensor, expert: Tensor, weight: Tensor, wq: Tensor, wscale: Tensor) -> Tensor:
    """y[t] = sum_j weight[t, j] W[expert[t, j]] x[t] for frozen experts W [experts, out, in] in
    4 bits (q4_store of the stack), x bfloat16 [T, in], expert and weight [T, k].

    Differentiable in x and weight.  Experts of more than one product (gate, up and down
    with an activation between) sort and send once:

        _, inverse, offsets = expert_sort(expert, experts)
        xs = expert_send(x, inverse, offsets)
        hs = act(matmul_q4(xs, gate_q, gate_scale, offsets)) * matmul_q4(xs, up_q, up_scale, offsets)
        y = expert_return(matmul_q4(hs, down_q, down_scale, offsets), inverse, offsets, weight)"""
    if wq.dim() != 3:
        raise ValueError(f"dora::experts_q4: a stack of weights [experts, out, in / 2], got {tuple(wq.shape)}")
    if expert.dim() != 2 or expert.shape[0] != x.shape[0] or weight.shape != expert.shape:
        raise ValueError(f"dora::experts_q4: expert and weight are [T, k] for x [T, in], got {tuple(expert.shape)}, "
                         f"{tuple(weight.shape)}, {tuple(x.shape)}")
    _, inverse, offsets = expert_sort(expert, wq.shape[0])
    ys = matmul_q4(expert_send(x, inverse, offsets), wq, wscale, offsets)
    return expert_return(ys, inverse, offsets, weight.float())
