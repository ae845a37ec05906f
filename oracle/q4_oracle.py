"""fp64 oracle of the 4-bit form, of the products with it and of the experts' routing.

TEST INFRASTRUCTURE ONLY, on the CPU, sharing no code with the CUDA library.

The form of a matrix x [rows, cols], cols a multiple of 32: a code c of 0 .. 15 per
element, two a byte with the even column in the low half, and b, a byte per 32 columns
of a row; the value is E2M1(c) 2^(b - 127), NaN where b = 255.  Definition of b: the
smallest integer k >= -125 with max |x| <= 6 * 2^k over the group, b = k + 127; of c: the
nearest E2M1 value to x / 2^k, ties to the even mantissa; a group that is not all
finite is zeros with b = 255.

Pins (tests/test_q4_oracle.py): hand-made bytes, the identity of encode and decode on
every representable value, the nearest value by brute force; the routing by hand.
"""
from __future__ import annotations

import math

import numpy as np

__all__ = ["e2m1_table", "q4_encode", "q4_decode", "matmul_q4", "matmul_q4_t", "expert_sort", "expert_send",
           "expert_return", "expert_return_bwd"]


def e2m1_table() -> np.ndarray:
    """float64 value of each code: sign, exponent (2 bits, bias 1), mantissa (1 bit)."""
    v = np.empty(16)
    for c in range(16):
        e, m = (c >> 1) & 3, c & 1
        mag = (2 + m) * 2.0 ** (e - 2) if e else 0.5 * m
        v[c] = -mag if c & 8 else mag
    return v


def q4_encode(x):
    """(q, scale) bytes of a float64 matrix (values of any narrower type widen exactly)."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    g = x.reshape(rows, cols // 32, 32)
    finite = np.isfinite(g).all(-1)
    top = np.where(np.isfinite(g), np.abs(g), 0.0).max(-1, initial=0.0)
    k = np.full(top.shape, -125)
    for i, v in np.ndenumerate(top):
        if v > 0:
            e = math.frexp(v / 6.0)[1] - 1
            while v > 6.0 * 2.0 ** e:
                e += 1
            while v <= 6.0 * 2.0 ** (e - 1):
                e -= 1
            k[i] = max(e, -125)
    u = np.where(finite[..., None], np.abs(g), 0.0) / np.exp2(k.astype(np.float64))[..., None]
    pos = e2m1_table()[:8]                            # increasing, codes 0 .. 7
    hi = np.clip(np.searchsorted(pos, u, side="left"), 0, 7)
    lo = np.maximum(hi - 1, 0)
    dlo, dhi = u - pos[lo], pos[hi] - u
    code = np.where((dlo < dhi) | ((dlo == dhi) & (lo % 2 == 0)), lo, hi)
    code = np.where(u == pos[hi], hi, code)
    code = np.where(finite[..., None], code | np.where(np.signbit(g), 8, 0), 0).reshape(rows, cols)
    return ((code[:, 0::2] | code[:, 1::2] << 4).astype(np.uint8),
            np.where(finite, k + 127, 255).astype(np.uint8))


def q4_decode(q, scale) -> np.ndarray:
    q = np.asarray(q)
    code = np.stack([q & 15, q >> 4], -1).reshape(*q.shape[:-1], 2 * q.shape[-1])
    s = np.where(np.asarray(scale) == 255, np.nan, np.exp2(np.asarray(scale, np.float64) - 127.0))
    with np.errstate(invalid="ignore"):
        return e2m1_table()[code] * np.repeat(s, 32, axis=-1)


def _by_expert(x, W, offsets, y):
    for e in range(W.shape[0]):
        a, b = offsets[e], offsets[e + 1]
        y[a:b] = x[a:b] @ W[e]
    return y


def matmul_q4(x, wq, wscale, offsets=None):
    """x W^T; with offsets by expert, NaN in the rows that no expert has."""
    W = q4_decode(wq, wscale)
    if offsets is None:
        return x @ W.T
    return _by_expert(x, W.transpose(0, 2, 1), offsets, np.full((x.shape[0], W.shape[1]), np.nan))


def matmul_q4_t(dy, wq, wscale, offsets=None):
    W = q4_decode(wq, wscale)
    if offsets is None:
        return dy @ W
    return _by_expert(dy, W, offsets, np.full((dy.shape[0], W.shape[2]), np.nan))


def expert_sort(expert, experts):
    """(order, inverse, offsets); entries of no expert behind all others, in order too."""
    flat = [int(e) if 0 <= int(e) < experts else experts for e in np.asarray(expert).ravel()]
    order = sorted(range(len(flat)), key=lambda i: (flat[i], i))
    inverse = np.empty(len(flat), np.int64)
    inverse[order] = np.arange(len(flat))
    offsets = [sum(f < e for f in flat) for e in range(experts + 1)]
    return np.asarray(order, np.int64), inverse.reshape(np.shape(expert)), np.asarray(offsets)


def expert_send(x, inverse, offsets, xs):
    xs = xs.copy()
    for (t, _), p in np.ndenumerate(inverse):
        if p < offsets[-1]:
            xs[p] = x[t]
    return xs


def expert_return(ys, inverse, offsets, weight):
    y = np.zeros((inverse.shape[0], ys.shape[1]))
    for (t, j), p in np.ndenumerate(inverse):
        if p < offsets[-1]:
            y[t] += (1.0 if weight is None else float(weight[t, j])) * ys[p]
    return y


def expert_return_bwd(dy, ys, inverse, offsets, weight, d_ys):
    d_ys, d_w = d_ys.copy(), np.zeros(inverse.shape)
    for (t, j), p in np.ndenumerate(inverse):
        if p < offsets[-1]:
            d_ys[p] = float(weight[t, j]) * dy[t]
            d_w[t, j] = dy[t] @ ys[p]
    return d_ys, d_w
