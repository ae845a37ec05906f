"""fp64 oracle of the 8-bit form and of the operators that use it.

TEST INFRASTRUCTURE ONLY, on the CPU, sharing no code with the CUDA library.

The form of a matrix x [rows, cols]: q[i, j], an E4M3 byte, and b, a byte per
block of block_rows x 128 elements that stands for 2^(b - 127); the value is
E4M3(q) 2^(b - 127).  Definition of b: the smallest integer k >= -117 with
max |x| <= 448 * 2^k over the block's finite elements, b = k + 127; of q: the
nearest E4M3 value to x / 2^k, ties to the even mantissa; NaN and infinities
become the byte 0x7f.

Pins (tests/test_q8_oracle.py): hand-made bytes, torch's own E4M3 cast, the
identity of encode and decode on every representable value.
"""
from __future__ import annotations

import math

import numpy as np

__all__ = ["e4m3_table", "q8_encode", "q8_decode", "compose_fwd_q8", "compose_bwd_q8", "lora_grad_q8", "matmul_q8",
           "matmul_q8_t"]


def e4m3_table() -> np.ndarray:
    """float64 value of each byte: sign, exponent (4 bits, bias 7), mantissa (3 bits); 0x7f / 0xff are NaN."""
    v = np.empty(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        mag = math.nan if (b & 127) == 127 else (8 + m) * 2.0 ** (e - 10) if e else m * 2.0 ** -9
        v[b] = -mag if b & 128 else mag
    return v


def _expand(s: np.ndarray, rows: int, cols: int, block_rows: int) -> np.ndarray:
    return np.repeat(np.repeat(s, block_rows, axis=0)[:rows], 128, axis=1)[:, :cols]


def q8_encode(x, block_rows: int = 1):
    """(q, scale) bytes of a float64 matrix (values of any narrower type widen exactly)."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    nr, nc = -(-rows // block_rows), -(-cols // 128)
    mag = np.zeros((nr * block_rows, nc * 128))
    mag[:rows, :cols] = np.where(np.isfinite(x), np.abs(x), 0.0)
    top = mag.reshape(nr, block_rows, nc, 128).max(axis=(1, 3))
    k = np.full(top.shape, -117)
    for i, v in np.ndenumerate(top):
        if v > 0:
            e = math.frexp(v / 448.0)[1] - 1          # 2^e <= v / 448 (rounded) < 2^(e + 1)
            while v > 448.0 * 2.0 ** e:
                e += 1
            while v <= 448.0 * 2.0 ** (e - 1):
                e -= 1
            k[i] = max(e, -117)
    u = np.abs(x) / _expand(np.exp2(k.astype(np.float64)), rows, cols, block_rows)
    pos = e4m3_table()[:127]                          # increasing, bytes 0 .. 126
    fin = np.where(np.isfinite(u), u, 0.0)
    hi = np.clip(np.searchsorted(pos, fin, side="left"), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dlo, dhi = fin - pos[lo], pos[hi] - fin
    byte = np.where((dlo < dhi) | ((dlo == dhi) & (lo % 2 == 0)), lo, hi)
    byte = np.where(fin == pos[hi], hi, byte)
    byte = np.where(np.isfinite(x), byte | np.where(np.signbit(x), 128, 0), 127)
    return byte.astype(np.uint8), (k + 127).astype(np.uint8)


def q8_decode(q, scale, block_rows: int = 1) -> np.ndarray:
    rows, cols = q.shape
    s = np.exp2(np.asarray(scale, np.float64) - 127.0)
    return e4m3_table()[q] * _expand(s, rows, cols, block_rows)


def compose_fwd_q8(base, lora, g, s):
    """y in fp64, and the 8-bit form of v, which is base + s lora rounded to fp32 after
    the product and after the sum (base, lora: values of the activation type; s as float32)."""
    b32, l32 = np.asarray(base, np.float32), np.asarray(lora, np.float32)
    v = b32 + np.float32(s) * l32
    y = np.asarray(g, np.float64) * (b32.astype(np.float64) + float(np.float32(s)) * l32.astype(np.float64))
    return y, q8_encode(v)


def compose_bwd_q8(dy, q, scale, g, norm, s):
    dy = np.asarray(dy, np.float64)
    d_base = np.asarray(g, np.float64) * dy
    return d_base, s * d_base, (dy * q8_decode(q, scale)).sum(0) / np.asarray(norm, np.float64)


def lora_grad_q8(dxa, q, scale):
    return np.asarray(dxa, np.float64).T @ q8_decode(q, scale)


def matmul_q8(q, scale, wq, wscale):
    return q8_decode(q, scale) @ q8_decode(wq, wscale, 128).T


def matmul_q8_t(q, scale, wq, wscale):
    return q8_decode(q, scale) @ q8_decode(wq, wscale, 128)
