"""NVFP4 (E2M1 values, an E4M3 scale per 16, a float32 scale per matrix) and
the product of BF16 activations with 4-bit weights — test infrastructure only.

The 4-bit checkpoint keeps its experts as E2M1 values with an E4M3 scale per
16 inputs and a float32 scale per expert, and without fast-math widens them
to 16 bits as it multiplies (Lernex/Metis-1.6-Praxis-NVFP4, "What is in
NVFP4" and "What --fast-math does"). The page gives no quantisation rule;
the reading taken here, every quotient and product rounded once to float32:

* the group's scale is g = amax / (6 * 448), so that the largest block's
  scale is the largest E4M3 magnitude and its largest value the largest
  E2M1 magnitude; not below 2**-96, and 1 for an all-zero group;
* a block's scale is E4M3(min((amax_b / 6) / g, 448)), to nearest even;
* a value is x / d with d = dec(scale) * g, rounded to E2M1 to nearest, ties
  to the even code, saturating at 6; a zero with the sign of x where d = 0.

The value of a code is dec(code) * dec(scale) * g. In the product the code
times its block scale has at most 6 significant bits and is exact in BF16;
the oracle multiplies in float64 and applies g to the sum.
"""
from __future__ import annotations

import numpy as np

from .bf16 import bf16_bits_to_f64, round_to_bf16_bits
from .e4m3 import decode, encode
from .mxfp4 import e2m1_decode, e2m1_encode, mx_dequant, mx_unpack

__all__ = ["NVFP4_GSCALE_MIN", "nvfp4_quantize", "nvfp4_scaled", "nvfp4_dequant_f32", "w4a16_linear"]

NVFP4_GSCALE_MIN = 2.0 ** -96


def _f32(v) -> np.ndarray:
    return np.asarray(v, np.float64).astype(np.float32).astype(np.float64)


def nvfp4_quantize(x, g=None):
    """One group [R, K] of float32 values -> (packed codes uint8 [R, K/2],
    E4M3 scales uint8 [R, K/16], g float32)."""
    x = np.asarray(x, np.float32).astype(np.float64)
    R, K = x.shape
    if K % 16:
        raise ValueError("K must be a multiple of 16")
    if g is None:
        amax = float(np.abs(x).max()) if x.size else 0.0
        g = max(float(_f32(amax / 2688.0)), NVFP4_GSCALE_MIN) if amax > 0 else 1.0
    g = float(np.float32(g))
    b = x.reshape(R, K // 16, 16)
    t = np.minimum(_f32(_f32(np.abs(b).max(-1) / 6.0) / g), 448.0)
    s = encode(t.astype(np.float32))
    d = _f32(decode(s) * g)[..., None]
    v = np.where(d > 0, _f32(b / np.where(d > 0, d, 1.0)), np.copysign(0.0, b))
    c = e2m1_encode(v).reshape(R, K)
    return (c[:, 0::2] | (c[:, 1::2] << 4)).astype(np.uint8), s.astype(np.uint8), np.float32(g)


def nvfp4_scaled(q, s) -> np.ndarray:
    """dec(code) * dec(block scale), float64 [rows, K] (exact)."""
    v = e2m1_decode(mx_unpack(q))
    return v * np.repeat(decode(s), 16, axis=1)


def nvfp4_dequant_f32(q, s, g) -> np.ndarray:
    """fl32(dec(code) * fl32(dec(scale) * g)), float32 [rows, K]."""
    d = _f32(decode(s) * float(np.float32(g)))
    return (e2m1_decode(mx_unpack(q)) * np.repeat(d, 16, axis=1)).astype(np.float32)


def w4a16_linear(x_bits, qw, sw, g=None):
    """Y = bf16(g * x . w^T): NVFP4 weights where ``g`` is given, else MXFP4.
    Returns (y64, y_bf16)."""
    x = bf16_bits_to_f64(x_bits)
    y = x @ (nvfp4_scaled(qw, sw) * float(np.float32(g)) if g is not None else mx_dequant(qw, sw)).T
    return y, round_to_bf16_bits(y)
