"""Helpers of the NVFP4, 4-bit product, router and few-token tests (test infrastructure)."""
from __future__ import annotations

import numpy as np

import oracle
import synth
from gpu_util import BF16_MFMA_ERR, U32, bf16_ulp

FORMATS = ("fp8", "mxfp4", "nvfp4")


def random_codes(rng, fmt, *rows_k, seed_scale=1.0):
    """Random weights of a format as a checkpoint's quantiser leaves them: the tuple the calls take
    (numpy arrays) and a function of the matrix index to its float64 values."""
    *lead, rows, K = rows_k
    E = lead[0] if lead else 1
    w = synth.bf16_bits_to_f32(synth.weights(rng, (E * rows, K))) * np.float32(seed_scale)
    if fmt == "fp8":
        q, s, _ = oracle.quantize_rows(w)
        q, s = q.reshape(E, rows, K), s.reshape(E, rows)
        return (q, s), lambda e: oracle.decode(q[e]) * s[e].astype(np.float64)[:, None]
    if fmt == "mxfp4":
        q, s = oracle.mx_quantize_rows(w)
        q, s = q.reshape(E, rows, K // 2), s.reshape(E, rows, K // 32)
        return (q, s), lambda e: oracle.mx_dequant(q[e], s[e])
    parts = [oracle.nvfp4_quantize(m) for m in w.reshape(E, rows, K)]
    q, s, g = (np.stack([p[i] for p in parts]) for i in range(3))
    return (q, s, g.astype(np.float32)), lambda e: oracle.nvfp4_scaled(q[e], s[e]) * float(g[e])


def few_bound(mag, H, I, k):
    """Bound on |out_gpu - out64| before the last rounding, from oracle.wide_pass's magnitudes.

    Gate/up: products are exact; the BF16 MFMA's own sum of 32 products is within 2^-20 of their sum of
    magnitudes, each of the H/32 instructions, the 3 sums of the waves' parts and the scale round once in float32.
    These errors reach the output through dh (the first magnitude). h itself: silu's float32 evaluation with the fast
    exponential and reciprocal, and the product with u, 2^-19 relative; the BF16 pair, 2^-17. Down: two MFMA chains of
    I/32 instructions (h's high part has up to 1 + 2^-8 of its magnitude), their sum, two scalings, then at most one
    addition per expert, part of K (at most 16) and wave.
    """
    gu = BF16_MFMA_ERR + (H / 32 + 6) * U32
    down = 2.0 ** -17 + 2.0 ** -19 + 1.01 * (BF16_MFMA_ERR + (I / 16 + 8) * U32) + (k + 34) * U32
    return 1.02 * (gu * mag[0] + down * mag[1])


def out_violations(got_bits, ref64, err):
    g = oracle.bf16_bits_to_f64(got_bits)
    return int((np.abs(g - ref64) > err + 0.5 * bf16_ulp(g) + 1e-37).sum())
