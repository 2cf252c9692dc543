"""The router, and a routed-expert pass in the default maths — test
infrastructure only.

The pages' router picks the top experts of each token in float32 with a
balance bias (Lernex/Metis-1.6-Praxis, "Architecture"; sglang-metis 0.1.0,
"How the model maps onto SGLang"); a step with few tokens uses the default
maths: BF16 activations times weights widened to 16 bits (Lernex/Metis-1.6-
Logos-FP8, "What --fast-math does"). Readings where they are silent: the
score is the softmax or the sigmoid of the logits; the bias is added for the
choice and not for the weights; equal scores go to the lower index; the
weights may be renormalised over the chosen. h = silu(g) * u and the
weighted sum over a token's experts are not rounded before the output.
"""
from __future__ import annotations

import numpy as np

from .bf16 import bf16_bits_to_f64, round_to_bf16_bits

__all__ = ["router", "wide_pass"]


def router(x_bits, w_bits, topk, bias=None, score="softmax", renormalize=True, scale=1.0):
    """(ids [T, topk], weights float64 [T, topk], what the choice went by [T, E])."""
    logits = bf16_bits_to_f64(x_bits) @ bf16_bits_to_f64(w_bits).T
    if score == "softmax":
        e = np.exp(logits - logits.max(1, keepdims=True))
        p = e / e.sum(1, keepdims=True)
    else:
        with np.errstate(over="ignore"):
            p = 1.0 / (1.0 + np.exp(-logits))
    by = p if bias is None else p + np.asarray(bias, np.float32).astype(np.float64)
    ids = np.argsort(-by, axis=1, kind="stable")[:, :topk]
    w = np.take_along_axis(p, ids, 1)
    if renormalize:
        w = w / w.sum(1, keepdims=True)
    return ids.astype(np.int32), w * scale, by


def wide_pass(x_bits, ids, w, w13, w2):
    """out[t] = sum over valid j of w[t, j] * W2[e] . (silu(g) * u), [g; u] = W13[e] . x[t].

    w13, w2: functions of an expert's index that return its float64 matrix
    ([2I, H] and [H, I]). Returns (out64, out_bf16, mag): mag[t] adds up
    |w| |W2| (|u| |dsilu/dg| |W13_g| |x| + |silu(g)| |W13_u| |x|) and |w| |W2| |h|, the
    magnitudes that a float32 evaluation's error is bounded by.
    """
    x = bf16_bits_to_f64(x_bits)
    ids = np.asarray(ids)
    w = np.asarray(w, np.float32).astype(np.float64)
    H = x.shape[1]
    out = np.zeros((x.shape[0], H))
    mag_gu, mag_h = np.zeros_like(out), np.zeros_like(out)
    valid = ids[ids >= 0]
    for e in np.unique(valid):
        a = w13(int(e))
        if a is None:
            continue
        I = a.shape[0] // 2
        b = w2(int(e))
        t, j = np.nonzero(ids == e)
        gu, m = x[t] @ a.T, np.abs(x[t]) @ np.abs(a).T
        g, u = gu[:, :I], gu[:, I:]
        sg = 1.0 / (1.0 + np.exp(-g))
        h = g * sg * u
        dh = 1.1 * m[:, :I] * (np.abs(u) + m[:, I:] * 2.0 ** -16) + np.abs(g * sg) * m[:, I:]
        wt = w[t, j][:, None]
        np.add.at(out, t, wt * (h @ b.T))
        np.add.at(mag_gu, t, np.abs(wt) * (dh @ np.abs(b).T))
        np.add.at(mag_h, t, np.abs(wt) * (np.abs(h) @ np.abs(b).T))
    return out, round_to_bf16_bits(out), (mag_gu, mag_h)
