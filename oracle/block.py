"""FP8 with a scale per block of 128, and the router's balance loss — test
infrastructure only.

The scheme is the per-row one (``quant``; Lernex/Metis-1.6-Logos-FP8, "What is
in FP8") on smaller pieces: a scale per 128 consecutive values of a row of
activations, per 128 x 128 values of a weight matrix, counted from index 0, the
last of a dimension shorter. Every block by itself: s = fl32(amax / 448), 1 for
an all-zero block; the code is E4M3 of fl32(x / s), to nearest even. Scales of
activations are kept as [blocks of K, M], of weights as [blocks of N, blocks of K].

The expert pass follows ``moe``: h = silu(g) * u rounded to float32 and quantised
by rows of 128, the weighted copies summed at full precision, one BF16 rounding.

The balance loss of a sequence with counts c_e of routed copies, n tokens that
name a valid expert, k copies a token and scores p that sum to one:
coef * sum_e (E c_e / (k n)) * mean_t p_e, averaged over the sequences; its
gradient keeps c constant.
"""
from __future__ import annotations

import numpy as np

from .bf16 import round_to_bf16_bits
from .e4m3 import decode, encode
from .moe import swiglu_f32
from .quant import row_scale

__all__ = ["BLOCK", "quantize_row_blocks", "quantize_weight_blocks", "row_values", "weight_values", "block_linear",
           "moe_block_pass", "balance_loss"]

BLOCK = 128


def _codes(x, s):
    return encode((x.astype(np.float64) / s.astype(np.float64)).astype(np.float32))


def quantize_row_blocks(x):
    """float32 [M, K] -> (codes uint8 [M, K], scales float32 [ceil(K/128), M])."""
    x = np.asarray(x, np.float32)
    M, K = x.shape
    q = np.zeros((M, K), np.uint8)
    s = np.ones((-(-K // BLOCK), M), np.float32)
    for b, k in enumerate(range(0, K, BLOCK)):
        piece = x[:, k:k + BLOCK]
        s[b] = row_scale(np.abs(piece).max(1)) if M else s[b]
        q[:, k:k + BLOCK] = _codes(piece, s[b][:, None])
    return q, s


def quantize_weight_blocks(w):
    """float32 [N, K] -> (codes uint8 [N, K], scales float32 [ceil(N/128), ceil(K/128)])."""
    w = np.asarray(w, np.float32)
    N, K = w.shape
    q = np.zeros((N, K), np.uint8)
    s = np.ones((-(-N // BLOCK), -(-K // BLOCK)), np.float32)
    for a, n in enumerate(range(0, N, BLOCK)):
        for b, k in enumerate(range(0, K, BLOCK)):
            piece = w[n:n + BLOCK, k:k + BLOCK]
            s[a, b] = row_scale(np.abs(piece).max())
            q[n:n + BLOCK, k:k + BLOCK] = _codes(piece, s[a, b])
    return q, s


def row_values(q, s):
    """Codes [M, K] and scales [blocks, M] -> float64 values."""
    return decode(q) * np.repeat(np.asarray(s, np.float64).T, BLOCK, axis=1)[:, :q.shape[1]]


def weight_values(q, s):
    """Codes [N, K] and scales [blocks, blocks] -> float64 values."""
    r = np.repeat(np.repeat(np.asarray(s, np.float64), BLOCK, axis=0), BLOCK, axis=1)
    return decode(q) * r[:q.shape[0], :q.shape[1]]


def block_linear(qx, sx, qw, sw):
    """(y float64 [M, N], sum of the products' magnitudes [M, N])."""
    x, w = row_values(qx, sx), weight_values(qw, sw)
    return x @ w.T, np.abs(x) @ np.abs(w).T


def moe_block_pass(qx, sx, ids, tw, q13, s13, q2, s2):
    """One routed-expert pass: (out float64 [T, H], its BF16 bits)."""
    T, k = ids.shape
    E, H, I = q2.shape
    x = row_values(qx, sx)
    out = np.zeros((T, H))
    for e in range(E):
        t, j = np.nonzero(ids == e)
        if t.size == 0:
            continue
        gu = x[t] @ weight_values(q13[e], s13[e]).T
        h = row_values(*quantize_row_blocks(swiglu_f32(gu)))
        np.add.at(out, t, (h @ weight_values(q2[e], s2[e]).T) * np.asarray(tw, np.float64)[t, j][:, None])
    return out, round_to_bf16_bits(out)


def balance_loss(logits, ids, coef, sequences=1, score="softmax"):
    """(loss float, counts int64 [S, E], gradient float64 [T, E], scores p [T, E]) of float64 logits [T, E]."""
    logits = np.asarray(logits, np.float64)
    T, E = logits.shape
    k, L = ids.shape[1], T // sequences
    valid = (ids >= 0) & (ids < E)
    counts = np.zeros((sequences, E), np.int64)
    grad, p = np.zeros((T, E)), np.zeros((T, E))
    loss = 0.0
    for s in range(sequences):
        rows = np.arange(s * L, (s + 1) * L)
        counts[s] = np.bincount(ids[rows][valid[rows]], minlength=E)
        rows = rows[valid[rows].any(1)]
        n = rows.size
        if n == 0:
            continue
        l = logits[rows]
        with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
            if score == "softmax":
                top = l.max(1, keepdims=True)
                v = np.exp(l - np.where(np.isneginf(top), 0.0, top))
                slope = np.ones_like(v)
            else:
                # over their largest: sigmoids themselves end at e^-745
                v = -np.logaddexp(0.0, -l)
                slope = -np.expm1(v)
                top = v.max(1, keepdims=True)
                v = np.exp(v - np.where(np.isneginf(top), 0.0, top))
        z = v.sum(1, keepdims=True)
        q = np.divide(v, z, out=np.zeros_like(v), where=z > 0)
        f = E * counts[s] / (k * n)
        loss += coef / sequences * float((f * q.mean(0)).sum())
        g = coef / (sequences * n) * f
        grad[rows] = q * slope * (g - (q * g).sum(1, keepdims=True))
        p[rows] = q
    return loss, counts, grad, p
