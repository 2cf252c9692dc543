"""Helpers of the block-scaled FP8 tests (test infrastructure)."""
from __future__ import annotations

import numpy as np

import oracle
import synth
from gpu_util import MFMA_GROUP_ERR, U32, bf16_ulp
from moe_util import swiglu_bound


def weights(rng, *shape):
    """float32 weights in BF16 values whose rows differ in size, so that neighbouring blocks' scales do."""
    w = synth.bf16_bits_to_f32(synth.weights(rng, shape))
    return synth.bf16_bits_to_f32(synth.f32_to_bf16_bits(w * np.exp(0.5 * rng.standard_normal((*shape[:-1], 1))).astype(np.float32)))


def quantized_stack(w):
    """[E, N, K] float32 -> (codes, scales) stacked."""
    parts = [oracle.quantize_weight_blocks(m) for m in w]
    return np.stack([p[0] for p in parts]), np.stack([p[1] for p in parts])


def product_err(K, mag):
    """Bound on |sum_gpu32 - sum64| of one product from the sum of the products' magnitudes: each group of 8 loses at
    most 8 x 2^-13 of its largest (gpu_util); the K / 128 block sums are each scaled and added with one rounding, the
    product of the scales has one, the instruction's own additions and the four parts of K a few."""
    return (MFMA_GROUP_ERR + (K / 128 + 8) * U32) * 1.01 * mag


def violations(got_bits, ref64, err):
    g = oracle.bf16_bits_to_f64(got_bits)
    return int((np.abs(g - ref64) > err + 0.5 * bf16_ulp(g) + 1e-37).sum())


def hidden_bound(h32, dh):
    """The oracle's quantised h (values), how far a GPU's may be off, given |h_gpu - h32| <= dh, and its scales [rows, blocks]: a block's scale
    moves by at most max dh / 448 and a rounding, and a code lies between those of the ends of its value's range."""
    q, s = oracle.quantize_row_blocks(h32)
    s_el = np.repeat(s.astype(np.float64).T, 128, axis=1)[:, :h32.shape[1]]
    dmax = np.stack([dh[:, b:b + 128].max(1) for b in range(0, h32.shape[1], 128)], 1)
    ds = np.repeat(dmax, 128, axis=1)[:, :h32.shape[1]] / 448.0 + 2.0 ** -22 * s_el
    v = h32 / s_el
    dv = dh / s_el + np.abs(v) * (ds / s_el) * 1.01 + 2.0 ** -22 * np.abs(v)
    ref = oracle.decode(q)
    lo = oracle.decode(oracle.encode((v - dv).astype(np.float32)))
    hi = oracle.decode(oracle.encode((v + dv).astype(np.float32)))
    off = np.maximum(np.abs(lo - ref), np.abs(hi - ref)) * s_el + np.maximum(np.abs(lo), np.abs(hi)) * ds
    return ref * s_el, off, s.T.astype(np.float64)


def moe_ref(qx, sx, ids, tw, q13, s13, q2, s2, tokens=None):
    """(out64, err) of the pass for ``tokens`` (default all): err bounds |out_gpu - out64| before the last rounding."""
    T, k = ids.shape
    E, H, I = q2.shape
    tokens = np.arange(T) if tokens is None else np.asarray(tokens)
    x = oracle.row_values(qx, sx)
    out, err, mag = (np.zeros((T, H)) for _ in range(3))
    sel = ids[tokens]
    for e in np.unique(sel[(sel >= 0) & (sel < E)]):
        ti, j = np.nonzero(sel == e)
        t = tokens[ti]
        w13, w2 = oracle.weight_values(q13[e], s13[e]), oracle.weight_values(q2[e], s2[e])
        gu = x[t] @ w13.T
        h32, dh = swiglu_bound(gu, product_err(H, np.abs(x[t]) @ np.abs(w13).T))
        h, off, hs = hidden_bound(h32, dh)
        w = np.asarray(tw, np.float64)[t, j][:, None]
        y, ymag = h @ w2.T, (np.abs(h) + off) @ np.abs(w2).T
        np.add.at(out, t, y * w)
        np.add.at(err, t, (off @ np.abs(w2).T + product_err(I, ymag)) * np.abs(w))
        np.add.at(mag, t, np.abs(y * w))
        if T * k > min(256, 8 * E):
            # beyond the few-row kernels a copy is float16 times a power of two p: off by half a step, 2^-11 of its
            # value, or by half of float16's smallest step, 2^-25 p. With size the sum of the blocks' scale products,
            # 2^x <= size and 2^y <= |tw| the powers next below, p = 2^(x + y + 2 + 26 - 15) <= 2^13 size |tw|.
            # 1.01 for the roundings of what is rounded and of size.
            size = np.repeat(1.01 * hs @ s2[e].astype(np.float64).T, 128, axis=1)[:, :H] * np.abs(w)
            np.add.at(err, t, 2.0 ** -11 * (np.abs(y * w) + off @ np.abs(w2).T * np.abs(w)) * 1.01 + 2.0 ** (13 - 25) * size)
    return out[tokens], (err + (k + 3) * U32 * 1.01 * mag)[tokens]


def balance_bound(logits, ids, coef, sequences, score, p, bf16):
    """How far a GPU's gradient may be from oracle.balance_loss's.

    Scores: the exponential's argument is within 30 here, times log2 e rounded to float32 (30 * 1.45 * 2^-24 off), the
    hardware exponential and reciprocal within a few ulps, the sum of up to 1024 of them and the division: eps = 2^-17
    relative, taken for p and for 1 - sigmoid times p. A gradient is p (w_j - sum w p) with w = (f - 1) * base: both
    factors' errors are relative to p, |w_j| and sum |w| p, four such errors in all; a BF16 gradient is off by another half step."""
    T, E = logits.shape
    k, L = ids.shape[1], T // sequences
    valid = (ids >= 0) & (ids < E)
    err = np.zeros((T, E))
    for s in range(sequences):
        rows = np.arange(s * L, (s + 1) * L)
        c = np.bincount(ids[rows][valid[rows]], minlength=E)
        rows = rows[valid[rows].any(1)]
        if rows.size:
            w = np.abs(E * c / (k * rows.size) - 1) * coef / (sequences * rows.size)
            err[rows] = 4 * 2.0 ** -17 * p[rows] * (w + (p[rows] * w).sum(1, keepdims=True))
    return err + 1e-37
