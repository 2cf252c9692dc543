"""The few-token experts where a value leaves the ordinary range, or another token's does.

* An expert with NaN or infinite scales reaches the tokens that picked it and no other bit.
* h between the two projections keeps float32's 24 bits and its range, infinities among it.
"""
import numpy as np
import pytest

import oracle
import synth
from few_util import FORMATS, random_codes
from gpu_util import U32, bf16_bits, bf16_ulp, to_dev, to_dev_bf16

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no GPU", allow_module_level=True)

import w8a8_fp8_linear_amd as w8  # noqa: E402


def _dev(w):
    return tuple(to_dev(a) for a in w)


def _poisoned(fmt, w, e):
    """The scales of expert e without a number: NaN, or an infinity where a scale is a float32."""
    codes, scales, *g = w
    scales = scales.copy()
    scales[e] = {"fp8": np.inf, "mxfp4": 0xFF, "nvfp4": 0x7F}[fmt]
    return (codes, scales, *g)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,E,k", [(2, 9, 2), (5, 192, 4), (8, 40, 8), (12, 60, 3), (40, 12, 2)])
def test_an_experts_nan_stays_with_its_tokens(fmt, T, E, k):
    """out[t] sums over the token's own experts: the others' NaN is no part of it, on every path."""
    print(f"[few NaN] {fmt} T={T} E={E} k={k}", flush=True)
    rng = np.random.default_rng(T * E + k)
    H, I = 96, 160
    w13, _ = random_codes(rng, fmt, E, 2 * I, H)
    w2, _ = random_codes(rng, fmt, E, H, I)
    x = to_dev_bf16(synth.activations(rng, T, H))
    ids, tw = synth.routing(rng, T, E, k)
    e = int(ids[0, 0])
    picked = (ids == e).any(1)
    ids, tw = to_dev(ids), to_dev(tw)
    want = bf16_bits(w8.moe_few_tokens(x, ids, tw, _dev(w13), _dev(w2)))
    for bad in ((w13, _poisoned(fmt, w2, e)), (_poisoned(fmt, w13, e), w2)):
        got = bf16_bits(w8.moe_few_tokens(x, ids, tw, *(_dev(w) for w in bad)))
        assert np.array_equal(got[~picked], want[~picked])
        assert ((got[picked] & 0x7F80) == 0x7F80).all()


def _ones(fmt, *shape):
    """The codes and scales of weights that are all 0, and the code of 1.0 with its place in a byte."""
    *lead, rows, K = shape
    if fmt == "fp8":
        return np.zeros(shape, np.uint8), np.ones((*lead, rows), np.float32)
    q = np.zeros((*lead, rows, K // 2), np.uint8)
    s = np.full((*lead, rows, K // (32 if fmt == "mxfp4" else 16)), 127 if fmt == "mxfp4" else 0x38, np.uint8)
    return (q, s) if fmt == "mxfp4" else (q, s, np.ones(lead, np.float32))


def _set(fmt, w, e, row, k, negative=False):
    """Weight [e, row, k] = +-1."""
    if fmt == "fp8":
        w[0][e, row, k] = 0xB8 if negative else 0x38
    else:
        w[0][e, row, k // 2] |= (0xA if negative else 0x2) << (4 * (k % 2))


# tokens that take: the small down projection, the grouped one by copies and by experts with one
# column tile, and with several
_STEPS = [(1, 5), (5, 40), (12, 60), (14, 3), (40, 2)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,E", _STEPS)
def test_h_is_held_in_float32(fmt, T, E):
    """Two experts whose h differ by a part in 4096, weighted 1 and -1: what is left shows how h was held.

    Expert 0: h = silu(g) x. Expert 1: h = silu(g) (x + x / 4096), the same g, so silu's own error is a part of the
    difference alone. In units of 2^-24 |h|: each product silu * u rounds once (1 each); u of expert 1 is a sum of two
    products on the matrix cores (2^-20: 16, and 1); each W2 row reads a single h, whose sum is 2^-20 off at most (16
    and 3 additions, each); the weighted rows add once (1). 60 in all; 16 bits of h would be 128 for each side."""
    print(f"[few h] {fmt} T={T} E={E}", flush=True)
    rng = np.random.default_rng(T + E)
    I, H = 64, 192
    xs = synth.bf16_bits_to_f32(synth.activations(rng, T, I)) + np.float32(0)
    xs = synth.bf16_bits_to_f32(synth.f32_to_bf16_bits(np.where(np.abs(xs) < 0.01, np.float32(0.5), xs)))
    g = synth.bf16_bits_to_f32(synth.f32_to_bf16_bits(rng.uniform(-4, 4, (T, I)).astype(np.float32)))
    x = np.concatenate([xs, xs / 4096, g], 1)
    w13, w2 = _ones(fmt, E, 2 * I, H), _ones(fmt, E, H, I)
    for e in range(2):
        for i in range(I):
            _set(fmt, w13, e, i, 2 * I + i)          # gate
            _set(fmt, w13, e, I + i, i)              # up
            if e:
                _set(fmt, w13, e, I + i, I + i)
        for c in range(H):
            _set(fmt, w2, e, c, (5 * c) % I, negative=bool(c & 1))
    ids = np.tile(np.int32([0, 1]), (T, 1))
    tw = np.tile(np.float32([1, -1]), (T, 1))
    got = w8.moe_few_tokens(to_dev_bf16(synth.f32_to_bf16_bits(x)), to_dev(ids), to_dev(tw), _dev(w13), _dev(w2))
    y = oracle.bf16_bits_to_f64(bf16_bits(got))
    g64 = g.astype(np.float64)
    h = g64 / (1 + np.exp(-g64)) * xs
    c = np.arange(H)
    h = h[:, (5 * c) % I] * np.where(c & 1, -1.0, 1.0)
    ref = h - h * (1 + 2.0 ** -12)
    off = np.abs(y - ref) - (60 * U32 * np.abs(h) + 2.0 ** -18 * np.abs(ref) + 0.5 * bf16_ulp(y))
    assert (off <= 0).all(), (int((off > 0).sum()), float((off / (U32 * np.abs(h))).max()))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,E", _STEPS)
def test_h_beyond_bf16_and_infinite(fmt, T, E):
    """h of each token has one value that is not 0: 2^127 (2 - 2^-15), which is finite and above the largest BF16 value,
    or +-infinity. W2 reads it with both signs; the outputs are that value's multiples, the router weight being 2^-10."""
    print(f"[few large h] {fmt} T={T} E={E}", flush=True)
    I, H = 64, 96
    x = np.zeros((T, H), np.float32)
    top = np.float32(2 - 2.0 ** -7) * np.float32(2.0 ** 122)
    kind = np.arange(T) % 3
    x[:, 0] = np.where(kind == 2, -top, top)
    x[:, 1] = x[:, 0] * np.float32(2.0 ** -8)       # u = 2^122 (2 - 2^-15) in two BF16 values
    x[:, 2] = np.where(kind == 0, 32.0, 4096.0)     # silu(32) = 32: 1 + e^-32 is 1 in float32
    w13, w2 = _ones(fmt, E, 2 * I, H), _ones(fmt, E, H, I)
    for e in range(E):
        _set(fmt, w13, e, 7, 2)
        _set(fmt, w13, e, I + 7, 0)
        _set(fmt, w13, e, I + 7, 1)
        for c in range(H):
            for i in range(I):
                _set(fmt, w2, e, c, i, negative=bool(c & 1))   # no zero: infinity times 0 is NaN
    ids = (np.arange(T, dtype=np.int32) % E)[:, None]
    tw = np.full((T, 1), 2.0 ** -10, np.float32)
    got = w8.moe_few_tokens(to_dev_bf16(synth.f32_to_bf16_bits(x)), to_dev(ids), to_dev(tw), _dev(w13), _dev(w2))
    y = oracle.bf16_bits_to_f64(bf16_bits(got))
    value = np.where(kind == 0, 2.0 ** 118, np.where(kind == 1, np.inf, -np.inf))   # 2^117 (2 - 2^-15) rounds up to 2^118
    assert np.array_equal(y, value[:, None] * np.where(np.arange(H) & 1, -1.0, 1.0))
