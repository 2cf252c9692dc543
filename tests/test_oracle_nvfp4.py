"""Pins of the oracle's NVFP4 format, its products with BF16 activations, the
router and the default-maths expert pass.

* Quantiser: brute force with exact rationals over the rule's steps (float32
  roundings by a second route, numpy's float32 arithmetic); the largest value
  of a group comes back exactly; scaling a group by a power of two moves only
  its scale; all-zero groups and blocks; the smallest scale.
* Products: exact rationals over several blocks, from the golden E2M1 table.
* Router: one-hot rows, equal scores (lower index first), the bias moving the
  choice and not the weights.
* Expert pass: one expert with weight one is the plain chain; a token that
  names an expert twice; ids that are dropped.
"""
from fractions import Fraction

import numpy as np

import oracle
from synth import bf16_bits_to_f32, f32_to_bf16_bits


def _bf16(a):
    return bf16_bits_to_f32(f32_to_bf16_bits(np.asarray(a, np.float32)))


def test_quantiser_brute_force():
    rng = np.random.default_rng(3)
    x = _bf16(rng.standard_normal((6, 64)) * np.exp2(rng.integers(-6, 6, (6, 1))))
    x[2, 16:32] = 0
    q, s, g = oracle.nvfp4_quantize(x)
    assert g == np.float32(np.abs(x).max()) / np.float32(2688)
    mags = [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    codes = oracle.mx_unpack(q)
    scales = oracle.decode_table()[:127]
    for r in range(6):
        for b in range(4):
            v = x[r, 16 * b:16 * b + 16]
            t = (np.abs(v).max() / np.float32(6)) / g          # numpy float32 arithmetic
            near = np.abs(scales - float(t)).argmin()
            assert s[r, b] == near or abs(abs(scales[s[r, b]] - float(t)) - abs(scales[near] - float(t))) == 0
            d = np.float32(scales[s[r, b]]) * g
            for i in range(16):
                c = codes[r, 16 * b + i]
                if d == 0:
                    assert c & 7 == 0
                    continue
                f = Fraction(float(abs(v[i]) / d))
                best = min(abs(f - Fraction(m)) for m in mags)
                assert abs(min(f, 6) - Fraction(mags[c & 7])) == min(best, abs(min(f, 6) - Fraction(mags[c & 7])))
                if f <= 6:
                    assert abs(f - Fraction(mags[c & 7])) == best
                assert (c >> 3) == np.signbit(v[i])


def test_quantiser_properties():
    rng = np.random.default_rng(4)
    x = _bf16(rng.standard_normal((8, 96)))
    q, s, g = oracle.nvfp4_quantize(x)
    q2, s2, g2 = oracle.nvfp4_quantize(x * np.float32(2.0 ** -20))
    assert np.array_equal(q, q2) and np.array_equal(s, s2) and g2 == g * np.float32(2.0 ** -20)
    back = oracle.nvfp4_dequant_f32(q, s, g)
    i = np.unravel_index(np.abs(x).argmax(), x.shape)
    assert abs(back[i] - x[i]) <= 2.0 ** -22 * abs(x[i])
    # off by at most half the spacing of the codes (1 at most, below 6) of the block's scale, and by half a step
    # of that scale (2^-4 relative, its values being normal here) at the largest magnitude
    d = np.repeat(oracle.decode(s) * float(g), 16, axis=1)
    assert np.all(np.abs(back - x) <= d * (1 + 6 * 2.0 ** -4) * 1.0001)
    qz, sz, gz = oracle.nvfp4_quantize(np.zeros((2, 32), np.float32))
    assert gz == 1 and not sz.any() and not (qz & 0x77).any()
    tiny = np.zeros((1, 16), np.float32)
    tiny[0, 3] = -2.0 ** -120
    qt, st, gt = oracle.nvfp4_quantize(tiny)
    assert gt == np.float32(oracle.NVFP4_GSCALE_MIN) and not st.any() and oracle.mx_unpack(qt)[0, 3] == 8


def test_given_scale_saturates():
    x = _bf16(np.linspace(-100, 100, 32).reshape(1, 32))
    q, s, g = oracle.nvfp4_quantize(x, g=2.0 ** -10)
    assert g == np.float32(2.0 ** -10) and np.all(oracle.decode(s) == 448)
    assert np.all(np.abs(oracle.e2m1_decode(oracle.mx_unpack(q)))[0, :8] == 6)


def test_products_exact_rationals():
    rng = np.random.default_rng(5)
    x = f32_to_bf16_bits(rng.standard_normal((3, 64)).astype(np.float32))
    q = rng.integers(0, 256, (4, 32), dtype=np.uint8)
    s = rng.integers(0, 0x78, (4, 4), dtype=np.uint8)
    e = rng.integers(120, 134, (4, 2), dtype=np.uint8)
    xf = [[Fraction(float(v)) for v in r] for r in bf16_bits_to_f32(x)]
    codes = oracle.mx_unpack(q)
    val = lambda c: Fraction([0, 0.5, 1, 1.5, 2, 3, 4, 6][c & 7]) * (-1 if c & 8 else 1)  # noqa: E731
    y, bits = oracle.w4a16_linear(x, q, s, g=np.float32(0.37))
    z, _ = oracle.w4a16_linear(x, q, e)
    for m in range(3):
        for n in range(4):
            a = sum(xf[m][k] * val(codes[n, k]) * Fraction(float(oracle.decode(s[n, k // 16]))) for k in range(64))
            assert abs(Fraction(y[m, n]) - a * Fraction(float(np.float32(0.37)))) <= Fraction(1, 2 ** 40) * (1 + abs(a))
            b = sum(xf[m][k] * val(codes[n, k]) * Fraction(2) ** (int(e[n, k // 32]) - 127) for k in range(64))
            assert abs(Fraction(z[m, n]) - b) <= Fraction(1, 2 ** 40) * (1 + abs(b))
    assert np.array_equal(bits, oracle.round_to_bf16_bits(y))


def test_router():
    E, H = 6, 16
    w = f32_to_bf16_bits(np.eye(E, H, dtype=np.float32))
    x = np.zeros((3, H), np.float32)
    x[0, :6] = [1, 3, 2, 3, 0, -1]      # a tie of experts 1 and 3
    x[1, :6] = [0, 0, 0, 0, 0, 0]       # all alike
    x[2, :6] = [5, 4, 3, 2, 1, 0]
    xb = f32_to_bf16_bits(x)
    for score in ("softmax", "sigmoid"):
        ids, wt, _ = oracle.router(xb, w, 3, score=score)
        assert ids.tolist() == [[1, 3, 2], [0, 1, 2], [0, 1, 2]]
        assert np.allclose(wt.sum(1), 1)
    bias = np.array([0, 0, 0, 0, 0, 10], np.float32)
    ids, wt, _ = oracle.router(xb, w, 2, bias=bias, renormalize=False, scale=2.0)
    assert ids[:, 0].tolist() == [5, 5, 5]
    p = np.exp(x[:, :6].astype(np.float64))
    p /= p.sum(1, keepdims=True)
    assert np.allclose(wt[:, 0], 2 * p[:, 5])


def test_wide_pass():
    rng = np.random.default_rng(6)
    a, b = rng.standard_normal((2, 32, 16)), rng.standard_normal((2, 16, 16))
    xb = f32_to_bf16_bits(rng.standard_normal((3, 16)).astype(np.float32))
    x = bf16_bits_to_f32(xb).astype(np.float64)

    def one(e):
        gu = x @ a[e].T
        return (gu[:, :16] / (1 + np.exp(-gu[:, :16])) * gu[:, 16:]) @ b[e].T

    take = lambda m: (lambda e: m[e])  # noqa: E731
    out, bits, _ = oracle.wide_pass(xb, np.array([[0], [1], [-1]]), np.ones((3, 1), np.float32), take(a), take(b))
    assert np.allclose(out[0], one(0)[0]) and np.allclose(out[1], one(1)[1]) and not out[2].any()
    assert np.array_equal(bits, oracle.round_to_bf16_bits(out))
    out, _, _ = oracle.wide_pass(xb, np.array([[1, 1]] * 3), np.float32([[0.25, 0.5]] * 3), take(a), take(b))
    assert np.allclose(out, 0.75 * one(1))
