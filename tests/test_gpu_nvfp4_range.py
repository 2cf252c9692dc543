"""NVFP4 quantisation and the 4-bit products at the ends of the number range.

* nvfp4_quantize with a given scale: values far beyond what the scale can hold saturate, with their sign;
  at the smallest scales quotients next to a border round as a division does.
* mxfp4_gemm at the ends of the scale byte.
"""
import numpy as np
import pytest

import oracle
import synth
from gpu_util import bf16_bits, to_dev, to_dev_bf16

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no GPU", allow_module_level=True)

import w8a8_fp8_linear_amd as w8  # noqa: E402


def _matches(x_bits, gscale=None):
    """Codes, block scales and group scale of a matrix against the oracle's, bit for bit."""
    given = None if gscale is None else to_dev(np.float32([gscale]))
    q, s, g = w8.nvfp4_quantize(to_dev_bf16(x_bits), gscale=given)
    with np.errstate(over="ignore"):
        rq, rs, rg = oracle.nvfp4_quantize(synth.bf16_bits_to_f32(x_bits), g=gscale)
    assert g.item() == rg
    assert np.array_equal(s.cpu().numpy(), rs)
    bad = np.nonzero((q.cpu().numpy() != rq).any(1))[0]
    assert not bad.size, (int((q.cpu().numpy() != rq).sum()), bad[:4])


def _every_bf16():
    bits = np.arange(0x7F80, dtype=np.uint32).astype(np.uint16)
    return np.concatenate([bits, bits | 0x8000]).reshape(16, -1)


@pytest.mark.parametrize("g", [2.0 ** -96, 2.0 ** -60, 1e-3, 1.0, 3.7e4, 2.0 ** 112])
def test_given_scale_with_every_bf16_value(g):
    """Every finite BF16 value, in ascending blocks and in blocks whose values are far apart: where x / d passes the
    largest float32 it still saturates at 6 with the sign of x."""
    print(f"[nvfp4 given] g={g}", flush=True)
    x = _every_bf16()
    _matches(x, np.float32(g))
    mixed = np.random.default_rng(3).permutation(x.reshape(-1)).reshape(x.shape)
    _matches(mixed, np.float32(g))
    _matches(synth.f32_to_bf16_bits(np.float32([[2.0 ** 42, -2.0 ** 42, 2.55e38, -2.55e38] * 4])), np.float32(g))


@pytest.mark.parametrize("given", [True, False])
def test_quotients_next_to_a_border_at_the_smallest_scales(given):
    """Scales near the smallest: x / d within a float32 step of a border between two codes is rounded as a division does.

    With d = 2^-104 (1 - 2^-24) and x = 2^-106, x / d is 0.25 (1 + 2^-24 + 2^-48): its float32 is above 0.25, so the code is
    1 (0.5). What is left of x after the product of a first quotient with d needs bits below the smallest float32 there."""
    g = np.float32(2.0 ** -95) * np.float32(1 - 2.0 ** -24)
    rng = np.random.default_rng(6)
    rows = []
    for k in range(64):
        # the block's maximum picks the scale byte (1 to some tens), its values the borders 0.25 .. 5 times d and near
        top = np.float32(2.0 ** -102) * np.float32(2.0 ** (k % 6)) * np.float32(1 + rng.integers(0, 128) / 128)
        near = np.float32(rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 0.5, 3.0], 15) * 2.0 ** -104)
        near = near * np.float32(2.0) ** rng.integers(0, 5, 15).astype(np.float32) * (1 + rng.integers(-1, 2, 15) / 128).astype(np.float32)
        rows.append(np.concatenate([[top], near * rng.choice([-1, 1], 15)]))
    rows.append(np.float32([2.0 ** -102] + [2.0 ** -106, -2.0 ** -106] * 7 + [2.0 ** -105]))
    x = np.float32(rows).reshape(-1, 16)
    if given:
        _matches(synth.f32_to_bf16_bits(x), g)
    else:
        # the group's maximum makes the scale: amax / 2688 in the same binade as g
        for amax in (2.0 ** -84, 2.0 ** -84 * (1 + 5 / 128), 2.0 ** -83 * (1 + 39 / 128), 2.0 ** -82 * (1 + 125 / 128)):
            y = np.concatenate([np.float32([[amax] + [0] * 15]), x])
            _matches(synth.f32_to_bf16_bits(y))


@pytest.mark.parametrize("M", [5, 20, 40, 700, 2100])
def test_mxfp4_products_at_both_ends_of_the_scale(M):
    """Every code under every scale byte that the format's quantiser writes (0 .. 252), one product a result: exact before the
    last rounding, subnormal values among them."""
    K, N = 32, 4112
    codes = np.tile(np.arange(K) % 16, (N, 1)).astype(np.uint8)
    q = (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)
    s = (np.arange(N) % 253).astype(np.uint8)[:, None]
    val = oracle.mx_dequant(q, s)
    for at in (1.0, 2.0 ** 20, 2.0 ** -20):
        x = np.zeros((M, K), np.float32)
        x[np.arange(M), np.arange(M) % K] = at
        y = oracle.bf16_bits_to_f64(bf16_bits(w8.mxfp4_gemm(to_dev_bf16(synth.f32_to_bf16_bits(x)), to_dev(q), to_dev(s))))
        ref = oracle.bf16_bits_to_f64(oracle.round_to_bf16_bits(val.T[np.arange(M) % K] * at))
        assert np.array_equal(y, ref)


@pytest.mark.parametrize("M", [5, 40, 2100])
def test_mxfp4_scale_bytes_beyond_the_range(M):
    """253 and 254: a value of 2^128 or more is infinite, as in float32, the others are exact; 255 is NaN."""
    K, N = 32, 4096
    code, byte = np.arange(N) % 16, 253 + np.arange(N) // 16 % 3
    q = np.repeat((code | (code << 4)).astype(np.uint8)[:, None], K // 2, 1)
    x = np.full((M, K), 2.0 ** -20, np.float32)
    y = oracle.bf16_bits_to_f64(bf16_bits(w8.mxfp4_gemm(to_dev_bf16(synth.f32_to_bf16_bits(x)), to_dev(q),
                                                    to_dev(byte.astype(np.uint8)[:, None]))))
    val = oracle.e2m1_decode(code) * np.exp2(byte - 127.0)
    with np.errstate(invalid="ignore"):
        val = np.where(np.abs(val) >= 2.0 ** 128, np.sign(val) * np.inf, val) * K * 2.0 ** -20
    val[byte == 255] = np.nan
    assert np.array_equal(y, np.tile(val, (M, 1)), equal_nan=True)
