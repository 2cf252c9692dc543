"""NVFP4 quantisation and the 4-bit products at the ends of the number range.

* nvfp4_quantize with a given scale: values far beyond what the scale can hold saturate, with their sign.
"""
import numpy as np
import pytest

import oracle
import synth
from gpu_util import to_dev, to_dev_bf16

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
