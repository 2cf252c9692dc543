"""The few-token experts where a value leaves the ordinary range, or another token's does.

* An expert with NaN or infinite scales reaches the tokens that picked it and no other bit.
"""
import numpy as np
import pytest

import synth
from few_util import FORMATS, random_codes
from gpu_util import bf16_bits, to_dev, to_dev_bf16

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
