"""The balance loss's f - 1 = (c E - k n) / (k n) is rounded to float32 once.

Every token's logits bar all experts but one (p = 1 there, exactly), and coef = n makes (f - 1) coef / n the quotient
itself: the loss is n times (the rounded quotient + 1), summed exactly in float64 and rounded once.
"""
import numpy as np
import pytest

from gpu_util import to_dev

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no GPU", allow_module_level=True)

import w8a8_fp8_linear_amd as w8  # noqa: E402


@pytest.mark.parametrize("T,E,k", [(3000, 1000, 64), (30, 1000, 64), (5000, 700, 37)])
def test_quotient_is_rounded_once(T, E, k):
    logits = torch.full((T, E), float("-inf"), device="cuda")
    logits[:, 0] = 1.0
    rng = np.random.default_rng(T + E)
    wrong = []
    for _ in range(12):
        ids = np.zeros((T, k), np.int32)
        ids[rng.random((T, k)) < rng.uniform(0, 0.6)] = 1
        ids[:, 0] = 0
        c = int((ids == 0).sum())
        loss, counts, _ = w8.moe_balance_loss(logits, to_dev(ids), coef=float(T))
        assert int(counts[0, 0]) == c
        quotient = np.float32((c * E - k * T) / (k * T))  # whole numbers below 2^53: one rounding to float64, one to float32
        want = np.float32(T * (float(quotient) + 1.0))
        if np.float32(loss.item()) != want:
            wrong.append((c, loss.item(), float(want)))
    assert not wrong, wrong
