"""The balance loss's gradient for sigmoid scores whose logits are high, where 1 - sigmoid(l) is about e^-l.

The bound is relative to p (1 - sigmoid), the gradient's own size. With u = 2^-24 and |l| <= 60:
* e^-l: the product l log2 e, its constant and the exponential put it off by (2 |l| + 2) u <= 122 u;
* sigmoid = 1 / (1 + e^-l): the exponential's error times e^-l sigmoid, at most that of l = -12 (26 u), the addition and
  the reciprocal: 30 u. p is that over the sum of at most 1024 such: 2 * 30 u, the sum's 24 u and two roundings: 86 u;
* 1 - sigmoid: by subtraction below one half, 30 u; else the product e^-l sigmoid, 122 u + 30 u + u;
* w_j - sum of w p: 4 u of |w_j|, and 90 u + 24 u of sum |w| p.
In all less than 86 + 153 + 118 + 4 u < 512 u = 2^-15 of p (1 - sigmoid) (|w_j| + sum |w| p). A BF16 gradient is off by
another half step.
"""
import numpy as np
import pytest

import oracle
from gpu_util import bf16_ulp, to_dev

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no GPU", allow_module_level=True)

import w8a8_fp8_linear_amd as w8  # noqa: E402

COEF = 0.01


def _bound(l, ids, S, p):
    T, E = l.shape
    k, L = ids.shape[1], T // S
    valid = (ids >= 0) & (ids < E)
    size = p * np.exp(-np.logaddexp(0.0, l.astype(np.float64)))  # p (1 - sigmoid)
    err = np.zeros((T, E))
    for s in range(S):
        rows = np.arange(s * L, (s + 1) * L)
        c = np.bincount(ids[rows][valid[rows]], minlength=E)
        rows = rows[valid[rows].any(1)]
        w = np.abs(E * c / (k * rows.size) - 1) * COEF / (S * rows.size)
        err[rows] = 2.0 ** -15 * size[rows] * (w + (p[rows] * w).sum(1, keepdims=True))
    return err + 1e-37


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("S,L,E,k", [(1, 40, 7, 2), (1, 64, 192, 4), (2, 50, 40, 3), (3, 200, 128, 4), (2, 60, 300, 5)])
def test_high_logits(S, L, E, k, bf16):
    """Tokens of all high logits (12 to 60, and every one alike), tokens with a few of them, ordinary tokens."""
    print(f"[balance] high {S}x{L} E{E} k{k} {bf16}", flush=True)
    rng = np.random.default_rng(S + L + E)
    l = (rng.standard_normal((S * L, E)) * 2 + rng.standard_normal(E)).clip(-12, 12)
    kind = np.arange(S * L) % 4
    l[kind == 0] = rng.uniform(12.0, 60.0, ((kind == 0).sum(), E))
    l[kind == 1] = np.where(rng.random(((kind == 1).sum(), E)) < 0.2, rng.uniform(12.0, 60.0, ((kind == 1).sum(), E)), l[kind == 1])
    l[kind == 2] = np.linspace(9.0, 58.0, (kind == 2).sum())[:, None]
    t = torch.from_numpy(l.astype(np.float32))
    t = t.bfloat16() if bf16 else t
    l = t.float().numpy()
    ids = np.argsort(rng.random((S * L, E)) - 0.2 * (np.arange(E) < E // 2), axis=1)[:, :k].astype(np.int32)
    ids[::9] = -1
    grad = w8.moe_balance_loss(t.cuda(), to_dev(ids), coef=COEF, sequences=S, score="sigmoid")[2].double().cpu().numpy()
    _, _, ref, p = oracle.balance_loss(l, ids, COEF, S, "sigmoid")
    err = _bound(l, ids, S, p) + (0.5 * bf16_ulp(grad) if bf16 else 0.0)
    worst = np.abs(grad - ref) / err
    assert worst.max() <= 1.0, (worst.max(), np.unravel_index(worst.argmax(), worst.shape))


def test_very_high_logits_stay_finite():
    """From about 88 on the slope leaves float32's range and the gradient is zero; nothing becomes NaN on the way."""
    l = torch.tensor([[80.0, 100.0, 1e4, 3e38], [-3e38, 3e38, -100.0, 100.0]], device="cuda")
    ids = torch.tensor([[0], [1]], dtype=torch.int32, device="cuda")
    loss, _, grad = w8.moe_balance_loss(l, ids, score="sigmoid")
    ref = oracle.balance_loss(l.cpu().numpy(), ids.cpu().numpy(), 1.0, 1, "sigmoid")
    # p as in the bound above; 86 u of each, times |w| <= 2 n coef / n
    assert abs(loss.item() - ref[0]) <= 2.0 ** -15 * 2 and bool(grad.isfinite().all())
    assert np.abs(grad.double().cpu().numpy() - ref[2]).max() <= 1e-37 + 2.0 ** -15 * np.abs(ref[2]).max()
