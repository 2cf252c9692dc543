"""GPU parity of the balance loss: loss, counts and gradient against the 64-bit oracle and against differences;
padding, empty sequences, barred experts; both types and scores; the router's logits; graphs; refused arguments."""
import numpy as np
import pytest

import oracle
import synth
from block_util import balance_bound
from gpu_util import bf16_ulp, to_dev, to_dev_bf16

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no GPU", allow_module_level=True)

import w8a8_fp8_linear_amd as w8  # noqa: E402

COEF = 0.01


def _inputs(S, L, E, k, seed, bf16=False, pad=0.3):
    rng = np.random.default_rng(seed)
    l = (rng.standard_normal((S * L, E)) * 2 + rng.standard_normal(E)).clip(-12, 12).astype(np.float32)
    t = torch.from_numpy(l)
    if bf16:
        t = t.bfloat16()
        l = t.float().numpy()
    ids = np.argsort(-l, axis=1, kind="stable")[:, :k].astype(np.int32)
    drop = rng.random((S * L, k)) < pad
    ids[drop] = rng.choice([-1, E, -(1 << 31), (1 << 31) - 1], int(drop.sum()))
    return t.cuda(), l, ids


def _check(t, l, ids, S, score, coef=COEF):
    loss, counts, grad = w8.moe_balance_loss(t, to_dev(ids), coef=coef, sequences=S, score=score)
    torch.cuda.synchronize()
    rl, rc, rg, p = oracle.balance_loss(l, ids, coef, S, score)
    assert np.array_equal(counts.cpu().numpy(), rc)
    # the loss: a sum of p-weighted terms of |f - 1| and the constant 1, each within 2^-17 of its size, rounded once
    size = abs(coef) * (2 + float((rc / np.maximum(rc.sum(1, keepdims=True), 1)).max()) * l.shape[1]) if l.size else 0.0
    assert abs(loss.item() - rl) <= 2.0 ** -17 * size + 1e-37, (loss.item(), rl)
    g = grad.double().cpu().numpy()
    err = balance_bound(l, ids, coef, S, score, p, False)
    if t.dtype is torch.bfloat16:
        err = err + 0.5 * bf16_ulp(g)
    assert grad.dtype is t.dtype and not (np.abs(g - rg) > err).any(), np.abs(g - rg).max()
    return loss, counts, grad


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("S,L,E,k", [(1, 1, 1, 1), (1, 1, 8, 2), (1, 64, 192, 4), (3, 7, 5, 3), (4, 100, 64, 8), (1, 1000, 65, 6),
                                     (2, 301, 128, 4), (5, 33, 255, 8), (1, 500, 257, 2), (2, 50, 1024, 64), (1, 5000, 16, 1),
                                     (70, 3, 31, 2), (1, 20000, 33, 4)])
def test_parity(S, L, E, k, bf16, score):
    print(f"[balance] {S}x{L} E{E} k{k} {bf16} {score}", flush=True)
    _check(*_inputs(S, L, E, k, S + L + E, bf16), S, score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_padding_is_not_looked_at(score):
    """Tokens without a valid id: NaN and infinities in their logits reach nothing, their gradient is zero; one
    sequence has no token at all."""
    S, L, E, k = 3, 40, 24, 4
    t, l, ids = _inputs(S, L, E, k, 2, pad=0.0)
    ids[30:40], ids[40:80], ids[100:] = -1, E, -7
    gone = np.r_[30:80, 100:120]
    l[gone] = np.tile([np.nan, np.inf, -np.inf, 1e38], (gone.size, 6))
    t = torch.from_numpy(l).cuda()
    l0 = l.copy()
    l0[gone] = 0.0
    loss, counts, grad = _check(t, l0, ids, S, score)
    assert not grad[torch.from_numpy(gone).cuda()].any() and not counts[1].any()
    rl = oracle.balance_loss(l0, ids, COEF, S, score)[0]
    assert np.isfinite(rl) and np.isfinite(loss.item())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_barred_experts(score):
    """Logits of -infinity and of the lowest float: no part of the scores, no gradient; a row of nothing else."""
    S, L, E, k = 1, 60, 40, 3
    t, l, ids = _inputs(S, L, E, k, 4, pad=0.1)
    l[:, 7], l[:, 11] = -np.inf, np.finfo(np.float32).min
    l[5], l[6, :39] = -np.inf, -np.inf
    t = torch.from_numpy(l).cuda()
    _, _, grad = _check(t, l, ids, S, score)
    assert not grad[:, 7].any() and not grad[:, 11].any() and not grad[5].any()
    l[8] = np.finfo(np.float32).min  # all alike, however low: an even choice
    _check(torch.from_numpy(l).cuda(), l, ids, S, score)


@pytest.mark.parametrize("E,k", [(40, 3), (128, 4), (300, 5)])
def test_sigmoids_below_float32(E, k):
    """Logits whose sigmoids float32 does not hold still choose between experts; beside tokens of ordinary logits."""
    t, l, ids = _inputs(2, 50, E, k, E, pad=0.1)
    for row, shift in ((3, -60.0), (4, -100.0), (50, -200.0), (51, -1.0e4), (99, -3.0e38)):
        l[row] = l[row] + np.float32(shift)
    _check(torch.from_numpy(l).cuda(), l, ids, 2, "sigmoid")


def test_gradient_against_differences():
    S, L, E, k = 2, 6, 10, 2
    for score in ("softmax", "sigmoid"):
        t, l, ids = _inputs(S, L, E, k, 6, pad=0.2)
        grad = w8.moe_balance_loss(t, to_dev(ids), coef=1.0, sequences=S, score=score)[2].cpu().double().numpy()
        for at in [(0, 0), (3, 4), (5, 9), (7, 2), (11, 5)]:
            h = 1e-4
            up, dn = l.astype(np.float64), l.astype(np.float64)
            up[at] += h
            dn[at] -= h
            d = (oracle.balance_loss(up, ids, 1.0, S, score)[0] - oracle.balance_loss(dn, ids, 1.0, S, score)[0]) / (2 * h)
            # central differences: h^2 / 6 times the third derivative (below 10 here) and rounding 2^-52 / h; the kernel's own error
            assert abs(grad[at] - d) <= 2e-8 + 2e-12 + 2.0 ** -15 * 4, (score, at)


def test_counts_that_are_even():
    """A perfectly even choice: f = 1, so loss = coef and the gradient is zero, exactly."""
    E, k = 32, 4
    ids = np.stack([(np.arange(k) + k * t) % E for t in range(64)]).astype(np.int32)
    l = np.random.default_rng(0).standard_normal((64, E)).astype(np.float32)
    loss, _, grad = w8.moe_balance_loss(torch.from_numpy(l).cuda(), to_dev(ids), coef=0.5)
    assert loss.item() == 0.5 and not grad.any()


def test_same_bits_every_call_and_without_gradient():
    t, l, ids = _inputs(3, 1500, 96, 4, 9)
    d = to_dev(ids)
    first = w8.moe_balance_loss(t, d, coef=COEF, sequences=3)
    for _ in range(3):
        again = w8.moe_balance_loss(t, d, coef=COEF, sequences=3)
        assert all(torch.equal(a, b) for a, b in zip(first, again))
    loss, counts, none = w8.moe_balance_loss(t, d, coef=COEF, sequences=3, with_grad=False)
    assert none is None and torch.equal(loss, first[0]) and torch.equal(counts, first[1])


def test_rows_behind_stay():
    t, l, ids = _inputs(1, 37, 21, 3, 1)
    buf = torch.full((60, 21), 5.0, device="cuda")
    w8.moe_balance_loss(t, to_dev(ids), grad=buf[:37])
    assert torch.equal(buf[37:], torch.full((23, 21), 5.0, device="cuda"))


def test_no_tokens():
    loss, counts, grad = w8.moe_balance_loss(torch.empty((0, 9), device="cuda"), torch.empty((0, 2), dtype=torch.int32, device="cuda"))
    assert loss.item() == 0.0 and not counts.any() and grad.shape == (0, 9)


@pytest.mark.parametrize("T,H,E,k", [(2, 64, 12, 2), (50, 256, 192, 4), (300, 512, 64, 8)])
def test_with_the_router(T, H, E, k):
    """moe_router's logits, its choice and the loss of it; the choice does not change for asking the logits."""
    rng = np.random.default_rng(T)
    x = to_dev_bf16(synth.activations(rng, T, H))
    wr = to_dev_bf16(synth.f32_to_bf16_bits((rng.standard_normal((E, H)) / H ** 0.5).astype(np.float32)))
    logits = torch.empty((T, E), device="cuda")
    ids, tw = w8.moe_router(x, wr, k, logits=logits)
    ids2, tw2 = w8.moe_router(x, wr, k)
    ref = x.cpu().double() @ wr.cpu().double().T
    assert torch.equal(ids, ids2) and torch.equal(tw, tw2)
    # float64 sums of exact products, rounded once: half a step, and the order of the float64 sums
    assert ((logits.cpu().double() - ref).abs() <= 2.0 ** -24 * ref.abs() + 1e-12).all()
    _check(logits, logits.cpu().numpy(), ids.cpu().numpy(), 1, "softmax")


def test_graph_with_a_shared_workspace():
    """Two captured losses on one workspace, replayed in turns with eager work between."""
    a, b = _inputs(2, 300, 64, 4, 3), _inputs(1, 40, 200, 8, 4, bf16=True)
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    cases = []
    for (t, _, ids), S in ((a, 2), (b, 1)):
        d = to_dev(ids)
        want = w8.moe_balance_loss(t, d, coef=COEF, sequences=S)
        bufs = [torch.zeros_like(w) for w in want]
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            w8.moe_balance_loss(t, d, coef=COEF, sequences=S, loss=bufs[0], counts=bufs[1], grad=bufs[2], workspace=ws)
        cases.append((g, bufs, want, d))  # the graph reads d: it has to live
    for i in range(4):
        for g, bufs, want, _ in cases:
            for x in bufs:
                x.zero_()
            ws.fill_(0x5A)
            g.replay()
            torch.zeros(1 << 18, device="cuda").sum()
            torch.cuda.synchronize()
            assert all(torch.equal(x, w) for x, w in zip(bufs, want)), i


def test_refusals():
    t, _, ids = _inputs(1, 8, 16, 2, 0)
    d = to_dev(ids)
    with pytest.raises(TypeError, match="logits must be"):
        w8.moe_balance_loss(t.double(), d)
    with pytest.raises(ValueError, match="sequences"):
        w8.moe_balance_loss(t, d, sequences=3)
    with pytest.raises(ValueError, match="sequences"):
        w8.moe_balance_loss(t, d, sequences=0)
    with pytest.raises(ValueError, match="score"):
        w8.moe_balance_loss(t, d, score="relu")
    with pytest.raises(ValueError, match="topk_ids"):
        w8.moe_balance_loss(t, d[:5].contiguous())
    with pytest.raises(ValueError, match="contiguous"):
        w8.moe_balance_loss(t.T.contiguous().T, d)
    with pytest.raises(TypeError, match="grad"):
        w8.moe_balance_loss(t, d, grad=torch.empty((8, 16), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(w8.W8A8Error, match="unsupported"):
        w8.moe_balance_loss(torch.zeros((2, 1025), device="cuda"), torch.zeros((2, 1), dtype=torch.int32, device="cuda"))
    with pytest.raises(w8.W8A8Error, match="workspace"):
        w8.moe_balance_loss(t, d, sequences=2, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
