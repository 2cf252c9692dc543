"""The block-scaled oracle and the balance loss against independent statements of the same rules."""
import numpy as np
import pytest

import oracle
from oracle.quant import quantize_rows


@pytest.mark.parametrize("M,K", [(1, 16), (3, 128), (5, 144), (2, 400)])
def test_rows_are_the_row_quantiser_on_pieces(M, K):
    x = np.random.default_rng(K).standard_normal((M, K)).astype(np.float32) * np.exp2(np.arange(K) // 50).astype(np.float32)
    q, s = oracle.quantize_row_blocks(x)
    for b, k in enumerate(range(0, K, 128)):
        rq, rs, _ = quantize_rows(x[:, k:k + 128])
        assert np.array_equal(q[:, k:k + 128], rq) and np.array_equal(s[b], rs)
    v = oracle.row_values(q, s)
    assert (np.abs(v - x) <= np.abs(x) * 2.0 ** -4 + np.repeat(s.T, 128, 1)[:, :K] * 2.0 ** -10).all()


def test_weights_are_the_row_quantiser_on_flat_blocks():
    w = np.random.default_rng(1).standard_normal((200, 272)).astype(np.float32)
    q, s = oracle.quantize_weight_blocks(w)
    assert s.shape == (2, 3)
    for a in range(2):
        for b in range(3):
            piece = w[128 * a:128 * a + 128, 128 * b:128 * b + 128]
            rq, rs, _ = quantize_rows(piece.reshape(1, -1))
            assert s[a, b] == rs[0] and np.array_equal(q[128 * a:128 * a + 128, 128 * b:128 * b + 128].ravel(), rq[0])


def test_zero_blocks_have_scale_one():
    q, s = oracle.quantize_row_blocks(np.zeros((2, 130), np.float32))
    assert not q.any() and (s == 1).all()


def test_linear_by_hand():
    rng = np.random.default_rng(2)
    qx, sx = oracle.quantize_row_blocks(rng.standard_normal((3, 272)).astype(np.float32))
    qw, sw = oracle.quantize_weight_blocks(rng.standard_normal((144, 272)).astype(np.float32))
    y, mag = oracle.block_linear(qx, sx, qw, sw)
    m, n = 2, 140
    t = [float(sx[k // 128, m]) * float(sw[n // 128, k // 128]) * oracle.decode(qx[m, k]) * oracle.decode(qw[n, k]) for k in range(272)]
    assert abs(y[m, n] - sum(t)) <= 1e-12 and abs(mag[m, n] - sum(map(abs, t))) <= 1e-12


def test_expert_pass_of_one_expert_is_two_linears():
    rng = np.random.default_rng(3)
    qx, sx = oracle.quantize_row_blocks(rng.standard_normal((4, 144)).astype(np.float32))
    q13, s13 = oracle.quantize_weight_blocks(0.1 * rng.standard_normal((256, 144)).astype(np.float32))
    q2, s2 = oracle.quantize_weight_blocks(0.1 * rng.standard_normal((144, 128)).astype(np.float32))
    ids = np.array([[0, 0], [0, -1], [5, 0], [-1, 9]], np.int32)
    tw = rng.random((4, 2)).astype(np.float32)
    out, _ = oracle.moe_block_pass(qx, sx, ids, tw, q13[None], s13[None], q2[None], s2[None])
    h = oracle.swiglu_f32(oracle.block_linear(qx, sx, q13, s13)[0])
    y = oracle.block_linear(*oracle.quantize_row_blocks(h), q2, s2)[0]
    w = np.where(ids == 0, tw.astype(np.float64), 0).sum(1)
    assert np.allclose(out, y * w[:, None], rtol=1e-12, atol=1e-14) and not out[3].any()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_balance_gradient_is_the_differences(score):
    rng = np.random.default_rng(4)
    l, ids = rng.standard_normal((12, 7)), rng.integers(-1, 8, (12, 3)).astype(np.int32)
    ids[8] = -1
    loss, counts, grad, p = oracle.balance_loss(l, ids, 0.3, 3, score)
    assert counts.sum() == ((ids >= 0) & (ids < 7)).sum() and not grad[8].any()
    for at in np.ndindex(l.shape):
        up, dn = l.copy(), l.copy()
        up[at] += 1e-5
        dn[at] -= 1e-5
        d = (oracle.balance_loss(up, ids, 0.3, 3, score)[0] - oracle.balance_loss(dn, ids, 0.3, 3, score)[0]) / 2e-5
        assert abs(grad[at] - d) <= 1e-9


def test_balance_of_an_even_choice_and_of_one_expert():
    E, k = 8, 2
    even = np.stack([(np.arange(k) + k * t) % E for t in range(16)]).astype(np.int32)
    l = np.random.default_rng(5).standard_normal((16, E))
    loss, counts, grad, _ = oracle.balance_loss(l, even, 0.7)
    assert abs(loss - 0.7) < 1e-15 and (counts == 4).all() and np.abs(grad).max() < 1e-16
    one = np.zeros((16, 1), np.int32)
    l = np.full((16, E), -np.inf)
    l[:, 0] = 3.0
    loss, counts, grad, _ = oracle.balance_loss(l, one, 0.7)
    assert abs(loss - 0.7 * E) < 1e-14 and counts[0, 0] == 16 and not grad.any()
