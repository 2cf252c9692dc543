"""Rows of the block-scaled operators do not depend on each other, bit for bit, through every kernel: other rows' values
change, or the rows move, and a row keeps its result. And the balance loss's gradient against differences, relative to
its own size."""
import numpy as np
import pytest

import oracle
import synth
from block_util import quantized_stack, weights
from gpu_util import to_dev, to_dev_bf16

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no GPU", allow_module_level=True)

import w8a8_fp8_linear_amd as w8  # noqa: E402


def _rows(rng, M, K):
    return to_dev_bf16(synth.activations(rng, M, K, n_outlier=max(1, K // 100)))


# one kernel of w8a8_block_gemm a line: up to 4, 16 and 32 rows, K split over the waves (two tiles), 64 x 64 tiles of two stages
# and of one, 64 x 128, 128 x 256, 128 x 128
PRODUCTS = [(4, 96, 2064), (11, 96, 2064), (27, 208, 2064), (90, 272, 1040), (301, 1040, 400), (700, 2064, 272), (600, 4112, 272),
            (1100, 5008, 272), (8192, 2048, 272), (4100, 6144, 144)]


@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_product_rows_on_their_own(M, N, K):
    print(f"[block] rows on their own {M}x{N}x{K}", flush=True)
    rng = np.random.default_rng(M + N + K)
    x = _rows(rng, M, K)
    w = [to_dev(a) for a in oracle.quantize_weight_blocks(weights(rng, N, K))]
    q, s = w8.quantize_blocks(x)
    y = w8.w8a8_block_gemm(q, s, *w)
    keep = torch.from_numpy(np.sort(rng.choice(M, max(1, M // 3), replace=False))).cuda()
    q2, s2 = w8.quantize_blocks(_rows(rng, M, K) * 4)
    s2[:, ::5] = float("nan")
    q2[keep], s2[:, keep] = q[keep], s[:, keep]
    assert torch.equal(w8.w8a8_block_gemm(q2, s2, *w)[keep], y[keep])
    for by in (1, 37, M // 2):
        rolled = w8.w8a8_block_gemm(q.roll(by, 0), s.roll(by, 1).contiguous(), *w)
        assert torch.equal(rolled, y.roll(by, 0))


@pytest.mark.parametrize("M,N,K", [(1, 96, 2064), (4, 96, 2064), (7, 96, 2064), (15, 208, 1040)])
def test_fused_rows_on_their_own(M, N, K):
    """The layer's kernels that quantise inside the product."""
    rng = np.random.default_rng(M + N)
    x, other = _rows(rng, M, K), _rows(rng, M, K)
    w = [to_dev(a) for a in oracle.quantize_weight_blocks(weights(rng, N, K))]
    y = w8.w8a8_block_linear(x, *w)
    for m in range(M):
        z = other.clone()
        z[(m + 1) % M] = float("nan")
        z[m] = x[m]
        assert torch.equal(w8.w8a8_block_linear(z, *w)[m], y[m])
    assert torch.equal(w8.w8a8_block_linear(x.flip(0), *w), y.flip(0))


# one path a line: the sum in the down projection; groups of few rows by copy and by expert; tiles of 32, of 64 and of 128 rows
EXPERTS = [(3, 400, 512, 20, 4), (9, 400, 512, 40, 4), (40, 400, 256, 20, 4), (150, 400, 256, 20, 4), (900, 272, 256, 12, 3), (1500, 272, 256, 6, 2)]


@pytest.mark.parametrize("T,H,I,E,k", EXPERTS)
def test_experts_tokens_on_their_own(T, H, I, E, k):
    """Other tokens that share the experts get other rows (some NaN) and other weights, with the ids kept."""
    print(f"[block] tokens on their own T{T} H{H} I{I} E{E} k{k}", flush=True)
    rng = np.random.default_rng(T + H + I)
    x, other = _rows(rng, T, H), _rows(rng, T, H) * 4
    w = [to_dev(a) for m in ((E, 2 * I, H), (E, H, I)) for a in quantized_stack(weights(rng, *m))]
    ids, tw = (to_dev(a) for a in synth.routing(rng, T, E, k))
    q, s = w8.quantize_blocks(x)
    out, oq, osc = w8.moe_w8a8_block_grouped(q, s, ids, tw, *w, quantize_output=True)
    assert bool(out.isfinite().all()) and bool(out.any())
    keep = torch.from_numpy(np.sort(rng.choice(T, max(1, T // 3), replace=False))).cuda()
    q2, s2 = w8.quantize_blocks(other)
    s2[:, ::5] = float("nan")
    q2[keep], s2[:, keep] = q[keep], s[:, keep]
    tw2 = torch.rand_like(tw)
    tw2[keep] = tw[keep]
    o2, oq2, osc2 = w8.moe_w8a8_block_grouped(q2, s2, ids, tw2, *w, quantize_output=True)
    assert torch.equal(o2[keep], out[keep]) and torch.equal(oq2[keep], oq[keep]) and torch.equal(osc2[:, keep], osc[:, keep])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("S,L,E,k", [(2, 6, 10, 2), (1, 5, 130, 3), (3, 4, 300, 2)])
def test_balance_gradient_against_differences(S, L, E, k, score):
    """Central differences of the 64-bit loss: off by h^2 / 6 times the third derivative, which is below 100 times the
    gradient's size p_j (|g_j| + sum |g| p) (g = coef f / (S n)), and by 2^-52 loss / h. The kernel's own error is below 2^-15
    of that size (f - 1 in f's place makes it no larger than twice)."""
    rng = np.random.default_rng(S + E)
    l = (rng.standard_normal((S * L, E)) * 2).astype(np.float32)
    ids = np.argsort(rng.random((S * L, E)), axis=1)[:, :k].astype(np.int32)
    ids[1] = -1
    grad = w8.moe_balance_loss(torch.from_numpy(l).cuda(), to_dev(ids), coef=1.0, sequences=S, score=score)[2].cpu().double().numpy()
    _, counts, _, p = oracle.balance_loss(l, ids, 1.0, S, score)
    h = 1e-4
    for t in range(S * L):
        n = (ids[t // L * L:(t // L + 1) * L] >= 0).any(1).sum()
        g = E * counts[t // L] / (k * n) / (S * n)
        size = p[t] * (g + (1 / (S * n)) + (p[t] * g).sum())
        for j in range(0, E, 1 + E // 12):
            up, dn = l.astype(np.float64), l.astype(np.float64)
            up[t, j] += h
            dn[t, j] -= h
            lu, ld = (oracle.balance_loss(a, ids, 1.0, S, score)[0] for a in (up, dn))
            d = (lu - ld) / (2 * h)
            assert abs(grad[t, j] - d) <= (2.0 ** -14 + 100 * h * h / 6) * size[j] + 2.0 ** -50 * lu / h, (t, j)
