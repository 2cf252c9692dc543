"""Block-scaled FP8 and the balance loss where offsets pass 31 and 32 bits, and where calls overlap.

The last rows of a large call are compared, bit for bit, with a call on those rows alone that runs the same kernels: a
row's result depends on its own operands only.
"""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no GPU", allow_module_level=True)

import w8a8_fp8_linear_amd as w8  # noqa: E402


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(shape, g, scale=1.0):
    """BF16 normals made in pieces (the float32 ones of a large tensor need not fit beside it)."""
    out = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    flat = out.view(-1)
    for i in range(0, flat.numel(), 1 << 28):
        flat[i:i + (1 << 28)] = torch.randn(min(1 << 28, flat.numel() - i), device="cuda", generator=g) * scale
    return out


def _experts(E, H, I, g):
    return (*w8.quantize_weight_blocks(_normal((E, 2 * I, H), g, 0.02)), *w8.quantize_weight_blocks(_normal((E, H, I), g, 0.02)))


def test_rows_beyond_32_bits():
    M, K = (1 << 21) + 5, 2064  # 4.3e9 values
    x = _normal((M, K), _gen(1))
    q, s = w8.quantize_blocks(x)
    q2, s2 = w8.quantize_blocks(x[-70:].contiguous())
    assert torch.equal(q[-70:], q2) and torch.equal(s[:, -70:], s2)


def test_weights_beyond_32_bits():
    E, N, K = 1030, 2048, 2064
    w = _normal((E, N, K), _gen(2))
    q, s = w8.quantize_weight_blocks(w)
    q2, s2 = w8.quantize_weight_blocks(w[-1])
    assert torch.equal(q[-1], q2) and torch.equal(s[-1], s2)


def test_product_beyond_32_bits():
    M, N, K = (1 << 19) + 1000, 8192, 144  # 4.3e9 outputs
    g = _gen(3)
    q, s = w8.quantize_blocks(_normal((M, K), g))
    w = w8.quantize_weight_blocks(_normal((N, K), g, 0.05))
    y = w8.w8a8_block_gemm(q, s, *w)
    # the last rows, beginning at a multiple of every tile's rows, and enough of them for the largest tiles
    n = M - (M - 16384) // 256 * 256
    assert torch.equal(y[-n:], w8.w8a8_block_gemm(q[-n:].contiguous(), s[:, -n:].contiguous(), *w))


def test_experts_beyond_32_bits():
    T, H, I, E, k = 140000, 2048, 128, 16, 8  # 2.3e9 values of the routed copies, 4.6e9 bytes
    g = _gen(4)
    w = _experts(E, H, I, g)
    q, s = w8.quantize_blocks(_normal((T, H), g))
    ids = torch.rand(T, E, device="cuda", generator=g).topk(k, 1).indices.int().contiguous()
    tw = torch.rand(T, k, device="cuda", generator=g)
    out = w8.moe_w8a8_block_grouped(q, s, ids, tw, *w)
    n = 3000  # groups of 1500 rows on average: the same kernels
    part = w8.moe_w8a8_block_grouped(q[-n:].contiguous(), s[:, -n:].contiguous(), ids[-n:].contiguous(),
                                     tw[-n:].contiguous(), *w)
    assert torch.equal(out[-n:], part)
    assert torch.equal(out, w8.moe_w8a8_block_grouped(q, s, ids, tw, *w))


def test_balance_beyond_32_bits():
    L, E, k = 1 << 13, 256, 4
    S = 1025  # 2.15e9 logits, 8.6e9 bytes
    g = _gen(5)
    logits = torch.empty(S * L, E, device="cuda")
    for i in range(0, S * L, 1 << 20):
        logits[i:i + (1 << 20)] = torch.randn(min(1 << 20, S * L - i), E, device="cuda", generator=g)
    ids = torch.randint(0, E, (S * L, k), device="cuda", generator=g, dtype=torch.int32)
    loss, counts, grad = w8.moe_balance_loss(logits, ids, coef=float(S), sequences=S)
    one, c1, g1 = w8.moe_balance_loss(logits[-L:].contiguous(), ids[-L:].contiguous(), coef=1.0)
    assert torch.equal(counts[-1:], c1) and int(counts.sum()) == S * L * k
    # coef / S is 1 in both: the same arithmetic a token but for the order of the float32 sum over experts
    assert float((grad[-L:] - g1).abs().max()) <= 2.0 ** -20 * float(g1.abs().max())
    assert abs(loss.item() / S - 1.0) < 1e-2 and abs(one.item() - 1.0) < 1e-2  # an even choice


@pytest.mark.parametrize("T", [2, 12, 60, 400, 1500])
def test_two_streams_at_once(T):
    """Two passes that overlap on two streams, each with its own workspace, give what each gives alone."""
    H, I, E, k = 272, 256, 6, 2
    g = _gen(6 + T)
    w = _experts(E, H, I, g)
    sets = []
    for _ in range(2):
        q, s = w8.quantize_blocks(_normal((T, H), g))
        ids = torch.rand(T, E, device="cuda", generator=g).topk(k, 1).indices.int().contiguous()
        sets.append((q, s, ids, torch.rand(T, k, device="cuda", generator=g)))
    want = [w8.moe_w8a8_block_grouped(*a, *w) for a in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    spaces = [w8.moe_w8a8_block_workspace(T, H, I, E, k) for _ in sets]
    outs = [torch.empty_like(want[0]) for _ in sets]
    torch.cuda.synchronize()
    for _ in range(20):
        for st, a, ws, o in zip(streams, sets, spaces, outs):
            with torch.cuda.stream(st):
                w8.moe_w8a8_block_grouped(*a, *w, out=o, workspace=ws)
    torch.cuda.synchronize()
    for o, y in zip(outs, want):
        assert torch.equal(o, y)


@pytest.mark.parametrize("T,E", [(2, 6), (12, 6), (60, 6), (400, 6), (1500, 6), (300, 600), (40000, 6)])
def test_captured_passes(T, E):
    """Every path of the pass, and of the order of its copies, captured and replayed on a soiled workspace."""
    H, I, k = 144, 128, 2
    g = _gen(60 + T)
    w = _experts(E, H, I, g)
    q, s = w8.quantize_blocks(_normal((T, H), g))
    ids = torch.randint(-1, E, (T, k), device="cuda", generator=g, dtype=torch.int32)
    tw = torch.rand(T, k, device="cuda", generator=g)
    want, wq, wsc = w8.moe_w8a8_block_grouped(q, s, ids, tw, *w, quantize_output=True)
    ws = w8.moe_w8a8_block_workspace(T, H, I, E, k)
    out = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _, oq, osc = w8.moe_w8a8_block_grouped(q, s, ids, tw, *w, out=out, workspace=ws, quantize_output=True)
    for i in range(3):
        ws.fill_(0x7F + i)
        out.zero_()
        oq.zero_()
        graph.replay()
        torch.ones(1 << 18, device="cuda").sum()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(oq, wq) and torch.equal(osc, wsc), i


@pytest.mark.parametrize("E1,E2", [(2, 8), (7, 20), (100, 700)])
def test_one_expert_takes_all(E1, E2):
    """Every copy goes to one expert: the same bits whichever it is and however many others get nothing (sizes on
    which both calls run the same kernels; 700 experts take the order of three launches)."""
    T, H, I = 3000, 272, 256
    g = _gen(90 + E2)
    one = _experts(1, H, I, g)
    q, s = w8.quantize_blocks(_normal((T, H), g))
    tw = torch.rand(T, 1, device="cuda", generator=g)
    outs = []
    for E, e in ((E1, E1 - 1), (E2, 0), (E2, E2 - 1)):
        w = [torch.full((E, *t.shape[1:]), 0x7F if t.dtype is torch.uint8 else float("nan"), dtype=t.dtype, device="cuda") for t in one]
        for big, t in zip(w, one):
            big[e] = t[0]
        outs.append(w8.moe_w8a8_block_grouped(q, s, torch.full((T, 1), e, dtype=torch.int32, device="cuda"), tw, *w))
    assert bool(outs[0].isfinite().all()) and bool(outs[0].any())
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
