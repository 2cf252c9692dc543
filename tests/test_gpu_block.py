"""GPU parity of FP8 with a scale per block of 128.

* quantize_blocks / quantize_weight_blocks are bit-exact against the oracle: ragged sizes, one value to many
  blocks, zero, subnormal and largest blocks, every finite BF16 value.
* w8a8_block_gemm: every output inside the E4M3 matrix core's bound, through every kernel, at ragged sizes;
  w8a8_block_linear gives quantize_blocks + w8a8_block_gemm's bits.
* moe_w8a8_block_grouped: every output inside the bound carried through both projections and h's codes; dropped
  ids, empty experts, equal ids; the fused quantisation of the output; a stack of two passes.
* Rows behind the output stay as they were; captured graphs, another stream; refused arguments.
"""
import numpy as np
import pytest

import oracle
import synth
from block_util import moe_ref, product_err, quantized_stack, violations, weights
from gpu_util import bf16_bits, to_dev, to_dev_bf16

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no GPU", allow_module_level=True)

import w8a8_fp8_linear_amd as w8  # noqa: E402


def _bf16(x):
    return to_dev_bf16(synth.f32_to_bf16_bits(np.asarray(x, np.float32)))


def _rows_match(x_bits):
    q, s = w8.quantize_blocks(to_dev_bf16(x_bits))
    torch.cuda.synchronize()
    rq, rs = oracle.quantize_row_blocks(synth.bf16_bits_to_f32(x_bits))
    assert np.array_equal(s.cpu().numpy(), rs) and np.array_equal(q.cpu().numpy(), rq)


@pytest.mark.parametrize("M,K", [(1, 16), (3, 128), (5, 144), (16, 512), (17, 528), (130, 1040), (33, 8208), (1, 65552)])
def test_quantize_rows_bit_exact(M, K):
    print(f"[block] rows {M}x{K}", flush=True)
    rng = np.random.default_rng(M + K)
    x = rng.standard_normal((M, K), dtype=np.float32) * np.exp2(rng.integers(-10, 10, (M, K // 16)).repeat(16, 1)).astype(np.float32)
    _rows_match(synth.f32_to_bf16_bits(x))


def test_quantize_every_bf16():
    """Every finite BF16 value in blocks of neighbours, subnormals and the largest among them, then against each binade's top."""
    bits = np.arange(0x7F80, dtype=np.uint32).astype(np.uint16)
    _rows_match(np.concatenate([bits, bits | 0x8000]).reshape(16, -1))
    rng = np.random.default_rng(3)
    x = rng.permutation(bits).reshape(-1, 64)
    _rows_match(np.concatenate([x, np.repeat(x[:, :1], 64, 1)], 1))


def test_quantize_zero_blocks():
    x = np.zeros((4, 400), np.float32)
    x[1, 130], x[2, 399], x[3] = -2.0 ** -130, 3.0, -0.0
    _rows_match(synth.f32_to_bf16_bits(x))


@pytest.mark.parametrize("E,N,K", [(0, 1, 16), (0, 128, 128), (0, 130, 272), (3, 16, 1040), (2, 400, 144), (5, 257, 512)])
def test_quantize_weights_bit_exact(E, N, K):
    print(f"[block] weights {E}x{N}x{K}", flush=True)
    rng = np.random.default_rng(N + K)
    w = weights(rng, max(E, 1), N, K)
    w[0, :, -16:] = 0.0
    q, s = w8.quantize_weight_blocks(_bf16(w if E else w[0]))
    torch.cuda.synchronize()
    rq, rs = quantized_stack(w)
    assert np.array_equal(s.cpu().numpy(), rs if E else rs[0]) and np.array_equal(q.cpu().numpy(), rq if E else rq[0])


SHAPES = [(1, 16, 16), (1, 8192, 256), (2, 48, 144), (5, 144, 1040), (8, 528, 2064), (16, 208, 528), (17, 1040, 2080), (31, 96, 4112),
          (8, 64, 4112), (9, 48, 2064), (12, 96, 4112), (32, 64, 128), (33, 16, 32), (64, 208, 96), (65, 192, 160), (257, 400, 1056), (301, 1040, 1056),
          (513, 272, 528), (600, 1040, 528), (1024, 2064, 400), (700, 6160, 272), (2049, 2320, 272), (3000, 5008, 272), (4100, 4112, 144)]


def _operands(M, N, K, seed):
    rng = np.random.default_rng(seed)
    x = synth.activations(rng, M, K, n_outlier=max(1, K // 100))
    qw, sw = oracle.quantize_weight_blocks(weights(rng, N, K))
    return x, qw, sw


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product_parity(M, N, K):
    print(f"[block] product {M}x{N}x{K}", flush=True)
    x, qw, sw = _operands(M, N, K, M + N + K)
    dw, ds = to_dev(qw), to_dev(sw)
    q, s = w8.quantize_blocks(to_dev_bf16(x))
    y = w8.w8a8_block_gemm(q, s, dw, ds)
    lin = w8.w8a8_block_linear(to_dev_bf16(x), dw, ds)
    torch.cuda.synchronize()
    got = bf16_bits(y)
    assert np.array_equal(got, bf16_bits(lin))
    rows = np.arange(M) if M <= 600 else np.unique(np.concatenate([np.arange(0, M, 37), [M - 1]]))
    rq, rs = oracle.quantize_row_blocks(synth.bf16_bits_to_f32(x[rows]))
    y64, mag = oracle.block_linear(rq, rs, qw, sw)
    assert violations(got[rows], y64, product_err(K, mag)) == 0
    if M > rows.size:  # the rows between: the same bits as alone, in a call of their own
        some = np.arange(5, M, 211)[:32]
        alone = w8.w8a8_block_gemm(q[some].contiguous(), s[:, some].contiguous(), dw, ds)
        diff = np.abs(oracle.bf16_bits_to_f64(bf16_bits(alone)) - oracle.bf16_bits_to_f64(got[some]))
        y64, mag = oracle.block_linear(*oracle.quantize_row_blocks(synth.bf16_bits_to_f32(x[some])), qw, sw)
        assert violations(got[some], y64, product_err(K, mag)) == 0 and np.isfinite(diff).all()


@pytest.mark.parametrize("M,N,K", [(3, 272, 400), (40, 272, 400), (300, 272, 400), (2100, 3088, 400)])
def test_scales_belong_to_their_block(M, N, K):
    """Codes of 1 everywhere, every scale its own power of two: each output is an exact sum that names its blocks."""
    print(f"[block] own scales {M}x{N}x{K}", flush=True)
    kb, nb = -(-K // 128), -(-N // 128)
    q = torch.full((M, K), 0x38, dtype=torch.uint8, device="cuda")
    w = torch.full((N, K), 0x38, dtype=torch.uint8, device="cuda")
    sa = torch.exp2(torch.arange(kb, device="cuda").float()[:, None] * 3 - torch.arange(M, device="cuda").float()[None] % 7)
    sw = torch.exp2(torch.arange(nb, device="cuda").float()[:, None] - torch.arange(kb, device="cuda").float()[None] * 2)
    y = w8.w8a8_block_gemm(q, sa.contiguous(), w, sw.contiguous())
    lens = torch.tensor([min(128, K - 128 * b) for b in range(kb)], device="cuda", dtype=torch.float64)
    ref = torch.einsum("bm,nb,b->mn", sa.double(), sw.double(), lens).repeat_interleave(128, 1)[:, :N]
    assert torch.equal(y, ref.bfloat16())


def test_one_rows_scale_stays_in_its_row():
    """An infinite or NaN scale of a row or of a weight block reaches its own outputs and no other bit."""
    M, N, K = 70, 400, 272
    x, qw, sw = _operands(M, N, K, 5)
    q, s = w8.quantize_blocks(to_dev_bf16(x))
    dw, ds = to_dev(qw), to_dev(sw)
    want = w8.w8a8_block_gemm(q, s, dw, ds)
    s2, ds2 = s.clone(), ds.clone()
    s2[2, 69], ds2[3, 0] = float("nan"), float("inf")
    y = w8.w8a8_block_gemm(q, s2, dw, ds2)
    assert torch.isnan(y[69].float()).all() and not torch.isfinite(y[:, 384:].float()).any()
    assert torch.equal(y[:69, :384], want[:69, :384])


@pytest.mark.parametrize("M", [9, 100, 1000])
def test_rows_behind_stay(M):
    N, K = 208, 272
    x, qw, sw = _operands(M, N, K, M)
    buf = torch.full((M + 40, N), 7.0, dtype=torch.bfloat16, device="cuda")
    w8.w8a8_block_linear(to_dev_bf16(x), to_dev(qw), to_dev(sw), out=buf[:M])
    assert torch.equal(buf[M:], torch.full_like(buf[M:], 7.0))
    qb = torch.full((M + 40, K), 9, dtype=torch.uint8, device="cuda")
    w8.quantize_blocks(to_dev_bf16(x), q=qb[:M])
    assert int((qb[M:] != 9).sum()) == 0


def _moe(T, H, I, E, k, seed, ids=None):
    rng = np.random.default_rng(seed)
    x = synth.activations(rng, T, H, n_outlier=max(1, H // 100))
    q13, s13 = quantized_stack(weights(rng, E, 2 * I, H))
    q2, s2 = quantized_stack(weights(rng, E, H, I))
    if ids is None:
        ids, tw = synth.routing(rng, T, E, k)
    else:
        tw = rng.random(ids.shape, dtype=np.float32)
    qx, sx = oracle.quantize_row_blocks(synth.bf16_bits_to_f32(x))
    return dict(x=x, qx=qx, sx=sx, ids=ids, tw=tw, w=(q13, s13, q2, s2))


def _moe_run(d, **kw):
    return w8.moe_w8a8_block_grouped(to_dev(d["qx"]), to_dev(d["sx"]), to_dev(d["ids"]), to_dev(d["tw"]),
                                     *(to_dev(a) for a in d["w"]), **kw)


MOE_SHAPES = [(1, 16, 128, 1, 1), (1, 1024, 512, 128, 4), (3, 144, 256, 5, 2), (17, 272, 384, 9, 4), (37, 1024, 512, 192, 4),
              (64, 400, 128, 3, 3), (200, 528, 256, 6, 2), (301, 1040, 384, 40, 8), (900, 272, 256, 4, 3), (1500, 528, 128, 2, 2),
              (4, 400, 512, 16, 4), (16, 272, 1024, 20, 1), (9, 144, 128, 3, 64), (130, 2064, 128, 8, 4), (70, 144, 1152, 40, 7),
              (300, 144, 128, 600, 2), (33000, 128, 128, 16, 2)]


@pytest.mark.parametrize("T,H,I,E,k", MOE_SHAPES)
def test_experts_parity(T, H, I, E, k):
    print(f"[block] experts T{T} H{H} I{I} E{E} k{k}", flush=True)
    d = _moe(T, H, I, E, k, T + H + I)
    out = _moe_run(d)
    torch.cuda.synchronize()
    tokens = np.arange(T) if T <= 64 else np.unique(np.r_[np.arange(0, T, 1 + T // 48), T - 1])
    ref, err = moe_ref(d["qx"], d["sx"], d["ids"], d["tw"], *d["w"], tokens=tokens)
    got = bf16_bits(out)
    assert violations(got[tokens], ref, err) == 0
    # a token's result does not depend on who else is in the batch where the same kernels run
    assert np.array_equal(got, bf16_bits(_moe_run(d)))


@pytest.mark.parametrize("T", [6, 150])
def test_experts_dropped_and_equal_ids(T):
    E, k = 7, 3
    rng = np.random.default_rng(T)
    ids = rng.integers(-2, E + 2, (T, k)).astype(np.int32)
    ids[0], ids[1], ids[2] = -1, [4, 4, 4], [E, 2, -5]
    d = _moe(T, 272, 256, E, k, T, ids=ids)
    got = bf16_bits(_moe_run(d))
    ref, err = moe_ref(d["qx"], d["sx"], ids, d["tw"], *d["w"])
    assert violations(got, ref, err) == 0 and not got[0].any()


def test_experts_nothing_routed():
    d = _moe(20, 144, 128, 4, 2, 1, ids=np.full((20, 2), -1, np.int32))
    assert not bf16_bits(_moe_run(d)).any()


@pytest.mark.parametrize("T,H", [(5, 144), (10, 144), (70, 512), (300, 1040)])
def test_experts_quantised_output(T, H):
    d = _moe(T, H, 256, 6, 3, T)
    out, q, s = _moe_run(d, quantize_output=True)
    q2, s2 = w8.quantize_blocks(out)
    assert torch.equal(q, q2) and torch.equal(s, s2)
    assert torch.equal(out, _moe_run(d))


@pytest.mark.parametrize("T", [2, 7, 40, 200, 1300])
def test_experts_scaled_by_powers_of_two(T):
    """Scales and router weights times powers of two move the output by their product and not a bit besides, up to
    where the bound on a copy's values is beyond float32 though the values are not; negated scales negate."""
    d = _moe(T, 272, 256, 6, 2, 31 + T)
    base = _moe_run(d)
    q13, s13, q2, s2 = d["w"]
    for a, b in ((100, 0), (60, 45), (-40, 20), (-60, -20), (20, -90)):
        e = dict(d, w=(q13, s13, q2, np.ldexp(s2, a).astype(np.float32)), tw=np.ldexp(d["tw"], b).astype(np.float32))
        want = torch.ldexp(base.double(), torch.tensor(a + b)).float().bfloat16()
        assert bool(want.isfinite().all())
        assert torch.equal(_moe_run(e), want)
    assert torch.equal(_moe_run(dict(d, w=(q13, s13, q2, -s2))), -base)


@pytest.mark.parametrize("T", [3, 260])
def test_two_passes(T):
    """moe_block_ffn is the chain of its calls; each pass is checked on the codes that the one before it left."""
    d = _moe(T, 400, 256, 8, 2, T)
    rng = np.random.default_rng(9)
    ids2, tw2 = synth.routing(rng, T, 8, 2)
    routes = [(to_dev(d["ids"]), to_dev(d["tw"])), (to_dev(ids2), to_dev(tw2))]
    dw = [to_dev(a) for a in d["w"]]
    o1, o2 = w8.moe_block_ffn(to_dev_bf16(d["x"]), routes, *dw)
    q, s = w8.quantize_blocks(o1)
    assert torch.equal(o1, _moe_run(d))
    assert torch.equal(o2, w8.moe_w8a8_block_grouped(q, s, *routes[1], *dw))
    ref, err = moe_ref(q.cpu().numpy(), s.cpu().numpy(), ids2, tw2, *d["w"], tokens=np.arange(min(T, 40)))
    assert violations(bf16_bits(o2)[:40], ref, err) == 0


def test_experts_nan_stays_with_its_expert():
    """An expert whose scales are NaN or infinite reaches the tokens that picked it and no other bit."""
    for T in (4, 200):
        d = _moe(T, 272, 256, 6, 2, 77 + T)
        want = bf16_bits(_moe_run(d))
        q13, s13, q2, s2 = d["w"]
        s13, s2 = s13.copy(), s2.copy()
        s13[2], s2[4] = np.nan, np.inf
        d["w"] = (q13, s13, q2, s2)
        hit = np.isin(d["ids"], (2, 4)).any(1)
        got = bf16_bits(_moe_run(d))
        assert np.array_equal(got[~hit], want[~hit])
        assert not np.isfinite(oracle.bf16_bits_to_f64(got[hit])).any()


def test_graphs_share_nothing_but_a_workspace():
    """Layers and a two-pass expert stage captured, replayed in turns on one workspace, with eager work between."""
    x, qw, sw = _operands(300, 528, 400, 8)
    d = _moe(150, 400, 256, 8, 2, 8)
    dx, dw, ds = to_dev_bf16(x), to_dev(qw), to_dev(sw)
    args = [to_dev(d["qx"]), to_dev(d["sx"]), to_dev(d["ids"]), to_dev(d["tw"]), *(to_dev(a) for a in d["w"])]
    ws = torch.empty(max(w8.moe_w8a8_block_workspace(150, 400, 256, 8, 2).numel(),
                         int(w8.lib().w8a8_block_linear_workspace_bytes(300, 400))), dtype=torch.uint8, device="cuda")
    want = [bf16_bits(w8.w8a8_block_linear(dx, dw, ds)), bf16_bits(w8.w8a8_block_linear(dx[:7], dw, ds)),
            bf16_bits(w8.moe_w8a8_block_grouped(*args))]
    runs = [lambda: w8.w8a8_block_linear(dx, dw, ds, out=outs[0], workspace=ws), lambda: w8.w8a8_block_linear(dx[:7], dw, ds, out=outs[1]),
            lambda: w8.moe_w8a8_block_grouped(*args, out=outs[2], workspace=ws)]
    outs = [torch.empty(w.shape, dtype=torch.bfloat16, device="cuda") for w in want]
    graphs = []
    for run in runs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run()
        graphs.append(g)
    for i in range(4):
        for g, o, w in zip(graphs, outs, want):
            o.zero_()
            ws.fill_(0xA5 + i)
            g.replay()
            torch.zeros(1 << 18, device="cuda").sum()
            torch.cuda.synchronize()
            assert np.array_equal(bf16_bits(o), w), i


def test_other_stream():
    x, qw, sw = _operands(90, 272, 400, 4)
    dx, dw, ds = to_dev_bf16(x), to_dev(qw), to_dev(sw)
    want = w8.w8a8_block_linear(dx, dw, ds)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        y = w8.w8a8_block_linear(dx, dw, ds)
    st.synchronize()
    assert torch.equal(y, want)


def test_empty():
    qw, sw = torch.zeros((16, 32), dtype=torch.uint8, device="cuda"), torch.ones((1, 1), device="cuda")
    assert w8.w8a8_block_linear(torch.empty((0, 32), dtype=torch.bfloat16, device="cuda"), qw, sw).shape == (0, 16)
    q, s = w8.quantize_blocks(torch.empty((0, 208), dtype=torch.bfloat16, device="cuda"))
    assert q.shape == (0, 208) and s.shape == (2, 0)
    assert w8.w8a8_block_gemm(q[:, :32].contiguous(), s[:1], qw, sw).shape == (0, 16)


def test_refusals():
    x = torch.zeros((4, 256), dtype=torch.bfloat16, device="cuda")
    w, s = torch.zeros((32, 256), dtype=torch.uint8, device="cuda"), torch.ones((1, 2), device="cuda")
    w8.w8a8_block_linear(x, w, s)
    with pytest.raises(ValueError, match="w_scale"):
        w8.w8a8_block_linear(x, w, torch.ones((32,), device="cuda"))
    with pytest.raises(TypeError, match="x must be"):
        w8.w8a8_block_linear(x.float(), w, s)
    with pytest.raises(ValueError, match="contiguous"):
        w8.w8a8_block_linear(x.T.contiguous().T, w, s)
    with pytest.raises(ValueError, match="a_scale"):
        w8.w8a8_block_gemm(w[:4], torch.ones((4, 2), device="cuda"), w, s)
    with pytest.raises(ValueError, match="on a GPU"):
        w8.quantize_blocks(torch.zeros((4, 256), dtype=torch.bfloat16))
    with pytest.raises(w8.W8A8Error, match="unsupported"):
        w8.quantize_blocks(torch.zeros((4, 24), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(w8.W8A8Error, match="aligned"):
        w8.quantize_blocks(torch.zeros(8 + 4 * 32, dtype=torch.bfloat16, device="cuda")[4:132].view(4, 32))
    big = torch.zeros((40, 256), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(w8.W8A8Error, match="workspace"):
        w8.w8a8_block_linear(big, w, s, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
