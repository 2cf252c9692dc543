"""GPU parity of NVFP4 quantisation and of the products with 4-bit weights.

* nvfp4_quantize is bit-exact against the oracle (codes, block scales, group
  scales) on ragged, multi-group and multi-chunk shapes, on ties, on all-zero
  and tiny blocks, with given group scales; nvfp4_dequantize is bit-exact.
* nvfp4_gemm / mxfp4_gemm: every element inside the BF16 matrix-core bound
  (gpu_util.BF16_MFMA_ERR), through both kernels, at ragged sizes; every code
  against every kind of block scale in single products, exactly.
* Rows beyond the output stay as they were; refused arguments.
"""
import numpy as np
import pytest

import oracle
import synth
from few_util import random_codes
from gpu_util import BF16_MFMA_ERR, U32, bf16_bits, bf16_ulp, to_dev, to_dev_bf16

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no GPU", allow_module_level=True)

import w8a8_fp8_linear_amd as w8  # noqa: E402


def _quant_matches(x_bits, gscale=None):
    G, R, K = x_bits.shape
    g_dev = to_dev(np.asarray(gscale, np.float32)) if gscale is not None else None
    q, s, g = w8.nvfp4_quantize(to_dev_bf16(x_bits), gscale=g_dev)
    y = w8.nvfp4_dequantize(q, s, g)
    torch.cuda.synchronize()
    x32 = synth.bf16_bits_to_f32(x_bits)
    for i in range(G):
        rq, rs, rg = oracle.nvfp4_quantize(x32[i], g=None if gscale is None else gscale[i])
        assert g[i].item() == rg, (i, g[i].item(), rg)
        assert np.array_equal(s[i].cpu().numpy(), rs), i
        assert np.array_equal(q[i].cpu().numpy(), rq), i
        ref = oracle.round_to_bf16_bits(oracle.nvfp4_dequant_f32(rq, rs, rg).astype(np.float64))
        assert np.array_equal(bf16_bits(y[i]), ref), i


@pytest.mark.parametrize("G,R,K", [(1, 1, 16), (1, 3, 48), (5, 7, 32), (3, 64, 1040), (2, 33, 4096), (1, 1, 65552),
                                   (9, 130, 272), (2, 2050, 4112), (130, 8, 16400)])
def test_quantize_bit_exact(G, R, K):
    print(f"[nvfp4] {G}x{R}x{K}", flush=True)
    rng = np.random.default_rng(G * R + K)
    x = rng.standard_normal((G, R, K), dtype=np.float32) * np.exp2(rng.integers(-8, 8, (G, R, 1))).astype(np.float32)
    x[:, :, :5] *= np.float32(50)
    _quant_matches(synth.f32_to_bf16_bits(x))


def test_quantize_every_bf16_in_a_group():
    """Every finite BF16 value, in ascending blocks: all ratios of a value to its block's maximum that a block of
    neighbours has, subnormals and the largest values among them."""
    bits = np.arange(0x7F80, dtype=np.uint32).astype(np.uint16)
    x = np.concatenate([bits, bits | 0x8000]).reshape(1, 16, -1)
    _quant_matches(x)


def test_quantize_ties():
    """A maximum of 6 * 2^j with g = 2^-9 or so gives d a power of two: multiples of 1/8 hit every midpoint."""
    v = np.arange(-48, 49, dtype=np.float32) / 8
    x = np.zeros((1, 8, 112), np.float32)
    for r in range(8):
        x[0, r, :97] = v * np.exp2(r - 4)
        x[0, r, 15::16] = 6 * np.exp2(r - 4)
    _quant_matches(synth.f32_to_bf16_bits(x), gscale=[np.float32(2.0 ** -6)])


def test_quantize_zero_and_tiny():
    x = np.zeros((4, 2, 64), np.float32)
    x[1, 0, 3] = -2.0 ** -120
    x[2, 1, 5], x[2, 0, :16] = 1.0, 2.0 ** -30
    x[3] = -0.0
    _quant_matches(synth.f32_to_bf16_bits(x))


@pytest.mark.parametrize("g", [2.0 ** -96, 1e-3, 1.0, 3.7e4])
def test_quantize_given_scale(g):
    rng = np.random.default_rng(8)
    x = synth.f32_to_bf16_bits(rng.standard_normal((2, 5, 160), dtype=np.float32))
    _quant_matches(x, gscale=[np.float32(g), np.float32(g / 3)])


def test_quantize_two_dims_and_buffers():
    x = to_dev_bf16(synth.f32_to_bf16_bits(np.random.default_rng(9).standard_normal((40, 64), dtype=np.float32)))
    q, s, g = w8.nvfp4_quantize(x)
    q3, s3, g3 = w8.nvfp4_quantize(x[None])
    assert g.shape == (1,) and torch.equal(q, q3[0]) and torch.equal(s, s3[0]) and torch.equal(g, g3)
    q2, s2 = torch.zeros_like(q), torch.zeros_like(s)
    r = w8.nvfp4_quantize(x, gscale=g, q=q2, scale=s2)
    assert r[0] is q2 and torch.equal(q2, q) and torch.equal(s2, s)


def _gemm(fmt, x_bits, w):
    d = [to_dev(a) for a in w]
    y = (w8.nvfp4_gemm if fmt == "nvfp4" else w8.mxfp4_gemm)(to_dev_bf16(x_bits), *d)
    torch.cuda.synchronize()
    return bf16_bits(y)


def _bound_ok(fmt, x_bits, w, got):
    x = oracle.bf16_bits_to_f64(x_bits)
    g = w[2].reshape(-1)[0] if fmt == "nvfp4" else None
    wv = oracle.nvfp4_scaled(w[0], w[1]) * float(g) if fmt == "nvfp4" else oracle.mx_dequant(w[0], w[1])
    y64 = x @ wv.T
    K = x.shape[1]
    y = oracle.bf16_bits_to_f64(got)
    # as gpu_util.w8a16_report: exact products, 2^-20 for the MFMA's own sum, one float32 rounding per instruction,
    # and a few for the parts of K and the scale
    err = (BF16_MFMA_ERR + (K / 32 + 5) * U32) * 1.01 * (np.abs(x) @ np.abs(wv).T)
    return int((np.abs(y - y64) > err + 0.5 * bf16_ulp(y) + 1e-37).sum())


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("M,N,K", [(1, 16, 32), (2, 48, 96), (16, 208, 544), (17, 1040, 2080), (32, 64, 64),
                                   (33, 16, 32), (64, 208, 96), (65, 192, 160), (257, 400, 1056), (300, 1040, 544)])
def test_gemm_parity(fmt, M, N, K):
    print(f"[{fmt}_gemm] {M}x{N}x{K}", flush=True)
    rng = np.random.default_rng(M + N + K)
    x = synth.activations(rng, M, K, n_outlier=2)
    w, _ = random_codes(rng, fmt, N, K)
    w = (w[0][0], w[1][0]) + tuple(w[2:])
    assert _bound_ok(fmt, x, w, _gemm(fmt, x, w)) == 0


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("M,N,K", [(2051, 3280, 96), (2050, 3088, 1056), (1800, 4112, 2112), (2048, 3264, 32),
                                   (500, 1552, 1120), (900, 2000, 1504), (257, 4096, 32), (1030, 2032, 1248), (4100, 2064, 1120),
                                   (2050, 6160, 96)])
def test_gemm_parity_many_tiles(fmt, M, N, K):
    """Sizes of the tiled kernel: ragged edges, one step, scales that begin inside a dword and run over chunks."""
    print(f"[{fmt}_gemm] {M}x{N}x{K}", flush=True)
    rng = np.random.default_rng(M + N + K)
    x = synth.activations(rng, M, K, n_outlier=2)
    q = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
    w = (q, rng.integers(120, 130, (N, K // 32), dtype=np.uint8)) if fmt == "mxfp4" else \
        (q, rng.integers(0, 0x70, (N, K // 16), dtype=np.uint8), np.float32([0.01]))
    assert _bound_ok(fmt, x, w, _gemm(fmt, x, w)) == 0


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("M", [3, 40])
def test_gemm_every_code_and_scale(fmt, M):
    """A one-hot activation row reads one weight: every code, under every block scale (E8M0 2^-126 .. 2^124, all
    finite E4M3 bytes, a zero scale among them), is exact before the last rounding."""
    K, N = 128, 256
    codes = np.tile(np.arange(256, dtype=np.uint8), (N, 1))[:, :K // 2].copy()
    codes[1::2] = codes[1::2, ::-1]
    if fmt == "mxfp4":
        e = np.clip(np.arange(N), 1, 251).astype(np.uint8)
        w = (codes, np.repeat(e[:, None], K // 32, 1))
        val = oracle.mx_dequant(*w)
    else:
        s = oracle.finite_codes()
        s = np.resize(s, N).astype(np.uint8)
        w = (codes, np.repeat(s[:, None], K // 16, 1), np.float32([1.0]))
        val = oracle.nvfp4_scaled(w[0], w[1])
    for k0 in range(0, K, M):
        x = np.zeros((M, K), np.float32)
        for m in range(min(M, K - k0)):
            x[m, k0 + m] = 1.0
        got = _gemm(fmt, synth.f32_to_bf16_bits(x), w)
        ref = np.zeros((M, N))
        n = min(M, K - k0)
        ref[:n] = val[:, k0:k0 + n].T
        assert np.array_equal(oracle.bf16_bits_to_f64(got), oracle.bf16_bits_to_f64(oracle.round_to_bf16_bits(ref))), k0


def test_gemm_gscale_from_a_vector_and_no_rows():
    rng = np.random.default_rng(11)
    x = synth.activations(rng, 5, 64)
    w, _ = random_codes(rng, "nvfp4", 3, 32, 64)
    dev = [to_dev(a) for a in w]
    for e in range(3):
        got = w8.nvfp4_gemm(to_dev_bf16(x), dev[0][e], dev[1][e], dev[2][e:e + 1])
        assert _bound_ok("nvfp4", x, (w[0][e], w[1][e], w[2][e:e + 1]), bf16_bits(got)) == 0
    assert w8.nvfp4_gemm(torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"), dev[0][0], dev[1][0], dev[2][:1]).shape == (0, 32)


@pytest.mark.parametrize("M", [7, 37])
def test_gemm_leaves_other_rows(M):
    rng = np.random.default_rng(12)
    x = synth.activations(rng, M, 96)
    w, _ = random_codes(rng, "mxfp4", 48, 96)
    buf = torch.full((M + 8, 48), 7.0, dtype=torch.bfloat16, device="cuda")
    w8.mxfp4_gemm(to_dev_bf16(x), to_dev(w[0][0]), to_dev(w[1][0]), out=buf[:M])
    torch.cuda.synchronize()
    assert torch.all(buf[M:] == 7.0) and _bound_ok("mxfp4", x, (w[0][0], w[1][0]), bf16_bits(buf[:M])) == 0


def test_quantised_weights_through_the_product():
    """quantise -> product, as a user converts a checkpoint and runs it: against the product with the values read back."""
    rng = np.random.default_rng(13)
    wb = synth.weights(rng, (96, 288))
    x = synth.activations(rng, 9, 288, n_outlier=2)
    q, s, g = w8.nvfp4_quantize(to_dev_bf16(wb))
    y = bf16_bits(w8.nvfp4_gemm(to_dev_bf16(x), q, s, g))
    assert _bound_ok("nvfp4", x, tuple(t.cpu().numpy() for t in (q, s, g)), y) == 0


def test_refusals():
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    q = torch.zeros((32, 32), dtype=torch.uint8, device="cuda")
    s16, s32 = (torch.zeros((32, n), dtype=torch.uint8, device="cuda") for n in (4, 2))
    g = torch.ones(1, device="cuda")
    with pytest.raises(ValueError):
        w8.nvfp4_gemm(x, q, s32, g)
    with pytest.raises(ValueError):
        w8.mxfp4_gemm(x, q, s16)
    with pytest.raises(TypeError):
        w8.mxfp4_gemm(x.float(), q, s32)
    with pytest.raises(ValueError):
        w8.nvfp4_gemm(x, q, s16, g.cpu())
    with pytest.raises(ValueError):
        w8.nvfp4_gemm(x, q, s16, torch.ones(2, device="cuda"))
    with pytest.raises(ValueError):
        w8.nvfp4_gemm(x.t(), q, s16, g)
    with pytest.raises(ValueError):
        w8.nvfp4_quantize(torch.zeros((4, 24), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(w8.W8A8Error) as e:   # 24 output rows
        w8.mxfp4_gemm(x, q[:24], s32[:24])
    assert e.value.status == 4
    with pytest.raises(w8.W8A8Error) as e:   # x starts 8 bytes into a row
        buf = torch.zeros(4 * 64 + 4, dtype=torch.bfloat16, device="cuda")
        w8.mxfp4_gemm(buf[4:].view(4, 64), q, s32)
    assert e.value.status == 3


@pytest.mark.parametrize("M", [1, 40, 700])
def test_quantise_and_multiply_in_a_graph(M):
    """Weights quantised, multiplied and read back in one captured stream: every replay gives the eager bits."""
    print(f"[graph] M {M}", flush=True)
    N, K = 1552, 608
    rng = np.random.default_rng(M)
    w = to_dev_bf16(synth.f32_to_bf16_bits(rng.standard_normal((N, K), dtype=np.float32)))
    xs = [to_dev_bf16(synth.f32_to_bf16_bits(rng.standard_normal((M, K), dtype=np.float32))) for _ in range(3)]

    def chain(x):
        q, s, g = w8.nvfp4_quantize(w)
        mq, ms = w8.mxfp4_quantize(w)
        return w8.nvfp4_gemm(x, q, s, g), w8.mxfp4_gemm(x, mq, ms), w8.nvfp4_dequantize(q, s, g)

    want = [[bf16_bits(y) for y in chain(x)] for x in xs]
    torch.cuda.synchronize()
    x = xs[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        chain(x)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = chain(x)
    for i in (0, 1, 2, 1):
        x.copy_(xs[i])
        for o in out:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for o, r in zip(out, want[i]):
            assert np.array_equal(bf16_bits(o), r)
        chain(xs[2])
        torch.cuda.synchronize()


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("M,N,K", [(1, 64, 96), (20, 4112, 160), (40, 96, 32), (500, 1552, 32), (900, 2000, 96), (1030, 2032, 1120),
                                   (4100, 2064, 32)])
def test_gemm_nan_scales_stay_in_their_row(fmt, M, N, K):
    """A NaN block scale is its row's alone: K ends inside a step, where the next bytes are the next row's."""
    print(f"[{fmt} NaN] {M}x{N}x{K}", flush=True)
    rng = np.random.default_rng(N)
    x = synth.activations(rng, M, K)
    (q, s, *g), _ = random_codes(rng, fmt, N, K)
    q, s, g = q[0], s[0].copy(), [np.float32([v[0]]) for v in g]
    want = _gemm(fmt, x, (q, s, *g))
    bad = np.arange(1, N, 5)
    s[bad] = 0xFF if fmt == "mxfp4" else 0x7F
    got = _gemm(fmt, x, (q, s, *g))
    keep = np.setdiff1d(np.arange(N), bad)
    assert np.array_equal(got[:, keep], want[:, keep])


def test_quantize_no_rows():
    q, s, g = w8.nvfp4_quantize(torch.empty((3, 0, 32), dtype=torch.bfloat16, device="cuda"))
    assert q.shape == (3, 0, 16) and s.shape == (3, 0, 2) and g.tolist() == [1.0, 1.0, 1.0]
