"""GPU parity of the router and of the few-token routed experts.

* Router: the ids equal the float64 oracle's, equal scores in index order;
  weights to float32 rounding of the float64 ones; many and few experts,
  odd lengths, several tokens a workgroup.
* Few-token experts in the three weight formats: every element inside the
  bound of few_util.few_bound; ids that are dropped, repeated or shared by
  all tokens, tokens without an expert, sizes at which the last load is
  ragged; by copies (fewer than experts) and by experts.
* The layer is the router followed by the experts, bit for bit; two passes;
  graph replays; other streams; two calls at once; refused arguments.
"""
import numpy as np
import pytest

import oracle
import synth
from few_util import FORMATS, few_bound, out_violations, random_codes
from gpu_util import bf16_bits, to_dev, to_dev_bf16

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no GPU", allow_module_level=True)

import w8a8_fp8_linear_amd as w8  # noqa: E402


def _router_inputs(rng, T, H, E):
    return synth.activations(rng, T, H, n_outlier=H // 100), synth.weights(rng, (E, H), std=1 / (2 * H ** 0.5))


def _check_router(x, wr, k, **kw):
    ids, w = w8.moe_router(to_dev_bf16(x), to_dev_bf16(wr), k, **{a: to_dev(b) if isinstance(b, np.ndarray) else b
                                                                 for a, b in kw.items()})
    torch.cuda.synchronize()
    if "route_scale" in kw:
        kw["scale"] = np.float64(np.float32(kw.pop("route_scale")))
    rid, rw, by = oracle.router(x, wr, k, **kw)
    # the float64 sums of the two sides differ by their order alone: 2^-53 relative per addition, far below 1e-11
    got = ids.cpu().numpy()
    srt = -np.sort(-by, axis=1)
    gap = (srt[:, :-1] - srt[:, 1:])[:, :k] if by.shape[1] > 1 else np.ones((by.shape[0], 0))
    clear = (gap > 1e-11).all(1) | (gap == 0).any(1)
    assert np.array_equal(got[clear], rid[clear])
    wt = w.cpu().numpy()
    # one rounding to float32 of a value that is right to 1e-12
    assert np.all(np.abs(wt[clear] - rw[clear]) <= 2.0 ** -24 * np.abs(rw[clear]) * 1.001 + 1e-44)
    return got


@pytest.mark.parametrize("T,H,E,k", [(1, 1024, 192, 4), (3, 8, 1, 1), (5, 24, 2, 2), (64, 520, 65, 8), (7, 2056, 8, 8),
                                     (2, 512, 1024, 64), (257, 96, 130, 6), (300, 1024, 64, 8), (263, 40, 1000, 33),
                                     (2051, 264, 50, 5)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_router(T, H, E, k, score):
    print(f"[router] T={T} H={H} E={E} k={k} {score}", flush=True)
    rng = np.random.default_rng(T + H + E)
    x, wr = _router_inputs(rng, T, H, E)
    _check_router(x, wr, k, score=score)
    _check_router(x, wr, k, score=score, bias=rng.standard_normal(E).astype(np.float32) * np.float32(0.1),
                  renormalize=False, route_scale=2.5)


@pytest.mark.parametrize("T", [2, 260])
def test_router_equal_scores(T):
    """Experts with the same row score alike: the lower index goes first; a token of zeros gets 0 .. k-1."""
    rng = np.random.default_rng(1)
    x, wr = _router_inputs(rng, T, 128, 24)
    wr[1::2] = wr[::2]
    x[-1] = 0
    got = _check_router(x, wr, 6)
    assert np.all(got[:-1, 0] % 2 == 0) and np.all(got[:-1, 1] == got[:-1, 0] + 1) and got[-1].tolist() == list(range(6))


def test_router_choice_does_not_depend_on_the_batch():
    rng = np.random.default_rng(2)
    x, wr = _router_inputs(rng, 300, 1024, 96)
    ids, w = w8.moe_router(to_dev_bf16(x), to_dev_bf16(wr), 8)
    for t in (0, 17, 299):
        i1, w1 = w8.moe_router(to_dev_bf16(x[t:t + 1]), to_dev_bf16(wr), 8)
        assert torch.equal(i1[0], ids[t]) and torch.equal(w1[0], w[t])


def test_router_nan_is_last():
    x = np.zeros((1, 16), np.float32)
    x[0, :4] = [1, 2, 3, 4]
    w = np.eye(4, 16, dtype=np.float32)
    w[3, 5] = np.nan
    ids, _ = w8.moe_router(to_dev_bf16(synth.f32_to_bf16_bits(x)), to_dev_bf16(synth.f32_to_bf16_bits(w)), 4,
                           score="sigmoid")
    assert ids[0].tolist() == [2, 1, 0, 3]


def test_router_barred_experts():
    """A bias of -inf bars an expert; where fewer than k are left, the barred follow by index."""
    rng = np.random.default_rng(4)
    x, wr = _router_inputs(rng, 6, 64, 70)
    bias = np.full(70, -np.inf, np.float32)
    bias[[5, 40, 69]] = 0
    ids, w = w8.moe_router(to_dev_bf16(x), to_dev_bf16(wr), 5, bias=to_dev(bias))
    got = ids.cpu().numpy()
    assert np.all(np.sort(got[:, :3], 1) == [5, 40, 69]) and np.all(got[:, 3:] == [0, 1])
    assert torch.isfinite(w).all()


def _experts(rng, fmt, E, I, H):
    w13, v13 = random_codes(rng, fmt, E, 2 * I, H)
    w2, v2 = random_codes(rng, fmt, E, H, I)
    return w13, w2, v13, v2


def _dev(w):
    return tuple(to_dev(a) for a in w)


def _check_few(rng, fmt, x, ids, tw, ex, E, **kw):
    w13, w2, v13, v2 = ex
    out = w8.moe_few_tokens(to_dev_bf16(x), to_dev(ids), to_dev(tw), _dev(w13), _dev(w2), **kw)
    torch.cuda.synchronize()
    H, I = x.shape[1], w2[0].shape[2] * (1 if fmt == "fp8" else 2)
    known = np.where((ids >= 0) & (ids < E), ids, -1)
    ref, _, mag = oracle.wide_pass(x, known, tw, v13, v2)
    got = bf16_bits(out)
    assert out_violations(got, ref, few_bound(mag, H, I, ids.shape[1])) == 0
    return got


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,H,I,E,k", [(1, 32, 32, 1, 1), (1, 1024, 512, 16, 4), (2, 160, 96, 5, 3), (5, 288, 32, 40, 4),
                                       (16, 96, 160, 7, 2), (17, 256, 128, 6, 3), (32, 64, 64, 33, 8), (33, 128, 96, 4, 2),
                                       (64, 160, 64, 3, 3), (64, 96, 224, 200, 16),
                                       # 8 tokens or fewer with more than 64 copies; 9 to 16 ids a token; inputs of several staged pieces
                                       (8, 64, 96, 40, 16), (5, 96, 64, 300, 33), (4, 128, 64, 600, 12),
                                       (64, 4128, 32, 2, 2), (24, 64, 2080, 3, 2), (16, 4128, 64, 2, 2)])
def test_few_tokens(fmt, T, H, I, E, k):
    print(f"[few] {fmt} T={T} H={H} I={I} E={E} k={k}", flush=True)
    rng = np.random.default_rng(T * 31 + H + I + E)
    x = synth.activations(rng, T, H, n_outlier=1)
    ids, tw = synth.routing(rng, T, E, k)
    _check_few(rng, fmt, x, ids, tw, _experts(rng, fmt, E, I, H), E)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,E", [(3, 40), (24, 8), (64, 6)])
def test_few_tokens_odd_routes(fmt, T, E):
    """Dropped ids (-1, E, far outside), a token without an expert, an expert named twice, one expert for all."""
    rng = np.random.default_rng(T + E)
    H, I, k = 96, 64, 4
    ex = _experts(rng, fmt, E, I, H)
    x = synth.activations(rng, T, H)
    ids = rng.integers(0, E, (T, k)).astype(np.int32)   # repeats within a token
    ids[0] = [1, 1, -1, 1]
    ids[1] = [-1, E, 1 << 30, -(1 << 31)]
    tw = rng.standard_normal((T, k)).astype(np.float32)
    got = _check_few(rng, fmt, x, ids, tw, ex, E)
    assert not (got[1] & 0x7FFF).any()
    one = np.full((T, k), E - 1, np.int32)
    _check_few(rng, fmt, x, one, tw, ex, E)
    assert not (_check_few(rng, fmt, x, np.full((T, k), -1, np.int32), tw, ex, E) & 0x7FFF).any()


def test_few_tokens_large_and_small_h():
    """h over many binades: the BF16 pair keeps 16 bits at any size of h."""
    rng = np.random.default_rng(5)
    E, I, H, k = 4, 64, 64, 2
    for up in (1e-12, 1e6):
        w13, v13 = random_codes(rng, "fp8", E, 2 * I, H)
        w13[1][:, I:] *= np.float32(up)
        v = lambda e: oracle.decode(w13[0][e]) * w13[1][e].astype(np.float64)[:, None]  # noqa: E731
        w2, v2 = random_codes(rng, "fp8", E, H, I)
        x = synth.activations(rng, 6, H)
        ids, tw = synth.routing(rng, 6, E, k)
        _check_few(rng, "fp8", x, ids, tw, (w13, w2, v, v2), E)


def _layer_state(fmt, T, H, I, E, seed=0):
    rng = np.random.default_rng(seed)
    w13, w2, v13, v2 = _experts(rng, fmt, E, I, H)
    x, wr = _router_inputs(rng, T, H, E)
    return to_dev_bf16(x), to_dev_bf16(wr), _dev(w13), _dev(w2)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T", [1, 9, 50])
def test_layer_is_router_then_experts(fmt, T):
    x, wr, w13, w2 = _layer_state(fmt, T, 224, 96, 24, seed=T)
    bias = torch.linspace(-0.1, 0.1, 24, device="cuda")
    out, ids, w = w8.moe_few_tokens_layer(x, wr, w13, w2, 4, bias=bias, score="sigmoid", route_scale=1.5)
    i2, t2 = w8.moe_router(x, wr, 4, bias=bias, score="sigmoid", route_scale=1.5)
    o2 = w8.moe_few_tokens(x, i2, t2, w13, w2)
    assert torch.equal(ids, i2) and torch.equal(w, t2) and torch.equal(out, o2)


@pytest.mark.parametrize("T,E,k,score", [(4, 300, 6, "softmax"), (4, 256, 3, "sigmoid"), (3, 65, 12, "softmax"),
                                         (2, 9, 9, "sigmoid"), (4, 3, 2, "softmax"), (5, 64, 4, "softmax")])
def test_layer_choice_in_the_first_projection(T, E, k, score):
    """Up to four tokens the layer may choose inside its first projection: the same choice, weights and output bits as
    the separate calls, by copies and by experts, below and above the sizes at which it does."""
    x, wr, w13, w2 = _layer_state("mxfp4", T, 160, 64, E, seed=E)
    out, ids, w = w8.moe_few_tokens_layer(x, wr, w13, w2, k, score=score, renormalize=k % 2 == 0)
    i2, t2 = w8.moe_router(x, wr, k, score=score, renormalize=k % 2 == 0)
    o2 = w8.moe_few_tokens(x, i2, t2, w13, w2)
    assert torch.equal(ids, i2) and torch.equal(w, t2) and torch.equal(out, o2)


@pytest.mark.parametrize("fmt", FORMATS)
def test_checkpoint_to_two_passes(fmt):
    """BF16 weights quantised by the framework, then the layer run twice on one set of experts, each pass checked on
    the device's own input and choice."""
    rng = np.random.default_rng(21)
    T, H, I, E, k = 11, 256, 128, 12, 3
    b13, b2 = synth.weights(rng, (E, 2 * I, H)), synth.weights(rng, (E, H, I))
    if fmt == "nvfp4":
        w13, w2 = (w8.nvfp4_quantize(to_dev_bf16(b)) for b in (b13, b2))
        val = lambda w: (lambda e: oracle.nvfp4_scaled(w[0][e].cpu().numpy(), w[1][e].cpu().numpy()) * float(w[2][e]))  # noqa: E731
    else:
        f = w8.quantize_per_token if fmt == "fp8" else w8.mxfp4_quantize
        w13, w2 = ([t.view(*b.shape[:2], *t.shape[1:]) for t in f(to_dev_bf16(b.reshape(-1, b.shape[2])))] for b in (b13, b2))
        dec = (lambda q, s: oracle.decode(q) * s.astype(np.float64)[:, None]) if fmt == "fp8" else oracle.mx_dequant
        val = lambda w: (lambda e: dec(w[0][e].cpu().numpy(), w[1][e].cpu().numpy()))  # noqa: E731
    x, _ = _router_inputs(rng, T, H, E)
    routers = [(to_dev_bf16(_router_inputs(rng, T, H, E)[1]), None) for _ in range(2)]
    inp = x
    for out, ids, w in w8.moe_few_tokens_ffn(to_dev_bf16(x), routers, tuple(w13), tuple(w2), k):
        ref, _, mag = oracle.wide_pass(inp, ids.cpu().numpy(), w.cpu().numpy(), val(w13), val(w2))
        got = bf16_bits(out)
        assert out_violations(got, ref, few_bound(mag, H, I, k)) == 0
        inp = got


@pytest.mark.parametrize("fmt,T", [("fp8", 1), ("nvfp4", 40)])
def test_layer_in_a_graph(fmt, T):
    x, wr, w13, w2 = _layer_state(fmt, T, 288, 96, 20, seed=3)
    ws = w8.moe_few_tokens_workspace(T, 288, 96, 20, 4)
    eager = [t.clone() for t in w8.moe_few_tokens_layer(x, wr, w13, w2, 4, workspace=ws)]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = w8.moe_few_tokens_layer(x, wr, w13, w2, 4, workspace=ws)
    for i in range(3):
        for o in outs:
            o.zero_()
        ws.zero_()
        torch.zeros(1 << 20, device="cuda").sum()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, eager)), f"replay {i}"


def test_two_streams_at_once():
    """Two layers on two streams, each with its own buffers, give what they give alone."""
    a, b = (_layer_state("mxfp4", T, 256, 128, 16, seed=T) for T in (8, 30))
    ref = [[t.clone() for t in w8.moe_few_tokens_layer(*s, 4)] for s in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(5):
        for n, (st, s) in enumerate(zip(streams, (a, b))):
            with torch.cuda.stream(st):
                got[n].append(w8.moe_few_tokens_layer(*s, 4))
    torch.cuda.synchronize()
    for n in range(2):
        for r in got[n]:
            assert all(torch.equal(p, q) for p, q in zip(r, ref[n]))


def test_results_repeat():
    s = _layer_state("fp8", 64, 512, 128, 16, seed=7)
    first = w8.moe_few_tokens_layer(*s, 8)[0]
    for _ in range(4):
        assert torch.equal(w8.moe_few_tokens_layer(*s, 8)[0], first)


def test_no_tokens():
    _, wr, w13, w2 = _layer_state("fp8", 1, 64, 32, 4)
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    out, ids, w = w8.moe_few_tokens_layer(x, wr, w13, w2, 2)
    assert out.shape == (0, 64) and ids.shape == (0, 2) and w.shape == (0, 2)


def test_refusals():
    x, wr, w13, w2 = _layer_state("nvfp4", 4, 64, 32, 8)
    ids, w = w8.moe_router(x, wr, 2)
    with pytest.raises(ValueError):
        w8.moe_few_tokens(x, ids, w, w13, w2[:2])
    with pytest.raises(ValueError):
        w8.moe_few_tokens(x, ids[:3], w, w13, w2)
    with pytest.raises(TypeError):
        w8.moe_few_tokens(x, ids.long(), w, w13, w2)
    with pytest.raises(ValueError):
        w8.moe_few_tokens(x, ids, w, (w13[0], w13[1][..., :2].contiguous(), w13[2]), w2)
    with pytest.raises(ValueError):
        w8.moe_router(x, wr, 2, score="relu")
    with pytest.raises(ValueError):
        w8.moe_few_tokens_layer(x, wr[:7], w13, w2, 2)
    with pytest.raises(w8.W8A8Error) as e:   # more experts asked for than there are
        w8.moe_router(x, wr, 9)
    assert e.value.status == 4
    with pytest.raises(w8.W8A8Error) as e:   # 65 tokens
        w8.moe_few_tokens_layer(x.repeat(17, 1)[:65], wr, w13, w2, 2)
    assert e.value.status == 4
    with pytest.raises(w8.W8A8Error) as e:
        w8.moe_few_tokens(x, ids, w, w13, w2, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 5


@pytest.mark.parametrize("fmt", FORMATS)
def test_layer_inputs_that_begin_inside_a_larger_tensor(fmt):
    """Views into larger tensors (a batch's rows, an expert range of a stack), the router's outputs given, canaries
    behind the output and in the rows that no token has."""
    T, H, I, E, k = 3, 96, 64, 12, 2
    x, wr, w13, w2 = _layer_state(fmt, T + 5, H, I, E + 4, seed=2)
    sub13, sub2 = (tuple(t[4:] for t in w) for w in (w13, w2))
    out = torch.full((T + 5, H), 7.0, dtype=torch.bfloat16, device="cuda")
    ids = torch.full((T + 5, k), 77, dtype=torch.int32, device="cuda")
    w = torch.full((T + 5, k), 7.0, device="cuda")
    w8.moe_few_tokens_layer(x[2:2 + T], wr[4:], sub13, sub2, k, out=out[:T], ids=ids[:T], weights=w[:T])
    o2, i2, t2 = w8.moe_few_tokens_layer(x[2:2 + T].clone(), wr[4:].clone(), tuple(t.clone() for t in sub13),
                                         tuple(t.clone() for t in sub2), k)
    assert torch.equal(out[:T], o2) and torch.equal(ids[:T], i2) and torch.equal(w[:T], t2)
    assert (out[T:] == 7).all() and (ids[T:] == 77).all() and (w[T:] == 7).all()


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("T,E", [(1, 8), (7, 8), (12, 60), (40, 5)])
def test_few_tokens_nan_scales_stay_in_their_row(fmt, T, E):
    """A NaN block scale of a W2 row is that output column's alone; I ends inside a step."""
    rng = np.random.default_rng(T)
    H, I, k = 96, 160, 3
    w13, w2, _, _ = _experts(rng, fmt, E, I, H)
    x = to_dev_bf16(synth.activations(rng, T, H))
    ids, tw = (to_dev(a) for a in synth.routing(rng, T, E, k))
    want = bf16_bits(w8.moe_few_tokens(x, ids, tw, _dev(w13), _dev(w2)))
    w2[1][:, 1::3] = 0xFF if fmt == "mxfp4" else 0x7F
    got = bf16_bits(w8.moe_few_tokens(x, ids, tw, _dev(w13), _dev(w2)))
    keep = np.setdiff1d(np.arange(H), np.arange(1, H, 3))
    assert np.array_equal(got[:, keep], want[:, keep])
