"""The default-maths operators of the routed experts and the 4-bit weights: what is measured of them.

Four families, each in its plain form here (elementary torch operations in 32 bits, 64 where the order
of two experts may hang on the last bits) and, where ``own`` is true, through the framework's calls:

* ``quant``   BF16 -> NVFP4 (E2M1 codes, an E4M3 scale per 16 values, a float32 scale per group) and back:
              what a checkpoint conversion does, and the emulation an accuracy check runs.
* ``linear``  BF16 activations times 4-bit weights (NVFP4 or MXFP4) widened as they are multiplied.
* ``router``  float32 router scores, the top-k experts of every token, their weights.
* ``layer``   a whole routed-expert layer for a few tokens: router, gate/up, SwiGLU, down, weighted sum,
              with FP8, MXFP4 or NVFP4 experts and BF16 activations.
"""
import math

import numpy as np
import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
GSCALE_MIN = 2.0 ** -96


def listed():
    return [
        # one 1024 x 1024 projection of a checkpoint being converted
        dict(name="quant 1024x1024", op="quant", G=1, R=1024, K=1024),
        # the gate/up weights of 128 experts, a float32 scale for each expert
        dict(name="quant 128x1024x1024", op="quant", G=128, R=1024, K=1024),
        # one conversation: a projection for a single token
        dict(name="nvfp4 M1 8192x2048", op="linear", fmt="nvfp4", M=1, N=8192, K=2048),
        # two dozen conversations, an output width that is no multiple of a tile
        dict(name="mxfp4 M24 6160x2048", op="linear", fmt="mxfp4", M=24, N=6160, K=2048),
        # a short prompt with ragged edges in all three sizes
        dict(name="mxfp4 M301 1040x1056", op="linear", fmt="mxfp4", M=301, N=1040, K=1056),
        # a 4096-token prompt through a wide projection
        dict(name="nvfp4 M4096 6144x2048", op="linear", fmt="nvfp4", M=4096, N=6144, K=2048),
        # one token's choice among 192 experts, sigmoid scores with a balance bias
        dict(name="router T1 E192", op="router", T=1, H=1024, E=192, k=4, score="sigmoid", bias=True),
        # a prompt's choices among 64 experts
        dict(name="router T4096 E64", op="router", T=4096, H=2048, E=64, k=8, score="softmax", bias=False),
        # one conversation through 128 FP8 experts in a 1024-wide latent space
        dict(name="layer fp8 T1 E128", op="layer", fmt="fp8", T=1, H=1024, I=512, E=128, k=4, score="softmax", bias=False),
        # eight conversations, 4-bit experts
        dict(name="layer nvfp4 T8 E64", op="layer", fmt="nvfp4", T=8, H=2048, I=512, E=64, k=8, score="softmax", bias=False),
        # an odd few, block scales that are powers of two, sigmoid scores with a balance bias
        dict(name="layer mxfp4 T5 E192", op="layer", fmt="mxfp4", T=5, H=1024, I=512, E=192, k=4, score="sigmoid", bias=True),
        # as many conversations as the few-token form takes: nearly every expert is read
        dict(name="layer fp8 T64 E64", op="layer", fmt="fp8", T=64, H=2048, I=512, E=64, k=8, score="softmax", bias=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quant", "linear", "router", "layer"])
    if op == "quant":
        K = 32 * _log_int(rng, 1, 128)
        G = _log_int(rng, 1, 128)
        R = _log_int(rng, 8, max(9, min(4096, (128 << 20) // (G * K))))
        return dict(op=op, G=G, R=R, K=K)
    if op == "linear":
        N, K = 16 * _log_int(rng, 16, 512), 32 * _log_int(rng, 4, 128)
        M = _log_int(rng, 1, max(2, min(4096, (4096 * 6144 * 2048) // (N * K))))
        return dict(op=op, fmt=rng.choice(["nvfp4", "mxfp4"]), M=M, N=N, K=K)
    if op == "router":
        E = _log_int(rng, 8, 256)
        H = 32 * _log_int(rng, 4, 128)
        T = _log_int(rng, 1, max(2, min(4096, (4096 * 2048 * 64) // (H * E))))
        return dict(op=op, T=T, H=H, E=E, k=rng.randint(1, 8), score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5)
    H, I = 32 * _log_int(rng, 8, 64), 32 * _log_int(rng, 4, 32)
    E = _log_int(rng, 8, max(9, min(192, (64 * 2048 * 512) // (H * I))))
    return dict(op=op, fmt=rng.choice(["fp8", "mxfp4", "nvfp4"]), T=_log_int(rng, 1, 64), H=H, I=I, E=E, k=rng.randint(1, 8),
                score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5)


# ---- inputs -------------------------------------------------------------------


def _activations(g, M, K):
    """BF16 [M, K]: N(0, 1) with one channel in a hundred 20 times as large."""
    x = torch.randn((M, K), device="cuda", generator=g)
    x[:, torch.randperm(K, device="cuda", generator=g)[: K // 100]] *= 20.0
    return x.bfloat16()


def _weights(g, *shape):
    return (0.02 * torch.randn(shape, device="cuda", generator=g)).bfloat16()


def _e2m1_codes(v):
    """float -> 4-bit codes, to nearest, ties to the even code, |v| > 6 saturating."""
    a = v.abs()
    c = (a > 0.25).to(torch.uint8)
    for i, t in enumerate((0.75, 1.25, 1.75, 2.5, 3.5, 5.0)):
        c += (a >= t) if i % 2 == 0 else (a > t)
    return c | (torch.signbit(v).to(torch.uint8) << 3)


def _pack(c):
    return (c[..., 0::2] | (c[..., 1::2] << 4)).contiguous()


def _as_fp8(w):
    """Per-row E4M3: codes as bytes, float32 scales."""
    s = w.float().abs().amax(-1) / 448.0
    return (w.float() / s[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), s


def _as_mxfp4(w):
    """One power of two per 32 values: codes, E8M0 bytes."""
    b = w.float().unflatten(-1, (-1, 32))
    e = torch.floor(torch.log2(b.abs().amax(-1).clamp_min(1e-30))) - 2
    return _pack(_e2m1_codes(b / torch.exp2(e)[..., None]).flatten(-2)), (e + 127).to(torch.uint8)


def _as_nvfp4(w):
    """One E4M3 scale per 16 values and one float32 scale per matrix: codes, E4M3 bytes, float32 scales."""
    g = w.float().abs().amax((-2, -1)) / 2688.0
    b = w.float().unflatten(-1, (-1, 16))
    s = (b.abs().amax(-1) / 6.0 / g[..., None, None]).clamp(max=448.0).to(torch.float8_e4m3fn)
    d = s.float() * g[..., None, None]
    return _pack(_e2m1_codes(b / d.clamp_min(1e-30)[..., None]).flatten(-2)), s.view(torch.uint8), g


def _packed(fmt, w):
    return {"fp8": _as_fp8, "mxfp4": _as_mxfp4, "nvfp4": _as_nvfp4}[fmt](w)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case)
    if case["op"] == "quant":
        s["x"] = _weights(g, case["G"], case["R"], case["K"])
    elif case["op"] == "linear":
        s["x"] = _activations(g, case["M"], case["K"])
        w = _weights(g, 1, case["N"], case["K"])
        q = _packed(case["fmt"], w)
        s["w"] = (q[0][0], q[1][0]) + tuple(q[2:])
        s["y"] = torch.empty((case["M"], case["N"]), dtype=torch.bfloat16, device="cuda")
    else:
        T, H, E = case["T"], case["H"], case["E"]
        s["x"] = _activations(g, T, H)
        s["wr"] = (torch.randn((E, H), device="cuda", generator=g) / (2 * H ** 0.5)).bfloat16()
        s["b"] = 0.05 * torch.randn(E, device="cuda", generator=g) if case["bias"] else None
        s["ids"] = torch.empty((T, case["k"]), dtype=torch.int32, device="cuda")
        s["tw"] = torch.empty((T, case["k"]), dtype=torch.float32, device="cuda")
        if case["op"] == "layer":
            I = case["I"]
            s["w13"] = _packed(case["fmt"], _weights(g, E, 2 * I, H))
            s["w2"] = _packed(case["fmt"], _weights(g, E, H, I))
            s["y"] = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
            s["work"] = torch.empty(T * case["k"] * (H + I) * 4 + 65536, dtype=torch.uint8, device="cuda")
    return s


# ---- plain forms --------------------------------------------------------------


def _value_table():
    """[256, 2] float32: the two values of a byte of E2M1 codes, the low nibble's first."""
    one = torch.tensor(E2M1 + tuple(-v for v in E2M1), device="cuda")
    return torch.stack([one.repeat(16), one.repeat_interleave(16)], -1)


def _widen(fmt, q, s, g=None):
    """Codes and scales -> float32 weights."""
    if fmt == "fp8":
        return q.view(torch.float8_e4m3fn).float() * s[..., None]
    v = _value_table()[q.int()].flatten(-2)
    if fmt == "mxfp4":
        return (v.unflatten(-1, (-1, 32)) * torch.exp2(s.float() - 127.0)[..., None]).flatten(-2)
    return (v.unflatten(-1, (-1, 16)) * (s.view(torch.float8_e4m3fn).float() * g[..., None, None])[..., None]).flatten(-2)


def _plain_quant(s):
    x = s["x"].float()
    amax = x.abs().amax((1, 2))
    # each quotient of the scales rounded once to float32 (a division by a number is a product with its reciprocal
    # in torch, off by a last bit, and a scale next to a border would fall to the other side)
    g = torch.where(amax > 0, (amax.double() / 2688.0).float().clamp_min(GSCALE_MIN), 1.0)
    b = x.unflatten(-1, (-1, 16))
    t = ((b.abs().amax(-1).double() / 6.0).float().double() / g.double()[:, None, None]).float()
    sb = t.clamp(max=448.0).to(torch.float8_e4m3fn)
    d = (sb.float() * g[:, None, None])[..., None]
    v = torch.where(d > 0, b / torch.where(d > 0, d, 1.0), 0.0)
    a = v.abs()
    up = (a > 0.25).float() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + 2 * (a > 2.5) + 2 * (a >= 3.5) + 4 * (a > 5.0)
    y = torch.copysign(up / 2, v) * d
    return y.flatten(-2).bfloat16(), sb, g


def _plain_router(s):
    logits = s["x"].double() @ s["wr"].double().T
    if s["score"] == "softmax":
        p = torch.exp(logits - logits.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
    else:
        p = 1 / (1 + torch.exp(-logits))
    by = p if s["b"] is None else p + s["b"].double()
    ids = torch.sort(by, dim=1, descending=True, stable=True).indices[:, : s["k"]]
    w = p.gather(1, ids)
    return ids.int(), (w / w.sum(1, keepdim=True)).float()


def _plain_layer(s):
    ids, tw = _plain_router(s)
    x, T, k, E, I = s["x"].float(), s["T"], s["k"], s["E"], s["I"]
    if T * k < E:  # fewer routed copies than experts: each copy's own weights
        at = ids.flatten().long()
        x = x.repeat_interleave(k, 0)[:, :, None]
        gu = (_widen(s["fmt"], *(t[at] for t in s["w13"])) @ x)[..., 0]
        h = gu[:, :I] / (1 + torch.exp(-gu[:, :I])) * gu[:, I:]
        y = (_widen(s["fmt"], *(t[at] for t in s["w2"])) @ h[:, :, None])[..., 0]
        out = (y.view(T, k, -1) * tw[..., None]).sum(1)
    else:  # every expert on every token, weighted by the router (nothing where it was not chosen)
        full = torch.zeros((T, E), device="cuda").scatter_(1, ids.long(), tw)
        gu = x @ _widen(s["fmt"], *s["w13"]).transpose(1, 2)
        h = gu[..., :I] / (1 + torch.exp(-gu[..., :I])) * gu[..., I:] * full.T[..., None]
        out = (h @ _widen(s["fmt"], *s["w2"]).transpose(1, 2)).sum(0)
    return out.bfloat16(), ids, tw


def run(s):
    if own:
        import w8a8_fp8_linear_amd as w8

        if s["op"] == "quant":
            q, sb, g = w8.nvfp4_quantize(s["x"])
            return w8.nvfp4_dequantize(q, sb, g), sb.view(torch.float8_e4m3fn), g
        if s["op"] == "linear":
            f = w8.nvfp4_gemm if s["fmt"] == "nvfp4" else w8.mxfp4_gemm
            return f(s["x"], *s["w"], out=s["y"])
        if s["op"] == "router":
            return w8.moe_router(s["x"], s["wr"], s["k"], bias=s["b"], score=s["score"], ids=s["ids"], weights=s["tw"])
        return w8.moe_few_tokens_layer(s["x"], s["wr"], s["w13"], s["w2"], s["k"], bias=s["b"], score=s["score"], out=s["y"],
                                       ids=s["ids"], weights=s["tw"], workspace=s["work"])
    if s["op"] == "quant":
        return _plain_quant(s)
    if s["op"] == "linear":
        w = tuple(t[None] if i < 2 else t for i, t in enumerate(s["w"]))
        return (s["x"].float() @ _widen(s["fmt"], *w)[0].T).bfloat16()
    return _plain_router(s) if s["op"] == "router" else _plain_layer(s)


# ---- what a pass cannot do without ----------------------------------------------


def _weight_bytes(fmt, rows, K):
    return rows * {"fp8": K + 4, "mxfp4": K // 2 + K // 32, "nvfp4": K // 2 + K // 16}[fmt]


def work(case):
    if case["op"] == "quant":
        n = case["G"] * case["R"] * case["K"]
        return {"bytes": 4 * n + 2 * (n // 2 + n // 16), "flops": 6 * n}
    if case["op"] == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": 2 * M * K + _weight_bytes(case["fmt"], N, K) + 2 * M * N, "flops": 2 * M * N * K}
    T, H, E, k = case["T"], case["H"], case["E"], case["k"]
    b, f = 2 * T * H + 2 * E * H + 8 * T * k, 2 * T * E * H
    if case["op"] == "layer":
        I = case["I"]
        # experts that at least one of T tokens picks, taking every choice of k of E as alike
        hit = E * (1 - (1 - k / E) ** T)
        b += hit * (_weight_bytes(case["fmt"], 2 * I, H) + _weight_bytes(case["fmt"], H, I)) + 2 * T * H
        f += 2 * T * k * 3 * I * H
    return {"bytes": float(b), "flops": float(f)}


# ---- the definition in 64 bits ---------------------------------------------------


def _exact_values(fmt, q, s, g):
    """One matrix of codes and scales -> float64, from the bit fields."""
    if fmt == "fp8":
        c = q.long()
        e, m = (c >> 3) & 15, (c & 7).double()
        v = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.exp2(e.double() - 10))
        return torch.where(c >= 128, -v, v) * s.double()[:, None]
    c = torch.stack([q & 15, q >> 4], -1).flatten(-2).long()
    e, m = (c >> 1) & 3, (c & 1).double()
    v = torch.where(e == 0, m / 2, (2 + m) * torch.exp2(e.double() - 2))
    v = torch.where(c >= 8, -v, v)
    if fmt == "mxfp4":
        return v * torch.exp2(s.double() - 127).repeat_interleave(32, -1)
    return v * _exact_values("fp8", s, torch.ones(s.shape[0], device="cuda"), None).repeat_interleave(16, -1) * float(g)


def _exact_router(s):
    logits = s["x"].double() @ s["wr"].double().T
    p = torch.softmax(logits, 1) if s["score"] == "softmax" else torch.sigmoid(logits)
    by = p + (0 if s["b"] is None else s["b"].double())
    order = np.argsort(-by.cpu().numpy(), axis=1, kind="stable")[:, : s["k"]]
    ids = torch.from_numpy(np.ascontiguousarray(order)).cuda()
    w = torch.stack([p[t, ids[t]] for t in range(ids.shape[0])])
    return ids, w / w.sum(1, keepdim=True)


def _exact_quant(s):
    """By the steps that define the codes: quotients are rounded to float32, then to the nearest code."""
    out, scales, groups = [], [], []
    f32 = lambda t: t.float().double()  # noqa: E731
    mags = torch.tensor([m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1],
                        dtype=torch.float64, device="cuda")
    for x in s["x"]:
        x = x.double()
        top = float(x.abs().max())
        g = float(np.float32(max(float(np.float32(top / 2688.0)), GSCALE_MIN) if top else 1.0))
        b = x.reshape(-1, 16)
        t = f32(f32(b.abs().amax(1) / 6.0) / g).clamp(max=448.0)
        i = torch.searchsorted(mags, t).clamp(1, 126)  # mags[i - 1] <= t <= mags[i], ties to the even code
        lo, hi = t - mags[i - 1], mags[i] - t
        sb = torch.where((hi < lo) | ((hi == lo) & (i % 2 == 0)), mags[i], mags[i - 1])
        d = f32(sb * g)[:, None]
        v = torch.where(d > 0, f32(b / torch.where(d > 0, d, 1.0)), 0.0)
        a = v.abs()
        r = torch.where(a < 2, torch.round(a * 2) / 2, torch.where(a < 4, torch.round(a), torch.round(a / 2) * 2)).clamp(max=6.0)
        out.append((torch.copysign(r, v) * d).reshape(x.shape))
        scales.append(sb.reshape(x.shape[0], -1))
        groups.append(g)
    return torch.stack(out), torch.stack(scales), torch.tensor(groups, dtype=torch.float64, device="cuda")


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quant":
        return _exact_quant(s)
    if case["op"] == "linear":
        q, sc, *g = s["w"]
        return s["x"].double() @ _exact_values(case["fmt"], q, sc, g[0] if g else None).T
    ids, w = _exact_router(s)
    if case["op"] == "router":
        return ids, w
    out = torch.zeros((case["T"], case["H"]), dtype=torch.float64, device="cuda")
    for e in ids.unique().tolist():
        t, j = (ids == e).nonzero(as_tuple=True)
        m = [_exact_values(case["fmt"], *(p[e] for p in s[n]), *([None] if len(s[n]) == 2 else [])) for n in ("w13", "w2")]
        gu = s["x"][t].double() @ m[0].T
        h = gu[:, : case["I"]] * torch.sigmoid(gu[:, : case["I"]]) * gu[:, case["I"]:]
        out.index_add_(0, t, (h @ m[1].T) * w[t, j][:, None])
    return out, ids, w
