"""FP8 with a scale per block of 128, and the router's balance loss: what is measured of them.

Four families, each in its plain form here (elementary torch operations in 32 bits) and, where ``own`` is true,
through the framework's calls:

* ``quant``    BF16 -> E4M3 codes with one float32 scale per 128 values of a row (activations) or per 128 x 128
               values (weights): what a step does with its input, and what a checkpoint conversion does.
* ``linear``   a linear layer: the BF16 input quantised by blocks, times the block-scaled weights.
* ``experts``  a routed-expert pass: input quantised by blocks, gate/up, SwiGLU, h quantised by blocks, down,
               weighted sum of a token's copies.
* ``balance``  the balance loss of a router's choice, tokens per expert, and the gradient of the logits.
"""
import math

import torch

own = False

B = 128  # values a scale covers along K, and rows of a weight block
COEF = 0.01


def listed():
    return [
        # the input of a projection, a 4096-token prompt
        dict(name="quant acts 4096x2048", op="quant", E=0, N=4096, K=2048),
        # the gate/up weights of 128 experts of a checkpoint being converted
        dict(name="quant weights 128x1024x1024", op="quant", E=128, N=1024, K=1024),
        # one conversation: a projection of a single token
        dict(name="linear M1 8192x2048", op="linear", M=1, N=8192, K=2048),
        # two dozen conversations, an output width that is no multiple of a block
        dict(name="linear M24 6160x2048", op="linear", M=24, N=6160, K=2048),
        # a short prompt, ragged edges in all three sizes
        dict(name="linear M301 1040x1056", op="linear", M=301, N=1040, K=1056),
        # a 4096-token prompt through a wide projection
        dict(name="linear M4096 6144x2048", op="linear", M=4096, N=6144, K=2048),
        # one conversation through 128 experts in a 1024-wide latent space
        dict(name="experts T1 E128", op="experts", T=1, H=1024, I=512, E=128, k=4),
        # some dozen conversations: most experts have one token or none
        dict(name="experts T37 E192", op="experts", T=37, H=1024, I=512, E=192, k=4),
        # a 4096-token prompt, 512 routed copies an expert
        dict(name="experts T4096 E64", op="experts", T=4096, H=2048, I=512, E=64, k=8),
        # the load of one decoding step, sigmoid scores
        dict(name="balance 1x64 E192", op="balance", S=1, L=64, E=192, k=4, score="sigmoid", dtype="float32", pad=False),
        # a batch of padded sequences, a loss for each, logits in 16 bits
        dict(name="balance 4x1000 E64 bf16", op="balance", S=4, L=1000, E=64, k=8, score="softmax", dtype="bfloat16", pad=True),
        # one loss over the whole batch of a training step
        dict(name="balance 1x65536 E128", op="balance", S=1, L=65536, E=128, k=4, score="softmax", dtype="float32", pad=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quant", "linear", "experts", "balance"])
    if op == "quant":
        K, E = 16 * _log_int(rng, 8, 512), rng.choice([0, _log_int(rng, 1, 128)])
        return dict(op=op, E=E, N=_log_int(rng, 1, max(2, min(8192, (1 << 27) // (max(E, 1) * K)))), K=K)
    if op == "linear":
        N, K = 16 * _log_int(rng, 16, 512), 16 * _log_int(rng, 8, 256)
        return dict(op=op, M=_log_int(rng, 1, max(2, min(4096, (4096 * 6144 * 2048) // (N * K)))), N=N, K=K)
    if op == "experts":
        H, I, k = 16 * _log_int(rng, 16, 128), B * _log_int(rng, 1, 8), rng.randint(1, 8)
        E = _log_int(rng, 8, max(9, min(192, (64 * 2048 * 512) // (H * I))))
        return dict(op=op, T=_log_int(rng, 1, max(2, min(4096, (4096 * 2048 * 512) // (H * I), (4096 * 2048 * 512 * 64) // (H * I * E)))), H=H, I=I, E=E, k=k)
    E = _log_int(rng, 8, 256)
    S = _log_int(rng, 1, 16)
    return dict(op=op, S=S, L=_log_int(rng, 1, (65536 * 128) // (S * E)), E=E, k=rng.randint(1, 8), score=rng.choice(["softmax", "sigmoid"]),
                dtype=rng.choice(["float32", "bfloat16"]), pad=rng.random() < 0.5)


# ---- inputs -------------------------------------------------------------------


def _activations(g, M, K):
    """BF16 [M, K]: N(0, 1) with one channel in a hundred 20 times as large."""
    x = torch.randn((M, K), device="cuda", generator=g)
    x[:, torch.randperm(K, device="cuda", generator=g)[: K // 100]] *= 20.0
    return x.bfloat16()


def _weights(g, *shape):
    """BF16 weights whose rows differ in size."""
    return (0.02 * torch.exp(0.3 * torch.randn((*shape[:-1], 1), device="cuda", generator=g))
            * torch.randn(shape, device="cuda", generator=g)).bfloat16()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case)
    if case["op"] == "quant":
        s["x"] = _weights(g, case["E"], case["N"], case["K"]) if case["E"] else _activations(g, case["N"], case["K"])
    elif case["op"] == "linear":
        s["x"] = _activations(g, case["M"], case["K"])
        s["w"] = _plain_weight_blocks(_weights(g, 1, case["N"], case["K"]))
        s["w"] = tuple(t[0] for t in s["w"])
        s["y"] = torch.empty((case["M"], case["N"]), dtype=torch.bfloat16, device="cuda")
    elif case["op"] == "experts":
        T, H, I, E, k = (case[n] for n in ("T", "H", "I", "E", "k"))
        s["x"] = _activations(g, T, H)
        s["w13"] = _plain_weight_blocks(_weights(g, E, 2 * I, H))
        s["w2"] = _plain_weight_blocks(_weights(g, E, H, I))
        likes = torch.randn((T, E), device="cuda", generator=g) + 0.5 * torch.randn(E, device="cuda", generator=g)
        top = torch.sort(likes, dim=1, descending=True, stable=True)
        s["ids"] = top.indices[:, :k].int().contiguous()
        w = torch.exp(top.values[:, :k])
        s["tw"] = (w / w.sum(1, keepdim=True)).contiguous()
        s["y"] = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    else:
        S, L, E, k = (case[n] for n in ("S", "L", "E", "k"))
        logits = torch.randn((S * L, E), device="cuda", generator=g) + 0.5 * torch.randn(E, device="cuda", generator=g)
        s["logits"] = logits.to(getattr(torch, case["dtype"]))
        s["ids"] = torch.sort(s["logits"].float(), dim=1, descending=True, stable=True).indices[:, :k].int().contiguous()
        if case["pad"]:  # the places behind a sequence's end name no expert
            ends = torch.randint(L // 2, L + 1, (S, 1), device="cuda", generator=g)
            behind = (torch.arange(L, device="cuda")[None] >= ends).flatten()
            s["ids"][behind] = -1
    return s


# ---- plain forms --------------------------------------------------------------


def _padded(x, rows):
    """float32, filled up with zeros to whole blocks: the last dimension, and with ``rows`` the one before it."""
    x = x.float()
    more = [0, -x.shape[-1] % B] + ([0, -x.shape[-2] % B] if rows else [])
    return torch.nn.functional.pad(x, more) if any(more) else x


def _scale(amax):
    # rounded once: torch takes a division by a number as a product with its reciprocal
    return torch.where(amax > 0, (amax.double() / 448.0).float(), 1.0)


def _plain_row_blocks(x):
    """Codes [M, K] as E4M3 and scales [blocks of K, M]."""
    b = _padded(x, False).unflatten(-1, (-1, B))
    sc = _scale(b.abs().amax(-1))
    q = (b / sc[..., None]).clamp(-448, 448).flatten(-2)[..., : x.shape[-1]].to(torch.float8_e4m3fn)
    return q, sc.transpose(0, 1).contiguous()


def _plain_weight_blocks(w):
    """Codes as bytes [E, N, K] and scales [E, blocks of N, blocks of K]."""
    b = _padded(w, True).unflatten(-1, (-1, B)).unflatten(1, (-1, B))  # [E, nb, B, kb, B]
    sc = _scale(b.abs().amax((2, 4)))
    q = (b / sc[:, :, None, :, None]).clamp(-448, 448).flatten(3, 4).flatten(1, 2)[:, : w.shape[1], : w.shape[2]]
    return q.to(torch.float8_e4m3fn).view(torch.uint8).contiguous(), sc


def _row_values(q, sc):
    """Codes [M, K] and scales [blocks, M] -> float32."""
    return q.float() * sc.T.repeat_interleave(B, 1)[:, : q.shape[1]]


def _weight_values(q, sc):
    q = q.view(torch.float8_e4m3fn).float()
    return q * sc.repeat_interleave(B, -1)[..., : q.shape[-1]].repeat_interleave(B, -2)[..., : q.shape[-2], :]


def _plain_experts(s):
    T, k, E, I, H = (s[n] for n in ("T", "k", "E", "I", "H"))
    x = _row_values(*_plain_row_blocks(s["x"]))

    def hidden(gu):  # [..., 2 I] -> h in its FP8 values
        h = gu[..., :I] / (1 + torch.exp(-gu[..., :I])) * gu[..., I:]
        return _row_values(*_plain_row_blocks(h.reshape(-1, I))).view(h.shape)

    if T * k < E:  # fewer routed copies than experts: each copy's own weights
        at = s["ids"].flatten().long()
        x = x.repeat_interleave(k, 0)[:, :, None]
        h = hidden((_weight_values(*(t[at] for t in s["w13"])) @ x)[..., 0])
        y = (_weight_values(*(t[at] for t in s["w2"])) @ h[:, :, None])[..., 0]
        return (y.view(T, k, H) * s["tw"][..., None]).sum(1).bfloat16()
    # every expert on every token, weighted by the router (nothing where it was not chosen)
    full = torch.zeros((T, E), device="cuda").scatter_(1, s["ids"].long(), s["tw"])
    h = hidden(x @ _weight_values(*s["w13"]).transpose(1, 2)) * full.T[..., None]
    return (h @ _weight_values(*s["w2"]).transpose(1, 2)).sum(0).bfloat16()


def _plain_balance(s):
    S, L, E, k = (s[n] for n in ("S", "L", "E", "k"))
    ids = s["ids"].view(S, L * k).long()
    real = (ids >= 0) & (ids < E)
    counts = torch.zeros((S, E + 1), dtype=torch.int32, device="cuda")
    counts.scatter_add_(1, torch.where(real, ids, E), torch.ones_like(ids, dtype=torch.int32))
    counts = counts[:, :E].contiguous()
    here = real.view(S, L, k).any(-1)  # the tokens that count
    n = here.sum(1).clamp_min(1).float()
    l = s["logits"].float().view(S, L, E)
    if s["score"] == "softmax":
        p = torch.exp(l - l.amax(-1, keepdim=True))
        slope = 1.0
    else:
        p = 1 / (1 + torch.exp(-l))
        slope = 1 - p
    p = p / p.sum(-1, keepdim=True)
    f = counts.float() * (E / (k * n))[:, None]
    loss = COEF / S * (f * (torch.where(here[..., None], p, 0.0).sum(1, dtype=torch.float64) / n[:, None])).sum()
    # f and f - 1 give the same gradient, as p sums to one; f - 1 loses less
    up = (f - 1)[:, None] * (COEF / (S * n))[:, None, None]
    grad = torch.where(here[..., None], p * slope * (up - (up * p).sum(-1, keepdim=True)), 0.0)
    return loss.float(), counts, grad.view(S * L, E).to(s["logits"].dtype)


def run(s):
    if own:
        import w8a8_fp8_linear_amd as w8

        if s["op"] == "quant":
            q, sc = w8.quantize_weight_blocks(s["x"]) if s["E"] else w8.quantize_blocks(s["x"])
            return q.view(torch.float8_e4m3fn), sc
        if s["op"] == "linear":
            return w8.w8a8_block_linear(s["x"], *s["w"], out=s["y"])
        if s["op"] == "experts":
            q, sc = w8.quantize_blocks(s["x"])
            return w8.moe_w8a8_block_grouped(q, sc, s["ids"], s["tw"], *s["w13"], *s["w2"], out=s["y"])
        return w8.moe_balance_loss(s["logits"], s["ids"], coef=COEF, sequences=s["S"], score=s["score"])
    if s["op"] == "quant":
        if not s["E"]:
            return _plain_row_blocks(s["x"])
        q, sc = _plain_weight_blocks(s["x"])
        return q.view(torch.float8_e4m3fn), sc
    if s["op"] == "linear":
        return (_row_values(*_plain_row_blocks(s["x"])) @ _weight_values(*s["w"]).T).bfloat16()
    return _plain_experts(s) if s["op"] == "experts" else _plain_balance(s)


# ---- what a pass cannot do without ----------------------------------------------


def _weight_bytes(N, K):
    return N * K + 4 * math.ceil(N / B) * math.ceil(K / B)


def work(case):
    if case["op"] == "quant":
        G, N, K = max(case["E"], 1), case["N"], case["K"]
        scales = math.ceil(N / B) if case["E"] else N
        return {"bytes": G * (3 * N * K + 4 * scales * math.ceil(K / B)), "flops": 3 * G * N * K}
    if case["op"] == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": 2 * M * K + _weight_bytes(N, K) + 2 * M * N, "flops": 2 * M * N * K}
    if case["op"] == "experts":
        T, H, I, E, k = (case[n] for n in ("T", "H", "I", "E", "k"))
        # experts that at least one of T tokens picks, taking every choice of k of E as alike
        hit = E * (1 - (1 - k / E) ** T)
        return {"bytes": float(4 * T * H + 8 * T * k + hit * (_weight_bytes(2 * I, H) + _weight_bytes(H, I))), "flops": 6 * T * k * I * H}
    T, E, k = case["S"] * case["L"], case["E"], case["k"]
    return {"bytes": 2 * T * E * (4 if case["dtype"] == "float32" else 2) + 4 * T * k + 4 * case["S"] * E + 4, "flops": 10 * T * E}


# ---- the definition in 64 bits ---------------------------------------------------


def _e4m3_near(v):
    """float64 -> the nearest E4M3 value, ties to the even code, saturating: by the spacing of the values around it."""
    a = v.abs().clamp(max=448.0)
    _, e = torch.frexp(a)
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3)
    return torch.copysign(torch.round(a / step) * step, v)


def _e4m3_read(c):
    """Bytes -> float64, from the bit fields."""
    c = c.long()
    e, m = (c >> 3) & 15, (c & 7).double()
    v = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.exp2(e.double() - 10))
    return torch.where(c >= 128, -v, v)


def _exact_rows(x):
    """(codes' values, scales [rows, blocks]) of [rows, K], by the steps that define them: both quotients are rounded to float32."""
    x = x.double()
    M, K = x.shape
    block = torch.arange(K, device="cuda") // B
    amax = torch.zeros((M, math.ceil(K / B)), dtype=torch.float64, device="cuda").scatter_reduce_(1, block.expand(M, K), x.abs(), "amax")
    sc = torch.where(amax == 0, 1.0, (amax / 448).float().double())
    return _e4m3_near((x / sc[:, block]).float().double()), sc


def _exact_matrix(q, sc):
    r, c = (torch.arange(n, device="cuda") // B for n in q.shape)
    return _e4m3_read(q) * sc.double()[r][:, c]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quant" and not case["E"]:
        v, sc = _exact_rows(s["x"])
        return v, sc.T
    if case["op"] == "quant":
        codes, scales = [], []
        for w in s["x"]:
            w = w.double()
            sc = torch.stack([torch.stack([piece.abs().max() for piece in band.split(B, 1)]) for band in w.split(B, 0)])
            sc = torch.where(sc == 0, 1.0, (sc / 448).float().double())
            r, c = (torch.arange(n, device="cuda") // B for n in w.shape)
            codes.append(_e4m3_near((w / sc[r][:, c]).float().double()))
            scales.append(sc)
        return torch.stack(codes), torch.stack(scales)
    if case["op"] in ("linear", "experts"):
        v, sc = _exact_rows(s["x"])
        x = v * sc.repeat_interleave(B, 1)[:, : v.shape[1]]
        if case["op"] == "linear":
            return x @ _exact_matrix(*s["w"]).T
        out = torch.zeros((case["T"], case["H"]), dtype=torch.float64, device="cuda")
        for e in s["ids"].unique().tolist():
            t, j = (s["ids"] == e).nonzero(as_tuple=True)
            gu = x[t] @ _exact_matrix(s["w13"][0][e], s["w13"][1][e]).T
            gate, up = gu.split(case["I"], 1)
            hv, hs = _exact_rows(gate * torch.sigmoid(gate) * up)
            y = (hv * hs.repeat_interleave(B, 1)) @ _exact_matrix(s["w2"][0][e], s["w2"][1][e]).T
            out.index_add_(0, t, y * s["tw"][t, j].double()[:, None])
        return out
    S, L, E, k = (case[n] for n in ("S", "L", "E", "k"))
    loss, counts = torch.zeros((), dtype=torch.float64, device="cuda"), []
    l = s["logits"].double().requires_grad_()
    for i in range(S):
        ids = s["ids"][i * L:(i + 1) * L]
        c = torch.bincount(ids[(ids >= 0) & (ids < E)].long(), minlength=E)
        counts.append(c)
        row = l[i * L:(i + 1) * L][((ids >= 0) & (ids < E)).any(1)]
        if len(row):
            p = torch.softmax(row, 1) if case["score"] == "softmax" else torch.sigmoid(row) / torch.sigmoid(row).sum(1, keepdim=True)
            loss = loss + COEF / S * E / (k * len(row)) * (c * p.mean(0)).sum()
    grad = torch.autograd.grad(loss, l)[0] if loss.requires_grad else torch.zeros_like(l)
    return loss.detach(), torch.stack(counts).int(), grad
