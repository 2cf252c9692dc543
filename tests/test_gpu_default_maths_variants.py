"""Parity with the float64 oracle at the sizes that take the launches' other variants.

* Products with 4-bit weights, up to 32 rows and 4096 outputs or more: two sets of 16 weight rows a workgroup, one or two
  row tiles, K that ends inside a step and inside a wave's part, N that ends inside the second set.
* Few-token experts: one column tile with K split over two waves or none; several sets of tiles a workgroup; input rows in
  pieces of half a round, of whole rounds and ragged; the small down projection over several rounds of K and with experts
  that several tokens share.

Weights are random codes: quantising as many as these sizes have would take longer than the tests.
"""
import numpy as np
import pytest

import oracle
import synth
from few_util import FORMATS, few_bound, out_violations
from gpu_util import BF16_MFMA_ERR, U32, bf16_bits, bf16_ulp, to_dev, to_dev_bf16

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no GPU", allow_module_level=True)

import w8a8_fp8_linear_amd as w8  # noqa: E402


def _codes(rng, fmt, *shape):
    """Weights of some 2^-4 in random codes: the tuple that the calls take, and their float64 values by matrix."""
    *lead, K = shape
    if fmt == "fp8":
        q = rng.integers(0, 256, shape, dtype=np.uint8)
        q[(q & 0x7F) == 0x7F] = 0
        s = rng.uniform(2e-4, 6e-4, lead).astype(np.float32)
        return (q, s), lambda e: oracle.decode(q[e]) * s[e].astype(np.float64)[:, None]
    q = rng.integers(0, 256, (*lead, K // 2), dtype=np.uint8)
    if fmt == "mxfp4":
        s = rng.integers(119, 124, (*lead, K // 32), dtype=np.uint8)
        return (q, s), lambda e: oracle.mx_dequant(q[e], s[e])
    s = rng.integers(0x28, 0x48, (*lead, K // 16), dtype=np.uint8)
    g = rng.uniform(0.02, 0.04, lead[:-1]).astype(np.float32)
    return (q, s, g), lambda e: oracle.nvfp4_scaled(q[e], s[e]) * float(g[e])


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("N", [4096, 4112])
@pytest.mark.parametrize("M", [1, 16, 17, 32])
def test_wide_products_of_few_rows(fmt, M, N):
    for K in (32, 96, 1056, 2080):
        print(f"[{fmt}_gemm] {M}x{N}x{K}", flush=True)
        rng = np.random.default_rng(M + N + K)
        x = synth.activations(rng, M, K, n_outlier=2)
        w, val = _codes(rng, fmt, 1, N, K)
        y = oracle.bf16_bits_to_f64(bf16_bits((w8.nvfp4_gemm if fmt == "nvfp4" else w8.mxfp4_gemm)(
            to_dev_bf16(x), *(to_dev(a[0] if i < 2 else a) for i, a in enumerate(w)))))
        wv, x64 = val(0), oracle.bf16_bits_to_f64(x)
        # exact products, 2^-20 for an MFMA's own sum, one rounding an instruction, and the waves' parts and the scale
        err = (BF16_MFMA_ERR + (K / 32 + 5) * U32) * 1.01 * (np.abs(x64) @ np.abs(wv).T)
        assert (np.abs(y - x64 @ wv.T) <= err + 0.5 * bf16_ulp(y)).all()


# T, H, I, E, k
_SIZES = [
    (16, 160, 96, 200, 16), (16, 1120, 672, 30, 4),               # one column tile, two waves a tile
    (16, 384, 192, 200, 16), (9, 288, 512, 160, 20),              # one column tile, a wave a tile
    (16, 512, 288, 256, 17), (64, 512, 288, 256, 8),              # several sets of tiles a workgroup
    (64, 96, 1120, 2, 2), (64, 64, 640, 2, 1), (40, 96, 1120, 1, 1), (43, 64, 416, 1, 1),   # pieces of h
    (16, 96, 1120, 4, 2), (12, 160, 1696, 30, 3), (13, 64, 544, 2, 2),                      # four waves a tile
    (8, 64, 1120, 6, 4), (3, 32, 2080, 5, 4), (8, 96, 544, 3, 3), (1, 64, 992, 64, 64), (7, 128, 32, 2, 1),  # small
]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,H,I,E,k", _SIZES)
def test_few_tokens(fmt, T, H, I, E, k):
    print(f"[few] {fmt} T={T} H={H} I={I} E={E} k={k}", flush=True)
    rng = np.random.default_rng(T * 31 + H + I + E)
    x = synth.activations(rng, T, H, n_outlier=1)
    ids, tw = synth.routing(rng, T, E, k)
    w13, v13 = _codes(rng, fmt, E, 2 * I, H)
    w2, v2 = _codes(rng, fmt, E, H, I)
    got = w8.moe_few_tokens(to_dev_bf16(x), to_dev(ids), to_dev(tw), *(tuple(to_dev(a) for a in w) for w in (w13, w2)))
    ref, _, mag = oracle.wide_pass(x, ids, tw, v13, v2)
    assert torch.isfinite(got).all() and np.isfinite(ref).all()
    assert out_violations(bf16_bits(got), ref, few_bound(mag, H, I, k)) == 0
