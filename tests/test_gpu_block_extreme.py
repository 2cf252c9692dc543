"""The expert pass in tiles where the scales' products come near the end of float32's range and past it, and the
outputs do not: a copy keeps the documented rounding, 2^-11 of its value or 2^-12 of topk_w times the sum of the
products of the scales.

Every row of W13 and of W2 has one code, so that every sum of a product is one exact term. Both blocks of 128 columns
of h are alike, so that the sum of a row's two scale products is twice one of them; W2's own code in a row is 2^-9 or
its negative in one of the blocks and nothing in the other, so that the values stay below 448 2^-9 of that.
"""
import numpy as np
import pytest

import oracle
from block_util import hidden_bound, violations
from gpu_util import U32, bf16_bits, to_dev
from moe_util import swiglu_bound

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no GPU", allow_module_level=True)

import w8a8_fp8_linear_amd as w8  # noqa: E402

H, I, E, K = 144, 256, 6, 2


def _one_code(rng, rows, cols, codes):
    q = np.zeros((rows, cols), np.uint8)
    at = rng.integers(0, cols, rows)
    q[np.arange(rows), at] = rng.choice(np.array(codes, np.uint8), rows)
    return q, at


# tiles of 32, 64 and 128 rows; 2^below under the end of the range
@pytest.mark.parametrize("below", [0, 1, 2, 3, 6, 10, 100])
@pytest.mark.parametrize("T", [40, 200, 1300])
def test_scales_at_the_end_of_the_range(T, below):
    print(f"[block] extreme scales T{T} 2^-{below}", flush=True)
    rng = np.random.default_rng(1000 * T + below)
    x = (rng.standard_normal((T, H)) * 2).astype(np.float32)
    qx, sx = oracle.quantize_row_blocks(x)
    q13 = np.zeros((E, 2 * I, H), np.uint8)
    q2 = np.zeros((E, H, I), np.uint8)
    col = np.zeros((E, H), np.int64)
    for e in range(E):
        for half in (0, 1):  # gate and up: the second block of columns repeats the first
            q, _ = _one_code(rng, 128, H, (0x38, 0xB8, 0x3A, 0xB4))
            q13[e, half * I:half * I + 128] = q13[e, half * I + 128:half * I + 256] = q
        q2[e], col[e] = _one_code(rng, H, I, (0x01, 0x81))
    ids = np.argsort(rng.random((T, E)), axis=1)[:, :K].astype(np.int32)
    tw = rng.random((T, K)).astype(np.float32) + np.float32(0.1)
    # h, exactly but for silu's roundings, with up's scales at 2^up
    up = 60
    s13 = np.ones((E, 2 * I // 128, 2), np.float32)
    s13[:, I // 128:] = 2.0 ** up
    xv = oracle.row_values(qx, sx)
    hid = []
    for e in range(E):
        w13 = oracle.weight_values(q13[e], s13[e])
        t, j = np.nonzero(ids == e)
        hid.append((t, j, *hidden_bound(*swiglu_bound(xv[t] @ w13.T, np.zeros((t.size, 2 * I))))))
    # the largest product of two scales just below 2^(128 - below)
    top = max(float(s.max()) for *_, s in hid)
    power = 128 - below - int(np.floor(np.log2(top * 1.001))) - 1
    s2 = np.full((E, 2, 2), 2.0 ** power, np.float32)
    tw = np.ldexp(tw, -70).astype(np.float32)
    ref, err = np.zeros((T, H)), np.zeros((T, H))
    past = 0
    for e, (t, j, h, off, s) in enumerate(hid):
        w2 = oracle.weight_values(q2[e], s2[e])
        w = tw[t, j].astype(np.float64)[:, None]
        y = (h @ w2.T) * w
        size = 1.001 * (s.sum(1) * 2.0 ** power)[:, None] * w
        past += int((s.sum(1) * 2.0 ** power >= 2.0 ** 128).sum())
        np.add.at(ref, t, y)
        # 8 U32: the roundings of the products of the scales, of the router weight and of the sum
        np.add.at(err, t, off[:, col[e]] * np.abs(w2[np.arange(H), col[e]]) * w + np.maximum(2.0 ** -11 * np.abs(y), 2.0 ** -12 * size) + 8 * U32 * np.abs(y))
    assert (past > 0) == (below == 0), past
    got = bf16_bits(w8.moe_w8a8_block_grouped(*(to_dev(a) for a in (qx, sx, ids, tw, q13, s13, q2, s2))))
    assert np.isfinite(oracle.bf16_bits_to_f64(got)).all()
    assert violations(got, ref, err) == 0
