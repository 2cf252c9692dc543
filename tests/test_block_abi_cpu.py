"""The block-scaled and balance entry points without a GPU: bad arguments are
rejected on the host with the documented status codes, and sizes that no launch
can take are refused.

The addresses are fake: a call that the checks let through is made where there is no GPU alone."""
import w8a8_fp8_linear_amd as w8

OK, NULL, SHAPE, MIS, UNSUP, WS, DEV = range(7)
P = 1 << 20


def _no_gpu():
    import torch
    return not torch.cuda.is_available()


def test_quantisers():
    f, g = w8.lib().quantize_blocks, w8.lib().quantize_weight_blocks
    assert f(P, -1, 16, P, P, None) == SHAPE and f(P, 1 << 40, 1 << 40, P, P, None) == SHAPE
    assert f(P, 4, 24, P, P, None) == UNSUP and f(P, 4, 0, P, P, None) == UNSUP
    assert f(P, (1 << 26) + 1, 16, P, P, None) == UNSUP and f(P, 4, (1 << 24) + 16, P, P, None) == UNSUP
    assert f(P, 1 << 26, 2064, P, P, None) == UNSUP          # 2^22 x 5 pieces
    assert f(None, 0, 16, None, None, None) == OK
    assert f(P, 4, 16, P, None, None) == NULL and f(P, 4, 16, P + 8, P, None) == MIS
    assert g(P, -1, 4, 16, P, P, None) == SHAPE and g(P, 1 << 30, 1 << 20, 1 << 20, P, P, None) == SHAPE
    assert g(P, 1, 4, 8, P, P, None) == UNSUP and g(P, 1, 1 << 20, 1 << 20, P, P, None) == UNSUP
    assert g(P, 1 << 18, 1 << 10, 1 << 10, P, P, None) == UNSUP   # 2^24 blocks
    assert g(None, 0, 4, 16, None, None, None) == OK and g(None, 3, 0, 16, None, None, None) == OK
    assert g(None, 1, 4, 16, P, P, None) == NULL and g(P, 1, 4, 16, P, P + 4, None) == MIS
    if _no_gpu():
        assert f(P, 1 << 26, 2048, P, P, None) == UNSUP and f(P, (1 << 26) - 16, 2048, P, P, None) == DEV
        assert g(P, (1 << 18) - 1, 1 << 10, 1 << 10, P, P, None) == DEV


def test_products():
    f, lin, need = w8.lib().w8a8_block_gemm, w8.lib().w8a8_block_linear, w8.lib().w8a8_block_linear_workspace_bytes
    assert need(16, 2048) == 0 and need(8, 1 << 20) == 0 and need(9, 2064) > 0 and need(33, 2048) == (33 * 2048 + 255) // 256 * 256 + (16 * 33 * 4 + 255) // 256 * 256
    assert need(33, 24) == 0 and need(-1, 16) == 0 and need(100, 1 << 21) == 0
    for call in (lambda M, N, K: f(P, P, P, P, P, M, N, K, None), lambda M, N, K: lin(P, P, P, P, M, N, K, P, 1 << 40, None)):
        assert call(-1, 16, 16) == SHAPE and call(4, 1 << 62, 16) == SHAPE
        assert call(4, 16, 24) == UNSUP and call(4, 24, 16) == UNSUP and call(4, 16, 0) == UNSUP
        assert call(4, 16, (1 << 20) + 16) == UNSUP and call((1 << 24) + 1, 16, 16) == UNSUP
        assert call(1 << 23, 4096, 16) == UNSUP              # 2^17 x 64 tiles
        assert call(0, 16, 16) == OK and call(4, 0, 16) == OK
        if _no_gpu():
            assert call(4, 16, 16) == DEV and call((1 << 23) - 64, 4096, 16) == DEV
    assert f(P, P, P, None, P, 4, 16, 16, None) == NULL and f(P, P + 8, P, P, P, 4, 16, 16, None) == MIS
    assert lin(P, P, P, P, 40, 16, 32, None, 0, None) == NULL
    assert lin(P, P, P, P, 40, 16, 32, P + 4, 1 << 20, None) == MIS
    assert lin(P, P, P, P, 40, 16, 32, P, need(40, 32) - 1, None) == WS
    if _no_gpu():
        assert lin(P, P, P, P, 16, 16, 32, None, 0, None) == DEV   # few rows need no workspace
        assert lin(P, P, P, P, 40, 16, 32, P, need(40, 32), None) == DEV


def test_experts():
    f, need = w8.lib().moe_w8a8_block_grouped, w8.lib().moe_w8a8_block_workspace_bytes
    size = need(4, 256, 128, 8, 2)

    def call(x=P, out=P, oq=None, os_=None, T=4, H=256, I=128, E=8, k=2, ws=P, n=size):
        return f(x, P, P, P, P, P, P, P, out, oq, os_, T, H, I, E, k, ws, n, None)

    assert size > 0 and need(4, 256, 64, 8, 2) == 0 and need(4, 24, 128, 8, 2) == 0
    assert call(T=-1) == SHAPE and call(E=0) == UNSUP and call(E=1025) == UNSUP and call(k=65) == UNSUP
    assert call(I=64) == UNSUP and call(H=24) == UNSUP and call(T=1 << 20, H=1 << 12) == UNSUP
    assert call(T=1 << 17, H=16, k=64, I=1 << 14) == UNSUP    # 2^17 x 2^7 tiles
    assert call(T=0) == OK
    assert call(x=None) == NULL and call(out=None) == NULL and call(ws=None) == NULL and call(oq=P) == NULL and call(os_=P) == NULL
    assert call(x=P + 8) == MIS and call(oq=P + 8, os_=P) == MIS and call(n=size - 1) == WS
    if _no_gpu():
        assert call() == DEV and call(oq=P, os_=P) == DEV


def test_balance():
    f, need = w8.lib().moe_balance_loss, w8.lib().moe_balance_loss_workspace_bytes

    def call(dtype=0, l=P, ids=P, T=12, S=3, E=8, k=2, score=0, loss=P, counts=P, grad=P, ws=P, n=1 << 40):
        return f(dtype, l, ids, T, S, E, k, score, 0.01, loss, counts, grad, ws, n, None)

    assert need(12, 3, 8) > 0 and need(12, 5, 8) == 0 and need(12, 0, 8) == 0 and need(-1, 1, 8) == 0 and need(12, 3, 1025) == 0
    assert call(T=-3) == SHAPE and call(S=5) == UNSUP and call(S=0) == UNSUP and call(S=1 << 21, T=1 << 22) == UNSUP
    assert call(E=0) == UNSUP and call(E=1025) == UNSUP and call(k=0) == UNSUP and call(k=65) == UNSUP
    assert call(dtype=2) == UNSUP and call(score=2) == UNSUP and call(T=3 << 24) == UNSUP
    assert call(l=None) == NULL and call(ids=None) == NULL and call(loss=None) == NULL and call(counts=None) == NULL and call(ws=None) == NULL
    assert call(l=P + 4) == MIS and call(grad=P + 8) == MIS and call(loss=P + 2) == MIS and call(counts=P + 4) == MIS
    assert call(n=need(12, 3, 8) - 1) == WS
    if _no_gpu():
        assert call() == DEV and call(grad=None) == DEV and call(loss=P + 4) == DEV and call(T=0, l=None, ids=None) == DEV


def test_router_with_logits():
    f = w8.lib().moe_router_with_logits

    def call(logits=P, T=4):
        return f(P, P, None, P, P, logits, T, 64, 8, 2, 0, 1, 1.0, P, 4 * 8 * 8, None)

    assert call(logits=None) == NULL and call(logits=P + 4) == MIS and call(T=0) == OK
    if _no_gpu():
        assert call() == DEV
