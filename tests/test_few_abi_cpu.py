"""The NVFP4, 4-bit product, router and few-token entry points without a GPU:
bad arguments are rejected on the host with the documented status codes."""
import pytest

import w8a8_fp8_linear_amd as w8

OK, NULL, SHAPE, MIS, UNSUP, WS, DEV = range(7)
P = 1 << 20   # a fake, 16-byte aligned address; never dereferenced (checks fail first)


def _no_gpu():
    import torch
    return not torch.cuda.is_available()


def test_nvfp4_quantize():
    f, need = w8.lib().nvfp4_quantize, w8.lib().nvfp4_quantize_workspace_bytes
    assert need(1, 1, 16) == 256 and need(5, 1024, 1024) == 5120 and need(1, 1 << 20, 1024) == 4096 and need(1, 1, 24) == 0 and need(-1, 1, 16) == 0
    assert f(P, -1, 1, 16, P, P, P, 0, P, 256, None) == SHAPE
    assert f(P, 1 << 40, 1 << 20, 1 << 20, P, P, P, 0, P, 256, None) == SHAPE
    assert f(P, 1, 4, 24, P, P, P, 0, P, 256, None) == UNSUP
    assert f(P, 1, 4, 0, P, P, P, 0, P, 256, None) == UNSUP
    assert f(P, 0, 4, 16, P, P, P, 0, P, 256, None) == OK
    assert f(None, 1, 4, 16, P, P, P, 0, P, 256, None) == NULL
    assert f(P, 1, 4, 16, P, P, None, 1, P, 256, None) == NULL
    assert f(P, 1, 4, 16, P, P, P, 0, None, 0, None) == NULL
    assert f(P, 1, 4, 16, P + 8, P, P, 0, P, 256, None) == MIS
    assert f(P, 1, 4, 16, P, P, P, 0, P, 255, None) == WS
    if _no_gpu():
        assert f(P, 1, 4, 16, P, P, P, 1, None, 0, None) == DEV   # a given scale needs no workspace
    d = w8.lib().nvfp4_dequantize
    assert d(P, P, P, 1, 4, 8, P, None) == UNSUP
    assert d(P, P, None, 1, 4, 16, P, None) == NULL
    assert d(P, P + 4, P, 1, 4, 16, P, None) == MIS
    assert d(None, None, None, 1, 0, 16, None, None) == OK


def test_products():
    f, g = w8.lib().nvfp4_gemm, w8.lib().mxfp4_gemm
    assert f(P, P, P, P, P, -1, 16, 32, None) == SHAPE and g(P, P, P, P, -1, 16, 32, None) == SHAPE
    assert f(P, P, P, P, P, 4, 16, 48, None) == UNSUP and g(P, P, P, P, 4, 16, 16, None) == UNSUP
    assert f(P, P, P, P, P, 4, 24, 32, None) == UNSUP
    assert f(P, P, P, P, P, 0, 16, 32, None) == OK and g(P, P, P, P, 4, 0, 32, None) == OK
    assert f(P, P, P, None, P, 4, 16, 32, None) == NULL and g(P, None, P, P, 4, 16, 32, None) == NULL
    assert f(P, P, P, P + 2, P, 4, 16, 32, None) == MIS and g(P, P + 8, P, P, 4, 16, 32, None) == MIS
    if _no_gpu():
        assert f(P, P, P, P + 4, P, 4, 16, 32, None) == DEV       # one float of a vector


def test_router():
    f = w8.lib().moe_router

    size = w8.lib().moe_router_workspace_bytes(4, 8)
    assert size == 4 * 8 * 8 and w8.lib().moe_router_workspace_bytes(4, 1025) == 0

    def call(x=P, wr=P, b=None, ids=P, tw=P, T=4, H=64, E=8, k=2, score=0, ws=P, n=size):
        return f(x, wr, b, ids, tw, T, H, E, k, score, 1, 1.0, ws, n, None)

    assert call(T=-1) == SHAPE
    assert call(H=12) == UNSUP and call(H=0) == UNSUP and call(E=0) == UNSUP and call(E=1025) == UNSUP
    assert call(k=0) == UNSUP and call(k=9) == UNSUP and call(E=128, k=65) == UNSUP and call(score=2) == UNSUP
    assert call(E=1024, H=1 << 20) == UNSUP and call(T=(1 << 24) + 1) == UNSUP
    assert call(T=0) == OK
    assert call(x=None) == NULL and call(tw=None) == NULL
    assert call(b=P + 4) == MIS and call(ids=P + 8) == MIS
    assert call(ws=None) == NULL and call(ws=P + 8) == MIS and call(n=size - 1) == WS
    if _no_gpu():
        assert call() == DEV


@pytest.mark.parametrize("fmt", [0, 1, 2])
def test_few_tokens(fmt):
    f, need = w8.lib().moe_few_tokens, w8.lib().moe_few_tokens_workspace_bytes
    size = need(4, 64, 32, 8, 2)
    assert size == 4 * 2 * 32 * 4 + 4 * 8 * 8                      # h and the logits
    assert need(16, 64, 32, 8, 2) == 16 * 2 * 32 * 4 + 16 * 2 * 64 * 4   # h and the float32 rows
    size = 4 * 2 * 32 * 4                                         # without a router: h

    def call(fmt=fmt, T=4, H=64, I=32, E=8, k=2, x=P, g=P, ws=P, n=size, out=P):
        return f(fmt, x, P, P, P, P, g, P, P, g, out, T, H, I, E, k, ws, n, None)

    assert call(T=-1) == SHAPE
    assert call(fmt=3) == UNSUP and call(fmt=-1) == UNSUP
    assert call(T=65) == UNSUP and call(T=64, k=17) == UNSUP and need(65, 64, 32, 8, 2) == 0
    assert call(H=48) == UNSUP and call(I=16) == UNSUP and call(E=1025) == UNSUP and call(k=0) == UNSUP
    assert call(H=1 << 17, I=1 << 14) == UNSUP
    assert call(T=0) == OK
    assert call(x=None) == NULL and call(ws=None) == NULL
    if fmt == 2:
        assert call(g=None) == NULL
    assert call(out=P + 8) == MIS and call(g=P + 4) == MIS
    assert call(n=size - 1) == WS
    if _no_gpu():
        assert call() == DEV


def test_layer():
    f = w8.lib().moe_few_tokens_layer

    def call(T=4, H=64, I=32, E=8, k=2, x=P, wr=P, b=None, ids=P, score=0, n=4096):
        return f(0, x, wr, b, score, 1, 1.0, ids, P, P, P, None, P, P, None, P, T, H, I, E, k, P, n, None)

    assert call(T=-1) == SHAPE and call(k=9) == UNSUP and call(score=5) == UNSUP and call(H=48) == UNSUP
    assert call(T=0) == OK and call(wr=None) == NULL and call(ids=None) == NULL and call(b=P + 8) == MIS
    assert call(n=16) == WS
    if _no_gpu():
        assert call() == DEV


def test_binding_refuses_host_tensors():
    import torch

    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    q, s = torch.zeros((32, 32), dtype=torch.uint8), torch.zeros((32, 2), dtype=torch.uint8)
    with pytest.raises(ValueError):
        w8.mxfp4_gemm(x, q, s)
    with pytest.raises(ValueError):
        w8.nvfp4_quantize(x)
    with pytest.raises(ValueError):
        w8.moe_router(x, torch.zeros((8, 64), dtype=torch.bfloat16), 2)
    with pytest.raises(ValueError):
        w8.nvfp4_quantize(torch.zeros((2, 2, 2, 16), dtype=torch.bfloat16))
