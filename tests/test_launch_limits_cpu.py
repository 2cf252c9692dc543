"""Sizes that no launch can take (2^32 work items or more in a grid) are refused on the host, and the last below them are not."""
import w8a8_fp8_linear_amd as w8

SHAPE, UNSUP, DEV = 2, 4, 6
P = 1 << 20   # a fake, 16-byte aligned address; never dereferenced (checks fail first)


def _no_gpu():
    import torch
    return not torch.cuda.is_available()


def _nvfp4(G, R, K, given=0):
    need = w8.lib().nvfp4_quantize_workspace_bytes(G, R, K)
    q = w8.lib().nvfp4_quantize(P, G, R, K, P, P, P, given, P, max(need, 16), None)
    return need, q, w8.lib().nvfp4_dequantize(P, P, P, G, R, K, P, None)


def test_nvfp4_workgroups():
    """256 threads a chunk of a group: 2^24 chunks are too many."""
    refused = [(1 << 24, 1, 16), (1 << 24, 7, 32), (1 << 14, 1024, 4096), (1 << 31, 1, 16)]
    for shape in refused:
        need, q, d = _nvfp4(*shape)
        assert need == 0 and q == UNSUP and d == UNSUP, shape
    for shape in ((1 << 24) - 1, 1, 16), ((1 << 13) - 1, 1024, 4096):
        assert _nvfp4(*shape)[0] > 0, shape
        if _no_gpu():
            assert _nvfp4(*shape)[1:] == (DEV, DEV), shape


def test_nvfp4_values():
    """2048 values a workgroup of the way back: 2^35 are too many."""
    for shape in ((32, 1 << 20, 1024), (1, 1 << 25, 1024), (1, 1, 1 << 35)):
        need, q, d = _nvfp4(*shape)
        assert need == 0 and q == UNSUP and d == UNSUP, shape
        assert _nvfp4(*shape, given=1)[1] == UNSUP
    for shape in ((31, 1 << 20, 1024), (1, (1 << 25) - 2, 1024)):
        assert _nvfp4(*shape)[0] > 0, shape
        if _no_gpu():
            assert _nvfp4(*shape)[1:] == (DEV, DEV), shape


def test_router_workgroups():
    """512 threads for 16 tokens and 16 experts: 2^23 such tiles are too many."""
    def call(T, E, H=8):
        n = w8.lib().moe_router_workspace_bytes(T, E)
        return n, w8.lib().moe_router(P, P, None, P, P, T, H, E, 1, 0, 1, 1.0, P, max(n, T * E * 8), None)

    for T, E in (1 << 23, 256), (1 << 21, 1024), ((1 << 21) - 15, 1009), (1 << 24, 113):
        assert call(T, E) == (0, UNSUP), (T, E)
    for T, E in ((1 << 23) - 16, 256), ((1 << 21) - 16, 1024), (1 << 24, 112):
        assert call(T, E)[0] == T * E * 8
        if _no_gpu():
            assert call(T, E)[1] == DEV
