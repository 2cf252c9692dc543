"""Sizes that no launch can take (2^32 work items or more in a grid) are refused on the host, and the last below them are not.

The addresses are fake: a call that the checks let through is made where there is no GPU alone."""
import w8a8_fp8_linear_amd as w8

UNSUP, DEV = 4, 6
P = 1 << 20   # a fake, 16-byte aligned address; never dereferenced (checks fail first)


def _no_gpu():
    import torch
    return not torch.cuda.is_available()


def _need(*shape):
    return w8.lib().nvfp4_quantize_workspace_bytes(*shape)


def _nvfp4(G, R, K):
    """The status of quantising with a scale to find, with a given one, and of the way back."""
    quant = [w8.lib().nvfp4_quantize(P, G, R, K, P, P, P, given, P, 1 << 40, None) for given in (0, 1)]
    return (*quant, w8.lib().nvfp4_dequantize(P, P, P, G, R, K, P, None))


def _check_nvfp4(refused, taken):
    for shape in refused:
        assert _need(*shape) == 0, shape           # as the shape check of the calls says
        if _no_gpu():
            assert _nvfp4(*shape) == (UNSUP,) * 3, shape
    for shape in taken:
        assert _need(*shape) > 0, shape
        if _no_gpu():
            assert _nvfp4(*shape) == (DEV,) * 3, shape


def test_nvfp4_workgroups():
    """256 threads a chunk of a group: 2^24 chunks are too many."""
    _check_nvfp4([(1 << 24, 1, 16), (1 << 24, 7, 32), (1 << 14, 1024, 4096), (1 << 31, 1, 16)],
                 [((1 << 24) - 1, 1, 16), ((1 << 13) - 1, 1024, 4096)])


def test_nvfp4_values():
    """2048 values a workgroup of the way back: 2^35 are too many."""
    _check_nvfp4([(32, 1 << 20, 1024), (1, 1 << 25, 1024), (1, 1, 1 << 35)],
                 [(31, 1 << 20, 1024), (1, (1 << 25) - 2, 1024)])


def test_router_workgroups():
    """512 threads for 16 tokens and 16 experts: 2^23 such tiles are too many."""
    def call(T, E, H=8):
        return w8.lib().moe_router(P, P, None, P, P, T, H, E, 1, 0, 1, 1.0, P, T * E * 8, None)

    def need(T, E):
        return w8.lib().moe_router_workspace_bytes(T, E)

    for T, E in (1 << 23, 256), (1 << 21, 1024), ((1 << 21) - 15, 1009), (1 << 24, 113):
        assert need(T, E) == 0, (T, E)
        if _no_gpu():
            assert call(T, E) == UNSUP, (T, E)
    for T, E in ((1 << 23) - 16, 256), ((1 << 21) - 16, 1024), (1 << 24, 112):
        assert need(T, E) == T * E * 8, (T, E)
        if _no_gpu():
            assert call(T, E) == DEV, (T, E)
