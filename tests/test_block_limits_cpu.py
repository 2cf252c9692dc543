"""Sizes of the block-scaled expert pass whose offsets inside a tile would leave 32 bits are refused on the host.

The addresses are fake: a call that the checks let through is made where there is no GPU alone."""
import pytest

import w8a8_fp8_linear_amd as w8

OK, NULL, SHAPE, MIS, UNSUP, WS, DEV = range(7)
P = 1 << 20


def _call(T, H, I, E, k):
    return w8.lib().moe_w8a8_block_grouped(P, P, P, P, P, P, P, P, P, None, None, T, H, I, E, k, P, 1 << 62, None)


# tiles of 128, 64 and 32 rows of h, few rows
@pytest.mark.parametrize("T,H,I,E,k", [(351, 16, 38346880, 1, 1), (351, 16, 1 << 24, 1, 1), (100, 16, 38346880, 1, 1),
                                       (40, 16, 1 << 25, 1, 1), (2, 16, 1 << 25, 1, 1), (2, 16, 1 << 24, 2, 2)])
def test_hidden_rows_beyond_32_bits(T, H, I, E, k):
    """127 I + I reaches 2^31 from I = 2^24 on; every other limit lets these sizes through."""
    assert 2 * I * H < 1 << 31 and T * k * I <= 1 << 40 and (T * k // 64 + E + 1) * (1 + I // 128) < 1 << 21
    assert _call(T, H, I, E, k) == UNSUP
    assert w8.lib().moe_w8a8_block_workspace_bytes(T, H, I, E, k) == 0
    with pytest.raises(ValueError, match="unsupported"):
        w8.moe_w8a8_block_workspace(T, H, I, E, k, device="cpu")


def test_the_widest_hidden_rows():
    I = (1 << 24) - 128
    assert w8.lib().moe_w8a8_block_workspace_bytes(351, 16, I, 1, 1) > 351 * I
    import torch

    if not torch.cuda.is_available():
        assert _call(351, 16, I, 1, 1) == DEV
