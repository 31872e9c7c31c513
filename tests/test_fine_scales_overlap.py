"""Outputs of the quantiser in the memory of its input, refused on the host before any CUDA call."""
import pytest

A, B, C = 1 << 20, 1 << 21, 1 << 22  # addresses that no refused call follows
BF16 = 0


@pytest.fixture(scope="module")
def m():
    import __graft_entry__

    __graft_entry__.build()
    import moe_decode_host_gb300 as mod

    return mod


@pytest.mark.parametrize("x,y,scale", [(A, A, C), (A, B, A), (A, B, B), (A, A, A)])
@pytest.mark.parametrize("T", [1, 3])
def test_quant_refuses_shared_memory(m, x, y, scale, T):
    assert m.lib.moe_quant_e4m3(x, BF16, 256, T, 256, y, 256, scale, 2, None) == m.MOE_ERR_INVALID_ARG


def test_no_rows_share_nothing(m):
    assert m.lib.moe_quant_e4m3(A, BF16, 256, 0, 256, A, 256, A, 2, None) == m.MOE_OK
