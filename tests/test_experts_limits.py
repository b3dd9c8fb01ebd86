"""Host-side limits of the routed-expert calls and what a Workspace holds: no
call here reaches a GPU."""
import pytest

A, A2 = 1 << 20, (1 << 20) + 4096  # fake, never dereferenced device addresses


@pytest.fixture(scope="module")
def lib():
    from w8a8_int8_gemm_calib_b200 import _lib

    return _lib


@pytest.mark.parametrize("top_k", [(1 << 30) + 1, (1 << 31) - 8, (1 << 31) - 1])
def test_choices_past_the_32_bit_counters(lib, top_k):
    """The combine and its gradient count a token's choices in eights in 32
    bits: from 2^31 - 8 choices on the count would never end.  Past 2^30 they
    are refused."""
    L = lib.lib
    assert L.sq_moe_combine(A, 1, 8, 16, A2, None, 1, top_k, None, A, None) == lib.SQ_ERR_SHAPE
    assert "top_k" in lib.last_error()
    assert L.sq_moe_combine_grad(A, 1, 1, 16, A2, None, top_k, A, 8, A, A, None) == lib.SQ_ERR_SHAPE
    assert "top_k" in lib.last_error()
