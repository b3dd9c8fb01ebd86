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


def test_workspace_keeps_less_than_it_uses():
    """Sizes that rise one by one: each buffer at least doubles, so the
    outgrown ones, which captured graphs may still use, stay below the one in
    use, and that below twice the largest size asked for."""
    import w8a8_int8_gemm_calib_b200 as sq

    ws = sq.Workspace("cpu")
    assert ws.get(0) is None
    handed = []
    for n in range(1000, 200000, 1000):
        b = ws.get(n)
        assert b.numel() >= n
        if not handed or handed[-1] is not b:
            handed.append(b)
    assert len(handed) <= 9  # 1000 x 2^8 >= 199000
    assert sum(b.numel() for b in handed[:-1]) < handed[-1].numel() < 2 * 199000
    assert all(any(b is kept for kept in ws._outgrown) for b in handed[:-1])
    assert ws.get(1) is handed[-1]  # a smaller size reuses it


def test_workspace_first_size_is_the_one_asked_for():
    import w8a8_int8_gemm_calib_b200 as sq

    ws = sq.Workspace("cpu")
    assert ws.get(12345).numel() == 12345
    assert ws.get(1 << 20).numel() == 1 << 20
