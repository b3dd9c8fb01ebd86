"""GPU tests of places that sq_moe_sort does not make: rows that several
assignments share, which the combine adds for each of them and dw allows."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U32 = 2.0 ** -24


@pytest.fixture(scope="module")
def sq():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import w8a8_int8_gemm_calib_b200 as m

    return m


@pytest.mark.parametrize("T,k", [(5, 3), (1031, 2), (770, 4), (40, 9)])
@pytest.mark.parametrize("N", [64, 257])
def test_shared_rows(sq, T, k, N):
    """Three rows for all assignments, the same row twice in a token too: the
    sum over assignments and its gradient to the weights, in 64 bits."""
    g = torch.Generator(device="cuda").manual_seed(T + N)
    R = 3
    pos = torch.randint(-1, R, (T, k), device="cuda", generator=g, dtype=torch.int32)
    pos[0] = 1
    z, dy = torch.randn(R, N, device="cuda", generator=g), torch.randn(T, N, device="cuda", generator=g)
    w = torch.rand(T, k, device="cuda", generator=g)
    y, dw = torch.empty(T, N, device="cuda"), torch.empty(T, k, device="cuda")
    sq.sq_moe_combine(z, pos, y, weights=w)
    sq.sq_moe_combine_grad(dy, pos, z=z, dweights=dw)
    sq.sq_sync_status()
    live = (pos >= 0).double()
    rows = z.double()[pos.clamp(min=0).long()] * live[..., None]  # [T, k, N]
    terms = rows * w.double()[..., None]
    # k additions, one rounding of the result
    assert bool(((y.double() - terms.sum(1)).abs() <= (k + 1) * U32 * terms.abs().sum(1)).all())
    prod = rows * dy.double()[:, None]
    # a thread's chain of up to 4 columns, 5 levels of lanes, up to 8 warps
    assert bool(((dw.double() - prod.sum(2)).abs() <= (4 + 5 + 8) * U32 * prod.abs().sum(2) * 1.001).all())
