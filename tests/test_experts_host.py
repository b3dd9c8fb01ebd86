"""Host-side checks of the routed-expert calls and the residual norm
quantizer: every refusal comes before anything reaches the GPU."""
import pytest
import torch

# fake, never dereferenced device addresses
A = 1 << 20
A2 = (1 << 20) + 4096
MIS = (1 << 20) + 8


@pytest.fixture(scope="module")
def lib():
    from w8a8_int8_gemm_calib_b200 import _lib

    return _lib


def test_add_rms_checks(lib):
    def call(x=A, res=A, xt=1, T=4, K=16, g=A2, eps=1e-5, gran=1, h=A, act=A2, xq=A2, ncl=None):
        return lib.lib.sq_add_rms_smooth_quant_act(x, res, xt, T, K, g, eps, gran, h, act, xq, ncl,
                                                   None)

    for name in ("x", "res", "g", "h", "act", "xq"):
        assert call(**{name: None}) == lib.SQ_ERR_INVALID_ARG, name
        assert call(**{name: MIS}) == lib.SQ_ERR_ALIGN, name
    for xt in (2, 3, 4, 7):  # int8 and the integer types are not activations
        assert call(xt=xt) == lib.SQ_ERR_DTYPE
    assert call(K=24) == lib.SQ_ERR_SHAPE and call(K=133152) == lib.SQ_ERR_SHAPE
    assert call(T=-1) == lib.SQ_ERR_SHAPE
    assert call(gran=3) == lib.SQ_ERR_INVALID_ARG
    assert call(ncl=A + 4) == lib.SQ_ERR_ALIGN
    for eps in (-1.0, float("nan"), float("inf")):
        assert call(eps=eps) == lib.SQ_ERR_INVALID_ARG
    assert "sq_add_rms_smooth_quant_act" in lib.last_error()
    for gran in (0, 1, 2):
        assert call(T=0, gran=gran) == lib.SQ_OK
        assert call(T=0, gran=gran, x=None, res=None, h=None, xq=None) == lib.SQ_OK


def test_moe_sort_checks(lib):
    def call(ids=A, it=4, T=4, k=2, E=8, off=A, pos=A2, ws=None, n=0):
        return lib.lib.sq_moe_sort(ids, it, T, k, E, off, pos, ws, n, None)

    for it in (0, 1, 2, 5):
        assert call(it=it) == lib.SQ_ERR_DTYPE
    for bad in (dict(T=-1), dict(k=0), dict(E=0), dict(E=1025), dict(T=1 << 31, k=1),
                dict(T=1 << 20, k=1 << 11), dict(T=0, k=0)):
        assert call(**bad) == lib.SQ_ERR_SHAPE, bad
    for name in ("ids", "off", "pos"):
        assert call(**{name: None}) == lib.SQ_ERR_INVALID_ARG
        assert call(**{name: MIS}) == lib.SQ_ERR_ALIGN
    L = lib.lib
    assert L.sq_moe_sort_workspace_bytes(1024, 2, 64) == 0
    need = L.sq_moe_sort_workspace_bytes(1025, 2, 64)
    assert need == 2 * 64 * 4
    assert L.sq_moe_sort_workspace_bytes(0, 2, 64) == 0
    assert L.sq_moe_sort_workspace_bytes(-1, 2, 64) == 0
    assert L.sq_moe_sort_workspace_bytes(1 << 30, 2, 64) == 0  # refused sizes need none
    big = dict(T=1025, k=2, E=64)
    assert call(**big) == lib.SQ_ERR_WORKSPACE
    assert call(ws=A, n=need - 1, **big) == lib.SQ_ERR_WORKSPACE
    assert call(ws=MIS, n=need, **big) == lib.SQ_ERR_ALIGN


def test_moe_gather_checks(lib):
    def call(x=A, xt=2, T=4, K=16, sc=None, pos=A2, k=2, R=8, xs=A, so=None):
        return lib.lib.sq_moe_gather(x, xt, T, K, sc, pos, k, R, xs, so, None)

    for xt in (3, 4, 9):
        assert call(xt=xt) == lib.SQ_ERR_DTYPE
    for bad in (dict(T=-1), dict(k=0), dict(K=0), dict(K=(1 << 20) + 1), dict(R=-1),
                dict(R=1 << 31), dict(T=1 << 30, k=2)):
        assert call(**bad) == lib.SQ_ERR_SHAPE, bad
    assert call(sc=A) == lib.SQ_ERR_INVALID_ARG and call(so=A) == lib.SQ_ERR_INVALID_ARG
    for name in ("x", "pos", "xs"):
        assert call(**{name: None}) == lib.SQ_ERR_INVALID_ARG
        assert call(**{name: MIS}) == lib.SQ_ERR_ALIGN
    assert call(sc=MIS, so=A) == lib.SQ_ERR_ALIGN
    assert call(T=0) == lib.SQ_OK and call(R=0) == lib.SQ_OK


def test_moe_combine_checks(lib):
    def call(z=A, t=1, R=8, N=16, pos=A2, w=None, T=4, k=2, res=None, y=A):
        return lib.lib.sq_moe_combine(z, t, R, N, pos, w, T, k, res, y, None)

    for t in (2, 3, 4):
        assert call(t=t) == lib.SQ_ERR_DTYPE
    for bad in (dict(T=-1), dict(k=0), dict(N=0), dict(N=(1 << 20) + 1), dict(R=-1), dict(R=1 << 31)):
        assert call(**bad) == lib.SQ_ERR_SHAPE, bad
    for name in ("z", "pos", "y"):
        assert call(**{name: None}) == lib.SQ_ERR_INVALID_ARG
    for name in ("z", "pos", "y", "w", "res"):
        assert call(**{name: MIS}) == lib.SQ_ERR_ALIGN
    assert call(T=0) == lib.SQ_OK


def test_moe_combine_grad_checks(lib):
    def call(dy=A, t=1, T=4, N=16, pos=A2, w=None, k=2, z=A, R=8, dz=A, dw=A):
        return lib.lib.sq_moe_combine_grad(dy, t, T, N, pos, w, k, z, R, dz, dw, None)

    assert call(t=2) == lib.SQ_ERR_DTYPE
    for bad in (dict(T=-1), dict(k=0), dict(N=0), dict(R=-1)):
        assert call(**bad) == lib.SQ_ERR_SHAPE, bad
    for name in ("dy", "pos", "z"):
        assert call(**{name: None}) == lib.SQ_ERR_INVALID_ARG
    for name in ("dy", "pos", "w", "z", "dz", "dw"):
        assert call(**{name: MIS}) == lib.SQ_ERR_ALIGN
    assert call(T=0) == lib.SQ_OK
    assert call(dz=None, dw=None) == lib.SQ_OK  # nothing asked for


def test_grouped_checks(lib):
    def call(xq=A, wq=A, off=A2, R=8, N=16, K=16, E=4, act=A, pt=1, ws=A, bias=None, y=A, yt=1,
             acc=None):
        return lib.lib.sq_gemm_w8a8_grouped(xq, wq, off, R, N, K, E, act, pt, ws, bias, y, yt, acc,
                                            None)

    for yt in (2, 3, 4):
        assert call(yt=yt) == lib.SQ_ERR_DTYPE
    for bad in (dict(R=-1), dict(N=-1), dict(K=0), dict(K=24), dict(K=133152), dict(E=0),
                dict(E=1025), dict(R=(1 << 30) + 1), dict(N=(1 << 30) + 1),
                dict(R=1 << 30, N=1 << 20)):
        assert call(**bad) == lib.SQ_ERR_SHAPE, bad
    for name in ("xq", "wq", "off", "act", "ws", "y"):
        assert call(**{name: None}) == lib.SQ_ERR_INVALID_ARG
    for name in ("xq", "wq", "off", "act", "ws", "y", "bias", "acc"):
        assert call(**{name: MIS}) == lib.SQ_ERR_ALIGN
    assert call(R=0) == lib.SQ_OK and call(N=0) == lib.SQ_OK


def test_python_arguments():
    """The wrappers refuse a wrong type or size before they look at a device."""
    import w8a8_int8_gemm_calib_b200 as sq

    f, i32 = torch.float32, torch.int32
    with pytest.raises(TypeError):
        sq.sq_moe_sort(torch.zeros(4, 2), 8, torch.zeros(9, dtype=i32), torch.zeros(4, 2, dtype=i32))
    z, pos, y = torch.zeros(8, 16), torch.zeros(4, 2, dtype=torch.int64), torch.zeros(4, 16)
    with pytest.raises((TypeError, ValueError)):  # int64 places (a CPU tensor either way)
        sq._arg(pos, "pos", i32, 8)
    with pytest.raises(ValueError):
        sq._arg(y, "y", f, 65)
    with pytest.raises(TypeError):
        sq.sq_moe_gather(z.half(), pos, z.half())
    with pytest.raises(ValueError):
        sq.sq_moe_combine_grad(y, pos, dweights=torch.zeros(4, 2))
    assert sq._arg(None, "bias", f, 3) is None
    with pytest.raises(ValueError):
        sq._scratch(None, 64, "sq_moe_sort")
    assert sq._scratch(None, 0, "sq_moe_sort") == (None, 0)
