"""GPU tests of the routing around the experts: the stable sort and the copies
exactly, the weighted sums and the gradients against 64 bits.

Tolerances: a value rounded to type t is off by at most eps(t) / 2 of it; a
sum of fp32 terms by 2^-24 of the terms' magnitudes for every addition one of
them goes through."""
import numpy as np
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


def _sorted(ids, E):
    """Offsets and places on the host, from the definition."""
    flat = ids.reshape(-1)
    live = (flat >= 0) & (flat < E)
    key = np.where(live, flat, E)
    order = np.argsort(key, kind="stable")
    place = np.empty(flat.size, np.int64)
    place[order] = np.arange(flat.size)
    off = np.searchsorted(key[order], np.arange(E + 1))
    return off, np.where(live, place, -1).reshape(ids.shape)


def _sort(sq, ids, E, ws=None):
    T, k = ids.shape
    off = torch.full((E + 1,), -7, dtype=torch.int32, device="cuda")
    pos = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    sq.sq_moe_sort(ids, E, off, pos, workspace=ws or sq.Workspace())
    sq.sq_sync_status()
    return off, pos


# around a block's 2048 assignments, several blocks, more than one per SM
SORTS = [(1, 1, 1), (1, 8, 64), (3, 2, 1024), (31, 1, 8), (255, 8, 60), (256, 8, 256), (257, 8, 256),
         (2049, 1, 1), (1025, 2, 1024), (5000, 7, 60), (16384, 8, 64), (200003, 3, 128),
         (60001, 8, 1000)]


@pytest.mark.parametrize("T,k,E", SORTS)
@pytest.mark.parametrize("dtype", ["int32", "int64"])
@pytest.mark.parametrize("how", ["even", "skewed", "padded"])
def test_sort(sq, T, k, E, dtype, how):
    r = np.random.default_rng(T + k + E)
    ids = r.integers(0, E, (T, k))
    if how == "skewed":
        ids = np.minimum((E * r.random((T, k)) ** 4).astype(np.int64), E - 1)
    if how == "padded":
        ids = r.integers(-2, E + 2, (T, k))
        ids[r.random(T) < 0.3] = -1
        if dtype == "int64":
            ids[r.random((T, k)) < 0.05] = (1 << 40) + E - 1  # its low half is an id
    off, pos = _sort(sq, torch.from_numpy(ids.astype(dtype)).cuda(), E)
    want_off, want_pos = _sorted(ids, E)
    np.testing.assert_array_equal(off.cpu().numpy(), want_off)
    np.testing.assert_array_equal(pos.cpu().numpy(), want_pos)


@pytest.mark.parametrize("T,E", [(1, 3), (300, 64), (9000, 5)])
def test_sort_one_expert_or_none(sq, T, E):
    """Every assignment to one expert (twice per token), and none to any."""
    ids = torch.full((T, 2), E - 1, device="cuda")
    off, pos = _sort(sq, ids, E)
    assert off.tolist() == [0] * E + [2 * T]
    assert torch.equal(pos.reshape(-1), torch.arange(2 * T, device="cuda", dtype=torch.int32))
    off, pos = _sort(sq, torch.full((T, 2), -1, device="cuda"), E)
    assert off.tolist() == [0] * (E + 1) and bool((pos == -1).all())


def test_sort_no_tokens(sq):
    off, _ = _sort(sq, torch.empty(0, 4, dtype=torch.int64, device="cuda"), 16)
    assert off.tolist() == [0] * 17


def _route(T, k, R, seed, drop=0.2):
    """Places of T x k assignments among R >= T k rows: some rows of no
    assignment, some assignments of no row (also places past R)."""
    r = np.random.default_rng(seed)
    pos = r.permutation(R)[:T * k].reshape(T, k)
    gone = r.random((T, k)) < drop
    pos[gone] = r.choice([-1, R, -5], gone.sum())
    if T > 2:
        pos[T // 2] = -1  # a token of none
    return pos


WIDTHS = [1, 7, 16, 250, 4096, 4100, 5003, 20480]


@pytest.mark.parametrize("K", WIDTHS)
@pytest.mark.parametrize("dtype", [torch.int8, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,k,scaled", [(1, 1, True), (37, 8, True), (65, 3, False), (5, 40, True)])
def test_gather(sq, K, dtype, T, k, scaled):
    R = T * k + 5
    pos = _route(T, k, R, K + T)
    g = torch.Generator(device="cuda").manual_seed(K)
    x = torch.randint(-127, 128, (T, K), device="cuda", generator=g).to(dtype)
    xs = torch.full((R, K), 55, device="cuda").to(dtype)
    sc = torch.rand(T, device="cuda", generator=g) if scaled else None
    ss = torch.full((R,), -3.0, device="cuda") if scaled else None
    want, want_s = xs.clone(), ss.clone() if scaled else None
    sq.sq_moe_gather(x, torch.from_numpy(pos.astype(np.int32)).cuda(), xs, scale=sc, scale_s=ss)
    sq.sq_sync_status()
    for t in range(T):
        for p in pos[t]:
            if 0 <= p < R:
                want[p] = x[t]
                if scaled:
                    want_s[p] = sc[t]
    assert torch.equal(xs, want)
    assert not scaled or torch.equal(ss, want_s)


def _half(t):
    return torch.finfo(t).eps / 2


@pytest.mark.parametrize("N", WIDTHS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,k,weighted,residual", [(1, 1, True, False), (37, 8, True, True),
                                                   (65, 3, False, False), (5, 19, True, True)])
def test_combine(sq, N, dtype, T, k, weighted, residual):
    R = T * k + 3
    pos = _route(T, k, R, N + T)
    g = torch.Generator(device="cuda").manual_seed(N + k)
    z = torch.randn(R, N, device="cuda", generator=g).to(dtype)
    w = torch.rand(T, k, device="cuda", generator=g) if weighted else None
    res = torch.randn(T, N, device="cuda", generator=g).to(dtype) if residual else None
    y = torch.full((T, N), 9.0, device="cuda").to(dtype)
    p32 = torch.from_numpy(pos.astype(np.int32)).cuda()
    sq.sq_moe_combine(z, p32, y, weights=w, residual=res)
    sq.sq_sync_status()
    want = res.double() if residual else torch.zeros(T, N, dtype=torch.float64, device="cuda")
    mag = want.abs()
    live = (pos >= 0) & (pos < R)
    for c in range(k):
        t = torch.from_numpy(np.flatnonzero(live[:, c])).cuda()
        term = z[p32[t, c].long()].double() * (w[t, c, None].double() if weighted else 1.0)
        want[t] += term
        mag[t] += term.abs()
    bound = _half(dtype) * want.abs() + (1 + _half(dtype)) * k * U32 * mag
    assert bool(((y.double() - want).abs() <= bound).all())
    if residual:  # over the residual itself: the same bits
        sq.sq_moe_combine(z, p32, res, weights=w, residual=res)
        sq.sq_sync_status()
        assert torch.equal(res, y)


def test_combine_skips_rows_it_has_no_place_in(sq):
    """A NaN or an infinity in a row of no assignment, or behind a dropped
    one, reaches no output; a token of none gives its residual, or 0."""
    z = torch.full((4, 64), float("nan"), device="cuda")
    z[1] = 2.0
    z[2] = float("inf")
    pos = torch.tensor([[1, -1], [-1, 4], [-2, 1 << 30]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[0.5, float("nan")], [float("inf"), 1.0], [1.0, 1.0]], device="cuda")
    y = torch.full((3, 64), 7.0, device="cuda")
    sq.sq_moe_combine(z, pos, y, weights=w)
    assert torch.equal(y, torch.tensor([1.0, 0.0, 0.0], device="cuda")[:, None].expand(3, 64))
    res = torch.full((3, 64), -4.0, device="cuda")
    sq.sq_moe_combine(z, pos, y, weights=w, residual=res)
    assert torch.equal(y, torch.tensor([-3.0, -4.0, -4.0], device="cuda")[:, None].expand(3, 64))
    # no rows at all
    sq.sq_moe_combine(z[:0], pos, y, weights=w, residual=res)
    sq.sq_sync_status()
    assert torch.equal(y, res)


@pytest.mark.parametrize("N", WIDTHS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,k,weighted", [(1, 1, True), (37, 8, True), (65, 3, False), (5, 19, True)])
@pytest.mark.parametrize("only", ["both", "dz", "dw"])
def test_combine_grad(sq, N, dtype, T, k, weighted, only):
    R = T * k + 3
    pos = _route(T, k, R, N + T + 1)
    g = torch.Generator(device="cuda").manual_seed(N + 2 * k)
    z = torch.randn(R, N, device="cuda", generator=g).to(dtype)
    dy = torch.randn(T, N, device="cuda", generator=g).to(dtype)
    w = torch.rand(T, k, device="cuda", generator=g) if weighted else None
    dz = torch.full((R, N), 9.0, device="cuda").to(dtype)
    dw = torch.full((T, k), 9.0, device="cuda")
    p32 = torch.from_numpy(pos.astype(np.int32)).cuda()
    sq.sq_moe_combine_grad(dy, p32, z=z if only != "dz" else None, weights=w,
                           dz=dz if only != "dw" else None, dweights=dw if only != "dz" else None)
    sq.sq_sync_status()
    live = (pos >= 0) & (pos < R)
    want_z = torch.full((R, N), 9.0, device="cuda", dtype=torch.float64)
    want_w = torch.zeros(T, k, device="cuda", dtype=torch.float64)
    mag_w = torch.zeros_like(want_w)
    for c in range(k):
        t = torch.from_numpy(np.flatnonzero(live[:, c])).cuda()
        p = p32[t, c].long()
        want_z[p] = dy[t].double() * (w[t, c, None].double() if weighted else 1.0)
        prod = dy[t].double() * z[p].double()
        want_w[t, c], mag_w[t, c] = prod.sum(1), prod.abs().sum(1)
    if only != "dw":
        bound = want_z.abs() * ((1 + _half(dtype)) * (1 + U32) - 1)
        assert bool(((dz.double() - want_z).abs() <= bound).all())
    if only != "dz":
        # at most 256 threads of 8 (4) columns a step: a term goes through its
        # thread's chain, 5 levels of lanes and up to 8 warps
        lanes = 8 if dtype is torch.bfloat16 else 4
        steps = 8 + lanes * (N // (256 * lanes) + 1) if N % lanes == 0 else 8 + N // 256 + 1
        bound = (steps + 8 + 5) * U32 * mag_w * 1.001
        assert bool(((dw.double() - want_w).abs() <= bound).all())
        assert bool((dw[torch.from_numpy(~live).cuda()] == 0).all())


def test_gradients_against_differences(sq):
    """The formula's gradients are those of sq_moe_combine and sq_moe_gather:
    along a direction, the change of <dy, y> over a step is the gradients'
    product with it (both are linear in each input: exact but for fp32's
    rounding of sums of 3 x 2 x 40 terms of magnitude below 30)."""
    T, k, N, R = 3, 2, 40, 7
    g = torch.Generator(device="cuda").manual_seed(0)
    pos = torch.tensor([[0, 3], [5, -1], [2, 6]], dtype=torch.int32, device="cuda")
    z, dz_dir = (torch.randn(R, N, device="cuda", generator=g) for _ in range(2))
    w, w_dir = (torch.rand(T, k, device="cuda", generator=g) for _ in range(2))
    dy = torch.randn(T, N, device="cuda", generator=g)

    def loss(z, w):
        y = torch.empty(T, N, device="cuda")
        sq.sq_moe_combine(z.contiguous(), pos, y, weights=w.contiguous())
        return float((y.double() * dy.double()).sum())

    dz, dw = torch.zeros(R, N, device="cuda"), torch.empty(T, k, device="cuda")
    sq.sq_moe_combine_grad(dy, pos, z=z, weights=w, dz=dz, dweights=dw)
    tol = 240 * 30 * 8 * U32
    dir_z = float((dz.double() * dz_dir.double()).sum())
    dir_w = float((dw.double() * w_dir.double()).sum())
    assert abs((loss(z + dz_dir, w) - loss(z - dz_dir, w)) / 2 - dir_z) <= tol
    assert abs((loss(z, w + w_dir) - loss(z, w - w_dir)) / 2 - dir_w) <= tol
    # gather: <dxs, gather(x)> against <combine(dxs), x>
    x, dxs = torch.randn(T, N, device="cuda", generator=g), torch.randn(R, N, device="cuda", generator=g)
    xs, dx = torch.zeros(R, N, device="cuda"), torch.empty(T, N, device="cuda")
    sq.sq_moe_gather(x, pos, xs)
    sq.sq_moe_combine(dxs, pos, dx)
    sq.sq_sync_status()
    a, b = float((dxs.double() * xs.double()).sum()), float((dx.double() * x.double()).sum())
    assert abs(a - b) <= tol


def test_offsets_past_32_bits(sq):
    """A sorted array of more than 2^31 elements: its far rows."""
    T, k, N = 4, 2, 1 << 18
    R = 10240  # 2.7e9 bf16 elements
    z = torch.empty(R, N, dtype=torch.bfloat16, device="cuda")
    pos = torch.tensor([[0, R - 1], [8192, 1], [R - 2, 4096], [-1, 8191]], dtype=torch.int32,
                       device="cuda")
    x = torch.randn(T, N, device="cuda").bfloat16()
    sq.sq_moe_gather(x, pos, z)
    y = torch.empty_like(x)
    sq.sq_moe_combine(z, pos, y)
    dw = torch.empty(T, k, device="cuda")
    sq.sq_moe_combine_grad(x, pos, z=z, dweights=dw)
    sq.sq_sync_status()
    for p, t in [(0, 0), (R - 1, 0), (8192, 1), (R - 2, 2), (8191, 3)]:
        assert torch.equal(z[p], x[t])
    twice = torch.tensor([2.0, 2.0, 2.0, 1.0], device="cuda")[:, None]
    assert torch.equal(y, (x.float() * twice).bfloat16())
    sq2 = x.double().square().sum(1)
    want = torch.stack([sq2, sq2], 1)
    want[3, 0] = 0
    assert bool(((dw.double() - want).abs() <= want * (8 + N // 256 + 13) * U32 * 1.001).all())
