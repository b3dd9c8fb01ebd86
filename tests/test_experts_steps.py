"""GPU tests of the combine and its gradient where a step takes one, two or
four tokens: every number of choices and pitch, token counts that no step
divides, dropped assignments, non-finite rows and weights behind them, against
64 bits; and a token's results do not depend on the batch around it.

Tolerances: a value rounded to type t is off by at most eps(t) / 2 of it; a
sum of fp32 terms by 2^-24 of the terms' magnitudes for every addition one of
them goes through."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U32 = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def sq():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import w8a8_int8_gemm_calib_b200 as m

    return m


def _piece(N, dtype):
    """A thread's columns at once: 16 bytes, or four pieces of what the pitch
    keeps aligned."""
    size = 2 if dtype is BF else 4
    if N * size % 16 == 0:
        return 16 // size
    return 4 * (4 if N * size % 4 == 0 else 2) // size


def _threads(N, dtype):
    n = -(-N // _piece(N, dtype))
    return 256 if n >= 256 else -(-n // 32) * 32


def _tokens_a_step(T, k, N, dtype, grad):
    """The library's choice, so that a shape here that no longer reaches its
    variant is noticed."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    nt = _threads(N, dtype)
    segs = 1 if grad else -(-(-(-N // _piece(N, dtype))) // nt)

    def plan(p):
        resident = (4 if p == 1 else 3) * sms * (256 // nt)
        return resident, -(-T // p), -(-resident // segs)

    resident, steps, _ = plan(4)
    if k <= 2 and 2 * steps * segs >= resident:
        return 4
    if k <= 4:
        rounds = {p: -(-plan(p)[1] // plan(p)[2]) for p in (1, 2)}
        if rounds[2] < rounds[1] and (not grad or k < 4 or rounds[2] == 1):
            return 2
    return 1


def _half(t):
    return torch.finfo(t).eps / 2


class _Case:
    def __init__(self, T, k, N, dtype, seed):
        r = np.random.default_rng(seed)
        self.T, self.k, self.N, self.dtype = T, k, N, dtype
        R = self.R = T * k + 3
        pos = r.permutation(R)[:T * k].reshape(T, k)
        gone = r.random((T, k)) < 0.2
        pos[gone] = r.choice([-1, R, -5, 2 ** 31 - 1], gone.sum())
        pos[T // 2] = -1  # tokens of none, the last one too
        pos[T - 1] = -1
        pos[T - 2, 0] = R  # beyond the rows
        self.live = torch.from_numpy((pos >= 0) & (pos < R)).cuda()
        self.pos = torch.from_numpy(pos.astype(np.int32)).cuda()
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.z = torch.randn(R, N, device="cuda", generator=g).to(dtype)
        used = torch.zeros(R, dtype=torch.bool, device="cuda")
        used[self.pos[self.live].long()] = True
        self.unused = ~used
        self.z[self.unused] = float("nan")  # rows of no assignment
        self.w = torch.rand(T, k, device="cuda", generator=g)
        self.w[~self.live] = float("inf")  # weights of none
        self.res = torch.randn(T, N, device="cuda", generator=g).to(dtype)
        self.dy = torch.randn(T, N, device="cuda", generator=g).to(dtype)

    def of(self, c):
        """Tokens with a live choice c, and their rows."""
        t = torch.nonzero(self.live[:, c])[:, 0]
        return t, self.pos[t, c].long()


# T, k, N and the tokens a step of the combine and of its gradient, on 148 SMs
SHAPES = [
    (1031, 1, 4096, BF, 4, 4), (1031, 2, 4096, BF, 4, 4), (770, 1, 4096, BF, 4, 2),
    (770, 2, 4096, BF, 4, 2), (770, 3, 4096, BF, 2, 2), (770, 4, 4096, BF, 2, 2),
    (2051, 3, 4096, BF, 2, 2), (2051, 4, 4096, BF, 2, 1),
    (1031, 1, 4094, BF, 4, 4), (1031, 2, 4094, BF, 4, 4), (770, 3, 4094, BF, 2, 2),
    (770, 4, 4094, BF, 2, 2),
    (1031, 1, 4095, BF, 4, 4), (1031, 2, 4095, BF, 4, 4), (770, 3, 4095, BF, 2, 2),
    (770, 4, 4095, BF, 2, 2),
    (1031, 1, 4096, F32, 4, 4), (1031, 2, 4096, F32, 4, 4), (770, 3, 4096, F32, 2, 2),
    (770, 4, 4096, F32, 2, 2),
    (1031, 1, 4095, F32, 4, 4), (1031, 2, 4095, F32, 4, 4), (770, 3, 4095, F32, 2, 2),
    (770, 4, 4095, F32, 2, 2),
    # narrow rows: one warp a block, the last pieces of it idle
    (7105, 1, 40, BF, 4, 4), (7106, 2, 42, BF, 4, 4), (7107, 2, 41, BF, 4, 4), (4739, 3, 41, BF, 2, 2),
    (4741, 4, 40, BF, 2, 2), (4739, 4, 42, BF, 2, 2), (7107, 2, 37, F32, 4, 4), (4739, 3, 36, F32, 2, 2),
    (7105, 1, 1, BF, 4, 4), (4739, 3, 1, F32, 2, 2),
    # one token a step next to them
    (511, 4, 4096, BF, 1, 1), (513, 2, 4096, BF, 4, 1), (1029, 4, 4095, BF, 2, 1),
]


def _id(v):
    return {BF: "bf16", F32: "f32"}.get(v, str(v))


@pytest.mark.parametrize("T,k,N,dtype,p_combine,p_grad", SHAPES, ids=_id)
@pytest.mark.parametrize("weighted", [True, False])
def test_combine_steps(sq, T, k, N, dtype, p_combine, p_grad, weighted):
    assert _tokens_a_step(T, k, N, dtype, False) == p_combine
    c = _Case(T, k, N, dtype, T + k + N)
    w = c.w if weighted else None
    res = c.res if weighted else None  # with neither: the gather's gradient
    out = torch.full((T + 1, N), 9.0, device="cuda").to(dtype)
    sq.sq_moe_combine(c.z, c.pos, out[:T], weights=w, residual=res)
    sq.sq_sync_status()
    y = out[:T]
    assert bool((out[T] == 9).all())  # behind the last token
    want = c.res.double() if weighted else torch.zeros(T, N, dtype=torch.float64, device="cuda")
    mag = want.abs()
    for j in range(k):
        t, rows = c.of(j)
        term = c.z[rows].double() * (c.w[t, j, None].double() if weighted else 1.0)
        want[t] += term
        mag[t] += term.abs()
    bound = _half(dtype) * want.abs() + (1 + _half(dtype)) * k * U32 * mag
    assert bool(((y.double() - want).abs() <= bound).all())
    # the first tokens by themselves, one token a step: the same bits
    few = 37
    assert _tokens_a_step(few, k, N, dtype, False) == 1
    alone = torch.empty(few, N, dtype=dtype, device="cuda")
    sq.sq_moe_combine(c.z, c.pos[:few], alone, weights=None if w is None else w[:few],
                      residual=None if res is None else res[:few])
    assert torch.equal(alone, y[:few])
    if weighted:  # over the residual itself
        sq.sq_moe_combine(c.z, c.pos, c.res, weights=w, residual=c.res)
        assert torch.equal(c.res, y)
    sq.sq_sync_status()


@pytest.mark.parametrize("T,k,N,dtype,p_combine,p_grad", SHAPES, ids=_id)
@pytest.mark.parametrize("weighted", [True, False])
def test_combine_grad_steps(sq, T, k, N, dtype, p_combine, p_grad, weighted):
    assert _tokens_a_step(T, k, N, dtype, True) == p_grad
    c = _Case(T, k, N, dtype, T + k + N + 1)
    w = c.w if weighted else None
    dz = torch.full((c.R, N), 9.0, device="cuda").to(dtype)
    dw = torch.full((T + 1, k), 9.0, device="cuda")
    sq.sq_moe_combine_grad(c.dy, c.pos, z=c.z, weights=w, dz=dz, dweights=dw[:T])
    sq.sq_sync_status()
    assert bool((dw[T] == 9).all()) and bool((dz[c.unused] == 9).all())
    # a thread's chain of columns, 5 levels of lanes, up to 8 warps
    e = _piece(N, dtype)
    adds = e * -(-N // (e * _threads(N, dtype))) + 5 + 8
    assert bool((dw[:T][~c.live] == 0).all())
    for j in range(k):
        t, rows = c.of(j)
        want = c.dy[t].double() * (c.w[t, j, None].double() if weighted else 1.0)
        bound = want.abs() * ((1 + _half(dtype)) * (1 + U32) - 1)
        assert bool(((dz[rows].double() - want).abs() <= bound).all())
        prod = c.dy[t].double() * c.z[rows].double()
        err = (dw[t, j].double() - prod.sum(1)).abs()
        assert bool((err <= adds * U32 * prod.abs().sum(1) * 1.001).all())
    # each output alone, and the first tokens by themselves: the same bits
    dz2, dw2 = torch.full_like(dz, 9.0), torch.full((T, k), 9.0, device="cuda")
    sq.sq_moe_combine_grad(c.dy, c.pos, weights=w, dz=dz2)
    sq.sq_moe_combine_grad(c.dy, c.pos, z=c.z, weights=w, dweights=dw2)
    assert torch.equal(dz2, dz) and torch.equal(dw2, dw[:T])
    few = 37
    assert _tokens_a_step(few, k, N, dtype, True) == 1
    dz3, dw3 = torch.full_like(dz, 9.0), torch.full((few, k), 9.0, device="cuda")
    sq.sq_moe_combine_grad(c.dy[:few], c.pos[:few], z=c.z, weights=None if w is None else w[:few],
                           dz=dz3, dweights=dw3)
    mine = c.pos[:few][c.live[:few]].long()
    assert torch.equal(dw3, dw[:few]) and torch.equal(dz3[mine], dz[mine])
    sq.sq_sync_status()


@pytest.mark.parametrize("T,k", [(770, 4), (1031, 2)])
def test_steps_captured_and_on_another_stream(sq, T, k):
    """Replayed from a CUDA graph on another stream after the inputs changed
    in place: the bits of the eager call."""
    c = _Case(T, k, 4096, BF, 3)
    dz, dw = torch.full((c.R, 4096), 9.0, device="cuda").to(BF), torch.empty(T, k, device="cuda")
    y = torch.empty(T, 4096, dtype=BF, device="cuda")

    def run():
        sq.sq_moe_combine(c.z, c.pos, y, weights=c.w, residual=c.res)
        sq.sq_moe_combine_grad(c.dy, c.pos, z=c.z, weights=c.w, dz=dz, dweights=dw)

    run()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        run()
    c.dy.mul_(-0.5)
    c.res.copy_(c.res.flip(0))
    c.pos.copy_(c.pos.flip(0))
    c.w.copy_(c.w.flip(0))
    run()
    want = [t.clone() for t in (y, dz, dw)]
    for t in (y, dw):
        t.fill_(7)
    dz.fill_(9)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph.replay()
    torch.cuda.synchronize()
    sq.sq_sync_status()
    assert torch.equal(y, want[0]) and torch.equal(dz, want[1]) and torch.equal(dw, want[2])
