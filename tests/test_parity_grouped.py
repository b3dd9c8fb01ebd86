"""GPU parity of the grouped INT8 GEMM (one weight matrix per group of rows,
the groups given on the device): accumulators exactly and outputs bit for bit
against integers and the epilogue's separately rounded fp32 steps, and the
whole routed block."""
import numpy as np
import pytest

from tests._util import assert_bits_equal, dev, host

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def sq():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import w8a8_int8_gemm_calib_b200 as m

    return m


def _operands(R, N, K, E, seed, per_token=True, bias=True):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def ints(*s):
        return torch.randint(-127, 128, s, dtype=torch.int8, device="cuda", generator=g)

    def rand(*s, lo, hi):
        return torch.rand(*s, device="cuda", generator=g) * (hi - lo) + lo

    return (ints(R, K), ints(E, N, K), rand(R if per_token else 1, lo=1e-3, hi=0.1),
            rand(E, N, lo=1e-4, hi=1e-2), rand(E, N, lo=-1, hi=1) if bias else None)


def _want(xq, wq, off, act, ws, bias, out, y0, acc0):
    """acc in fp64 (exact integers), then one fp32 rounding per operation."""
    y, acc = y0.clone(), acc0.clone()
    for e in range(wq.shape[0]):
        a, b = off[e], off[e + 1]
        if b <= a:
            continue
        acc[a:b] = (xq[a:b].double() @ wq[e].double().t()).to(torch.int32)
        v = acc[a:b].float() * ((act[a:b, None] if act.numel() > 1 else act) * ws[e])
        if bias is not None:
            v = v + bias[e]
        y[a:b] = v.to(out)
    return y, acc


def _check(sq, counts, N, K, out, seed=0, per_token=True, bias=True, first=0, spare=0):
    E, R = len(counts), first + sum(counts) + spare
    off = [first] + list(first + np.cumsum(counts))
    xq, wq, act, ws, b = _operands(R, N, K, E, seed, per_token, bias)
    y = torch.full((R, N), 77.0, device="cuda").to(out)
    acc = torch.full((R, N), -5, dtype=torch.int32, device="cuda")
    want_y, want_acc = _want(xq, wq, off, act, ws, b, out, y, acc)
    sq.sq_gemm_w8a8_grouped(xq, wq, torch.tensor(off, dtype=torch.int32, device="cuda"), act, ws, y,
                            per_token=per_token, bias=b, acc_out=acc)
    sq.sq_sync_status()
    assert torch.equal(acc, want_acc)
    view = torch.int16 if out == torch.bfloat16 else torch.int32
    assert torch.equal(y.view(view), want_y.view(view))


OUT = [torch.bfloat16, torch.float32]
GROUPS = [
    [1], [0, 1], [1, 0, 0, 2], [127, 128, 129], [5, 0, 300, 1, 64, 33], [0, 0, 0], [1000], [7] * 9,
    [1] * 40, [16, 17, 31, 32, 33, 63, 64, 65, 8, 9], [260, 0, 511, 513], [3] + [0] * 62 + [200], [4700, 3],
]


@pytest.mark.parametrize("counts", GROUPS, ids=lambda c: "-".join(map(str, c[:6])) + f"x{len(c)}")
@pytest.mark.parametrize("N,K", [(256, 128), (17, 48), (1000, 2064), (520, 16), (264, 640), (1, 32), (602, 272)])
@pytest.mark.parametrize("out", OUT, ids=["bf16", "f32"])
def test_grouped(sq, counts, N, K, out):
    _check(sq, counts, N, K, out, seed=sum(counts) + N + K)


@pytest.mark.parametrize("per_token", [True, False])
@pytest.mark.parametrize("bias", [True, False])
@pytest.mark.parametrize("counts", [[3, 0, 5], [40, 170, 90], [700, 900]])
def test_grouped_scales_and_bias(sq, per_token, bias, counts):
    _check(sq, counts, 300, 528, torch.float32, per_token=per_token, bias=bias)


@pytest.mark.parametrize("counts", [[1, 2], [100, 0, 150], [600, 900]])
@pytest.mark.parametrize("N", [255, 256])
@pytest.mark.parametrize("out", OUT, ids=["bf16", "f32"])
def test_rows_of_no_expert_keep_what_they_held(sq, counts, N, out):
    _check(sq, counts, N, 256, out, first=37, spare=203)


def test_many_experts(sq):
    r = np.random.default_rng(1)
    _check(sq, r.integers(0, 4, 1024).tolist(), 130, 144, torch.bfloat16)
    _check(sq, r.integers(0, 200, 300).tolist(), 130, 144, torch.float32)


def test_extreme_codes_and_the_widest_k(sq):
    """The largest accumulators: 127 * 127 * 133136 stays below 2^31."""
    K, N = 133136, 130
    xq = torch.full((5, K), 127, dtype=torch.int8, device="cuda")
    wq = torch.full((2, N, K), 127, dtype=torch.int8, device="cuda")
    wq[1] = -127
    off = torch.tensor([0, 2, 5], dtype=torch.int32, device="cuda")
    acc = torch.empty(5, N, dtype=torch.int32, device="cuda")
    y = torch.empty(5, N, device="cuda")
    sq.sq_gemm_w8a8_grouped(xq, wq, off, torch.ones(1, device="cuda"), torch.ones(2, N, device="cuda"),
                            y, per_token=False, acc_out=acc)
    sq.sq_sync_status()
    top = 127 * 127 * K
    assert bool((acc[:2] == top).all()) and bool((acc[2:] == -top).all())
    assert torch.equal(y, acc.float())


@pytest.mark.parametrize("rows", [24, 3000])
def test_bad_offsets_stay_inside(sq, rows):
    """Offsets that fall or leave [0, R] are clamped to a rising sequence:
    the documented result, and nothing outside the arrays."""
    N, K, E = 144, 144, 6
    xq, wq, act, ws, _ = _operands(rows + 8, N, K, E, 3, bias=False)
    bad = [-5, rows // 3, rows // 4, 1 << 30, 7, -(1 << 30), rows]
    rise, top = [], 0
    for v in bad:
        top = max(top, min(max(v, 0), rows))
        rise.append(top)
    y = torch.full((rows + 8, N), 3.0, device="cuda")
    acc = torch.full((rows + 8, N), -5, dtype=torch.int32, device="cuda")
    want, _ = _want(xq, wq, rise, act, ws, None, torch.float32, y, acc)
    sq.sq_gemm_w8a8_grouped(xq[:rows], wq, torch.tensor(bad, dtype=torch.int32, device="cuda"),
                            act[:rows], ws, y[:rows])
    sq.sq_sync_status()
    assert torch.equal(y, want)


@pytest.mark.parametrize("R,E", [(16, 8), (512, 64), (4096, 8)])
def test_against_the_plain_gemm(sq, orc, R, E):
    """Each group equals sq_gemm_w8a8 on its rows, and the oracle on a few."""
    N, K = 1040, 1040
    xq, wq, act, ws, b = _operands(R, N, K, E, R)
    cut = np.sort(np.random.default_rng(R).integers(0, R + 1, E - 1))
    off = [0, *cut.tolist(), R]
    y = torch.empty(R, N, dtype=torch.bfloat16, device="cuda")
    sq.sq_gemm_w8a8_grouped(xq, wq, torch.tensor(off, dtype=torch.int32, device="cuda"), act, ws, y,
                            bias=b)
    work = sq.Workspace()
    for e in range(E):
        a, z = off[e], off[e + 1]
        if z > a:
            one = torch.empty(z - a, N, dtype=torch.bfloat16, device="cuda")
            x, s = xq[a:z].clone(), act[a:z].clone()
            sq.sq_gemm_w8a8(x, wq[e].clone(), s, ws[e].clone(), one, bias=b[e].clone(), workspace=work)
            sq.sq_sync_status()
            assert torch.equal(y[a:z].view(torch.int16), one.view(torch.int16)), e
    e = int(np.argmax(np.diff(off)))
    a = off[e]
    o_y, _ = orc.gemm_w8a8(host(xq[a:a + 2]), host(wq[e]), host(act[a:a + 2]), host(ws[e]),
                           out_bf16=True, bias=host(b[e]))
    assert_bits_equal(host(y[a:a + 2]), o_y, "y")


def test_weights_past_32_bits(sq):
    """[E, N, K] of more than 2^31 elements: the last expert's weights."""
    E, N, K = 20, 8192, 16384
    wq = torch.zeros(E, N, K, dtype=torch.int8, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(4)
    wq[E - 1, N - 130:] = torch.randint(-127, 128, (130, K), dtype=torch.int8, device="cuda", generator=g)
    for R in (3, 2000):
        xq = torch.randint(-127, 128, (R, K), dtype=torch.int8, device="cuda", generator=g)
        off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        off[E] = R
        y = torch.empty(R, N, device="cuda")
        acc = torch.empty(R, N, dtype=torch.int32, device="cuda")
        sq.sq_gemm_w8a8_grouped(xq, wq, off, torch.ones(R, device="cuda"),
                                torch.ones(E, N, device="cuda"), y, acc_out=acc)
        sq.sq_sync_status()
        assert torch.equal(acc[:, N - 130:], (xq.double() @ wq[E - 1, N - 130:].double().t()).int())
        assert not bool(acc[:, :N - 130].any()) and torch.equal(y, acc.float())


# ------------------------------------------------------------------ the block
class _Block:
    """One pre-norm block of routed W8A8 experts and its buffers."""

    def __init__(self, sq, T, K, N, E, k, seed=0):
        self.sq, self.k, self.E = sq, k, E
        g = torch.Generator(device="cuda").manual_seed(seed)

        def randn(*s, std=1.0):
            return torch.randn(*s, device="cuda", generator=g) * std

        def empty(*s, dtype=torch.float32):
            return torch.empty(*s, dtype=dtype, device="cuda")

        self.x, self.res = randn(T, K).bfloat16(), randn(T, K).bfloat16()
        self.gamma = 1 + randn(K, std=0.1)
        self.ids = torch.randn(T, E, device="cuda", generator=g).topk(k, 1).indices
        if T > 3:
            self.ids[3] = -1  # a padding token
        self.wts = torch.softmax(randn(T, k), 1)
        self.up, self.ups = empty(E, 2 * N, K, dtype=torch.int8), empty(E, 2 * N)
        self.dn, self.dns = empty(E, K, N, dtype=torch.int8), empty(E, K)
        one = torch.ones(max(K, N), device="cuda")
        for e in range(E):
            sq.sq_fuse_weights_q8(randn(2 * N, K, std=0.05), one[:K], self.up[e], self.ups[e])
            sq.sq_fuse_weights_q8(randn(K, N, std=0.05), one[:N], self.dn[e], self.dns[e])
        R = T * k
        self.h, self.y = empty(T, K, dtype=torch.bfloat16), empty(T, K, dtype=torch.bfloat16)
        self.xq, self.act = empty(T, K, dtype=torch.int8), empty(T)
        self.off, self.pos = empty(E + 1, dtype=torch.int32), empty(T, k, dtype=torch.int32)
        self.xs, self.acts = torch.zeros(R, K, dtype=torch.int8, device="cuda"), torch.zeros(R, device="cuda")
        self.u = torch.zeros(R, 2 * N, dtype=torch.bfloat16, device="cuda")
        self.uq, self.ua = empty(R, N, dtype=torch.int8), empty(R)
        self.z = torch.zeros(R, K, dtype=torch.bfloat16, device="cuda")
        self.work = sq.Workspace()
        self.work.get(sq.sq_moe_sort_workspace_bytes(T, k, E))

    def run(self):
        sq = self.sq
        sq.sq_add_rms_smooth_quant_act(self.x, self.res, self.h, self.xq, self.act, self.gamma)
        sq.sq_moe_sort(self.ids, self.E, self.off, self.pos, workspace=self.work)
        sq.sq_moe_gather(self.xq, self.pos, self.xs, scale=self.act, scale_s=self.acts)
        sq.sq_gemm_w8a8_grouped(self.xs, self.up, self.off, self.acts, self.ups, self.u)
        gate, up = self.u.float().chunk(2, 1)
        self.a = (torch.nn.functional.silu(gate) * up).bfloat16()
        sq.sq_ln_smooth_quant_act(self.a, self.uq, self.ua)
        sq.sq_gemm_w8a8_grouped(self.uq, self.dn, self.off, self.ua, self.dns, self.z)
        sq.sq_moe_combine(self.z, self.pos, self.y, weights=self.wts, residual=self.h)
        return self.y


@pytest.mark.parametrize("T,k,E", [(1, 2, 8), (16, 8, 64), (300, 2, 8), (2100, 4, 16)])
def test_routed_block(sq, T, k, E):
    """add + norm + quantize -> sort, gather -> experts -> activation and
    quantizer -> experts -> combine, every token against its own experts in
    64 bits from the same codes."""
    K, N = 512, 384
    b = _Block(sq, T, K, N, E, k, seed=T)
    y = b.run()
    sq.sq_sync_status()
    half = 2.0 ** -8
    for t in sorted({0, min(3, T - 1), T // 2, T - 1}):
        want = b.h[t].double()
        mag = want.abs()
        for c in range(k):
            e = int(b.ids[t, c])
            p = int(b.pos[t, c])
            if e < 0:
                assert p == -1
                continue
            u = (b.up[e].double() @ b.xq[t].double()) * b.act[t].double() * b.ups[e].double()
            # three fp32 roundings and the one to bf16
            assert bool(((b.u[p].double() - u).abs() <= u.abs() * (half + 4 * 2.0 ** -24)).all())
            z = (b.dn[e].double() @ b.uq[p].double()) * b.ua[p].double() * b.dns[e].double()
            assert bool(((b.z[p].double() - z).abs() <= z.abs() * (half + 4 * 2.0 ** -24)).all())
            term = b.wts[t, c].double() * b.z[p].double()
            want, mag = want + term, mag + term.abs()
        bound = half * want.abs() + (1 + half) * k * 2.0 ** -24 * mag
        assert bool(((y[t].double() - want).abs() <= bound).all()), t


@pytest.mark.parametrize("T", [5, 700, 2100])
def test_routed_block_captured_and_on_another_stream(sq, T):
    """The block on a side stream, and replayed from a CUDA graph after its
    inputs changed in place: the same bits as the eager call."""
    b = _Block(sq, T, 256, 128, 8, 2)
    b.run()
    sq.sq_sync_status()
    first = b.y.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b.y.zero_()
        b.run()
        sq.sq_sync_status()
    assert torch.equal(b.y, first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.run()
    b.x.mul_(-0.5)
    b.ids.copy_(b.ids.flip(0))
    graph.replay()
    sq.sq_sync_status()
    replayed = b.y.clone()
    b.y.zero_()
    b.run()
    sq.sq_sync_status()
    assert torch.equal(b.y, replayed) and not torch.equal(first, replayed)


def test_no_tokens(sq):
    """An empty batch through every call: nothing is written but offsets."""
    K, N, E, k = 256, 128, 8, 2

    def empty(*s, dtype=torch.bfloat16):
        return torch.empty(*s, dtype=dtype, device="cuda")

    x, act = empty(0, K), empty(0, dtype=torch.float32)
    xq, pos = empty(0, K, dtype=torch.int8), empty(0, k, dtype=torch.int32)
    off = torch.full((E + 1,), 5, dtype=torch.int32, device="cuda")
    for kw in (dict(), dict(per_token=False), dict(per_tensor_dynamic=True)):
        step = torch.full((1,), 0.5, device="cuda") if kw else act
        sq.sq_add_rms_smooth_quant_act(x, x, x, xq, step, torch.ones(K, device="cuda"), **kw)
        assert not kw or float(step) == 0.5
    sq.sq_moe_sort(empty(0, k, dtype=torch.int64), E, off, pos)
    sq.sq_moe_gather(xq, pos, xq, scale=act, scale_s=act)
    sq.sq_gemm_w8a8_grouped(xq, torch.ones(E, N, K, dtype=torch.int8, device="cuda"), off, act,
                            torch.ones(E, N, device="cuda"), empty(0, N))
    z = empty(0, N)
    sq.sq_moe_combine(z, pos, z)
    sq.sq_moe_combine_grad(z, pos, z=z, dz=z, dweights=empty(0, k, dtype=torch.float32))
    sq.sq_sync_status()
    assert off.tolist() == [0] * (E + 1)


def test_two_blocks_at_once(sq):
    """Two calls on two streams, each with its own workspace."""
    blocks = [_Block(sq, T, 256, 128, 16, 2, seed=T) for T in (9, 600)]
    want = [b.run().clone() for b in blocks]
    sq.sq_sync_status()
    streams = [torch.cuda.Stream() for _ in blocks]
    for _ in range(5):
        for b, s in zip(blocks, streams):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                b.y.zero_()
                b.run()
    torch.cuda.synchronize()
    sq.sq_sync_status()
    for b, w in zip(blocks, want):
        assert torch.equal(b.y, w)
