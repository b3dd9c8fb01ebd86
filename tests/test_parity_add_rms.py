"""GPU parity of the residual addition + RMSNorm quantizer: h against the
rounded sum, codes, steps and clip counts against the oracle's RMSNorm
quantizer on that h, bit for bit, and the codes' values against 64 bits."""
import numpy as np
import pytest

import synth
from tests._util import assert_bits_equal, dev, host

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def sq():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import w8a8_int8_gemm_calib_b200 as m

    return m


def _inputs(seed, T, K, dtype):
    x = synth.activations(seed, f"add{T}x{K}", T, K, synth.outlier_pattern(seed, K, 0.01))
    r = synth.activations(seed + 1, f"res{T}x{K}", T, K, synth.outlier_pattern(seed + 1, K, 0.01))
    if dtype == "bf16":
        x, r = synth.bf16_bits(x), synth.bf16_bits(r)
    g = (synth.ln_params(seed, f"addg{K}", K)[0]
         / np.random.default_rng(K).uniform(0.2, 4.0, K)).astype(np.float32)
    return x, r, g


def _sum(x, r):
    """h on the host: one fp32 addition, then bf16 (nearest even) for bf16."""
    if x.dtype == np.uint16:
        return synth.bf16_bits(synth.bf16_bits_to_f32(x) + synth.bf16_bits_to_f32(r))
    return x + r


def _run(sq, x, r, g, gran, delta=0.02, eps=1e-5, h=None):
    T, K = x.shape
    xd, rd = dev(x), dev(r)
    h = torch.empty_like(xd) if h is None else {"x": xd, "r": rd}[h]
    xq = torch.full((T, K), 99, dtype=torch.int8, device="cuda")
    act = torch.full((T if gran == "token" else 1,), delta, device="cuda")
    ncl = torch.zeros(1, dtype=torch.int64, device="cuda")
    sq.sq_add_rms_smooth_quant_act(xd, rd, h, xq, act, dev(g), eps=eps, per_token=gran == "token",
                                   n_clipped=ncl, per_tensor_dynamic=gran == "tensor")
    sq.sq_sync_status()
    return host(h), host(xq), host(act), int(ncl)


# every register variant (up to 2, 4, 8, 16 chunks of a thread), its edges,
# the widths beyond, and row counts around the grid
SHAPES = [(1, 16), (5, 48), (33, 1040), (3, 2048), (7, 2064), (130, 4096), (64, 5120), (9, 8192),
          (5, 8208), (12, 12288), (3, 16400), (3, 20480), (2, 53248), (1, 133136), (2400, 256),
          (593, 1024)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("gran", ["token", "static", "tensor"])
@pytest.mark.parametrize("T,K", SHAPES)
def test_add_rms(sq, orc, dtype, gran, T, K):
    x, r, g = _inputs(T + 3 * K, T, K, dtype)
    want_h = _sum(x, r)
    want_q, want_act, want_clip = orc.quant_act_rms(
        want_h, g, per_token=gran == "token", per_tensor_dynamic=gran == "tensor",
        static_delta=np.float32(0.02))
    h, xq, act, clip = _run(sq, x, r, g, gran)
    assert_bits_equal(h, want_h, "h")
    assert_bits_equal(xq, want_q, "xq")
    assert_bits_equal(act, want_act, "act_scale")
    assert clip == want_clip


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("gran", ["token", "static", "tensor"])
@pytest.mark.parametrize("into", ["x", "r"])
def test_add_rms_in_place(sq, dtype, gran, into):
    """h written over x or over the residual: the same outputs."""
    x, r, g = _inputs(11, 700, 4096, dtype)
    a, b = _run(sq, x, r, g, gran), _run(sq, x, r, g, gran, h=into)
    for u, v, what in zip(a, b, ("h", "xq", "act")):
        assert_bits_equal(np.asarray(v), np.asarray(u), what)
    assert a[3] == b[3]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("gran", ["token", "static", "tensor"])
@pytest.mark.parametrize("K", [64, 4096, 20480])
def test_add_rms_special_values(sq, orc, dtype, gran, K):
    """Rows of zeros, with an infinity, with a NaN, of nothing else, with
    opposite infinities (their sum is NaN), of the type's largest values
    (the sum overflows) and of tiny ones: as the oracle on the same h."""
    T = 8
    x, r, g = _inputs(5, T, K, "f32")
    big = np.float32(3.3895314e38)  # bf16's largest
    x[0] = r[0] = 0
    x[1, 3] = np.inf
    x[2, 5] = np.nan
    x[3] = np.nan
    x[4, 1], r[4, 1] = np.inf, -np.inf
    x[5, 7] = r[5, 7] = big
    x[6] = r[6] = np.float32(1e-38)
    if dtype == "bf16":
        def bits(a):
            return host(torch.from_numpy(a).to(torch.bfloat16))
        x, r = bits(x), bits(r)
        want_h = host((torch.from_numpy(x.view(np.int16)).view(torch.bfloat16).float()
                       + torch.from_numpy(r.view(np.int16)).view(torch.bfloat16).float())
                      .to(torch.bfloat16))
    else:
        with np.errstate(all="ignore"):
            want_h = x + r
    want_q, want_act, want_clip = orc.quant_act_rms(
        want_h, g, per_token=gran == "token", per_tensor_dynamic=gran == "tensor",
        static_delta=np.float32(0.02))
    h, xq, act, clip = _run(sq, x, r, g, gran)
    hv, wv = (synth.bf16_bits_to_f32(h), synth.bf16_bits_to_f32(want_h)) if dtype == "bf16" else (h, want_h)
    np.testing.assert_array_equal(hv, wv)  # NaN equals NaN here
    assert_bits_equal(xq, want_q, "xq")
    np.testing.assert_array_equal(act, want_act)
    assert clip == want_clip


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_add_rms_against_64_bits(sq, dtype):
    """A code stands for a value within half a step of the exact y, plus y's
    own rounding: the mean of K squares is summed by 128 slots of K/128
    fused steps and 7 levels, so rstd is off by at most (K/128 + 7 + 4) / 2
    + 2 half-ulps relative (the square root halves the sum's), y by two more,
    and y / step by three more."""
    T, K = 64, 4096
    x, r, g = _inputs(21, T, K, dtype)
    h, xq, act, _ = _run(sq, x, r, g, "token")
    h64 = (synth.bf16_bits_to_f32(h) if dtype == "bf16" else h).astype(np.float64)
    y = h64 / np.sqrt((h64 ** 2).mean(1, keepdims=True) + np.float32(1e-5)) * g
    step = act.astype(np.float64)[:, None]
    rel = ((K / 128 + 11) / 2 + 7) * 2.0 ** -24
    assert (np.abs(xq * step - y) <= step / 2 + np.abs(y) * rel).all()
    peak = np.abs(y).max(1)
    assert (np.abs(act * 127.0 - peak) <= peak * rel).all()


def test_add_rms_equals_the_two_calls(sq):
    """At the large prefill's width: the same bits as the addition and
    sq_rms_smooth_quant_act of its result, every row."""
    T, K = 4099, 8192
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(T, K, device="cuda", generator=gen).bfloat16()
    r = (torch.randn(T, K, device="cuda", generator=gen) * 3).bfloat16()
    g = torch.rand(K, device="cuda", generator=gen) + 0.5
    for kw in (dict(), dict(per_token=False), dict(per_tensor_dynamic=True)):
        n = T if not kw else 1
        a1, a2 = torch.full((n,), 0.03, device="cuda"), torch.full((n,), 0.03, device="cuda")
        h = torch.empty_like(x)
        q1 = torch.empty(T, K, dtype=torch.int8, device="cuda")
        q2 = torch.empty_like(q1)
        sq.sq_add_rms_smooth_quant_act(x, r, h, q1, a1, g, **kw)
        want = x + r
        sq.sq_rms_smooth_quant_act(want, q2, a2, g, **kw)
        sq.sq_sync_status()
        assert torch.equal(h.view(torch.int16), want.view(torch.int16))
        assert torch.equal(q1, q2) and torch.equal(a1, a2)
