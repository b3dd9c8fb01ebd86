"""The routed-expert operators and the residual norm quantizer, as cases to measure.

A case is one call (or the calls that always go together) of a smoothed W8A8
layer whose linears are experts chosen per token:

* ``norm``     h = x + residual, RMSNorm(h; gamma / s), INT8 codes and steps;
* ``dispatch`` the routed assignments sorted by expert, and the tokens' codes
               and steps copied to their sorted rows;
* ``experts``  the INT8 product of every expert's rows with its weights;
* ``combine``  the experts' rows back to their tokens, weighted and added;
* ``grad``     the gradients of ``combine`` (rows and routing weights) and of
               the copies that ``dispatch`` makes.

``run`` computes a case in elementary torch operations, or, with ``own``, by
this package's entry points.  ``exact`` computes it in 64 bits.
"""
import math

import torch

own = False

EPS = 1e-5
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decoded token behind an OPT-6.7B-wide block: latency
        dict(name="norm 1x4096 token", kind="norm", T=1, K=4096, dtype="bf16", gran="token"),
        # the OPT-6.7B prompt of 2048 tokens
        dict(name="norm 2048x4096 token", kind="norm", T=2048, K=4096, dtype="bf16", gran="token"),
        # the large prefill (16384 x 8192), calibrated static step
        dict(name="norm 16384x8192 static", kind="norm", T=16384, K=8192, dtype="bf16",
             gran="static"),
        # a decode batch of 16 tokens, two of 8 experts each
        dict(name="dispatch 16 of 8x2", kind="dispatch", T=16, top_k=2, E=8, K=4096, dtype="i8",
             drop=0.0),
        # a prefill of 16384 tokens, eight of 64 experts each
        dict(name="dispatch 16384 of 64x8", kind="dispatch", T=16384, top_k=8, E=64, K=4096,
             dtype="i8", drop=0.0),
        # one decoded token: eight experts' weights stream past one row each
        dict(name="experts 1 of 64x8", kind="experts", T=1, top_k=8, E=64, N=4096, K=4096,
             dtype="bf16", drop=0.0, per_token=True, bias=False),
        # a decode batch of 64 tokens over all 64 experts, an odd output width
        dict(name="experts 64 of 64x8", kind="experts", T=64, top_k=8, E=64, N=4100, K=4096,
             dtype="bf16", drop=0.0, per_token=True, bias=False),
        # a prefill of 16384 tokens over 8 wide experts
        dict(name="experts 16384 of 8x2", kind="experts", T=16384, top_k=2, E=8, N=14336, K=4096,
             dtype="bf16", drop=0.0, per_token=True, bias=False),
        # a decode batch's outputs back to their tokens, added to the residual
        dict(name="combine 16x8", kind="combine", T=16, top_k=8, N=4096, dtype="bf16", drop=0.0,
             residual=True),
        # the prefill's outputs back to their tokens
        dict(name="combine 16384x8", kind="combine", T=16384, top_k=8, N=4096, dtype="bf16",
             drop=0.0, residual=True),
        # router tuning behind frozen experts: a small batch, then a large one
        dict(name="grad 512x2", kind="grad", T=512, top_k=2, N=4096, dtype="bf16", drop=0.0),
        dict(name="grad 8192x8", kind="grad", T=8192, top_k=8, N=4096, dtype="bf16", drop=0.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["norm", "dispatch", "experts", "combine", "grad"])
    drop = rng.choice([0.0, 0.0, 0.2])  # padding tokens among the batch
    if kind == "norm":
        K = 16 * _log(rng, 16, 768)
        T = _log(rng, 1, min(16384, (1 << 27) // K))
        return dict(kind=kind, T=T, K=K, dtype=rng.choice(["bf16", "bf16", "f32"]) if T * K <= 1 << 26 else "bf16",
                    gran=rng.choice(["token", "token", "static", "tensor"]))
    top_k = rng.choice([1, 2, 3, 4, 6, 8])
    if kind == "dispatch":
        K = 16 * _log(rng, 16, 512)
        T = _log(rng, 1, min(16384, (1 << 29) // (K * top_k)))
        return dict(kind=kind, T=T, top_k=top_k, E=rng.choice([8, 16, 60, 64, 128, 256]), K=K,
                    dtype=rng.choice(["i8", "i8", "i8", "bf16"]) if T * top_k * K <= 1 << 28 else "i8", drop=drop)
    if kind == "experts":
        E = rng.choice([8, 16, 60, 64, 128])
        top_k = min(top_k, E)
        K = 16 * _log(rng, 32, 256)
        N = _log(rng, 500, min(14336, (1 << 30) // (E * K)))
        T = _log(rng, 1, min(16384, int(3.8e12 / (2 * N * K * top_k)), (1 << 28) // (N * top_k)))
        return dict(kind=kind, T=T, top_k=top_k, E=E, N=N, K=K,
                    dtype=rng.choice(["bf16", "bf16", "f32"]), drop=drop,
                    per_token=rng.choice([True, True, False]), bias=rng.choice([False, True]))
    N = _log(rng, 250, 8192)
    T = _log(rng, 1, min(16384, (1 << (29 if kind == "combine" else 28)) // (N * top_k)))
    dtype = rng.choice(["bf16", "bf16", "f32"]) if T * top_k * N <= 1 << 27 else "bf16"
    c = dict(kind=kind, T=T, top_k=top_k, N=N, dtype=dtype, drop=drop)
    if kind == "combine":
        c["residual"] = rng.choice([True, False])
    return c


# ------------------------------------------------------------------ inputs
def _route(c, g, E):
    """Routed experts [T, top_k] int64 as torch.topk gives them (-1: padding)
    and their weights [T, top_k] fp32; some experts are more popular."""
    T, k = c["T"], c["top_k"]
    pull = torch.randn(E, device="cuda", generator=g) * 0.5
    logits = torch.randn(T, E, device="cuda", generator=g) + pull
    val, ids = logits.topk(k, dim=1)
    if c["drop"]:
        ids[torch.rand(T, device="cuda", generator=g) < c["drop"]] = -1
    return ids, val.softmax(1)


def _places(ids, E):
    """Offsets [E + 1] and sorted places [T, top_k] (-1: none), int32."""
    flat = ids.reshape(-1)
    key = torch.where(flat < 0, E, flat)
    order = torch.sort(key, stable=True).indices
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device=order.device)
    pos = torch.where(flat < 0, -1, place).reshape(ids.shape).int()
    counts = (key[:, None] == torch.arange(E, device=key.device)).sum(0)
    off = torch.zeros(E + 1, dtype=torch.int32, device=key.device)
    off[1:] = counts.cumsum(0)
    return off, pos


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(*shape, device="cuda", generator=g) * std).to(dtype)

    def codes(*shape):
        return (torch.randn(*shape, device="cuda", generator=g) * 32).round_().clamp_(-127, 127).to(torch.int8)

    def steps(*shape, at=0.01):
        return torch.exp(torch.randn(*shape, device="cuda", generator=g) * 0.3) * at

    s = dict(case=c)
    T = c["T"]
    if c["kind"] == "norm":
        K, dt = c["K"], DTYPES[c["dtype"]]
        out = 1 + 59 * (torch.rand(K, device="cuda", generator=g) < 0.01).float()  # outlier channels
        s["x"] = randn(T, K, std=0.5, dtype=dt)
        s["residual"] = (torch.randn(T, K, device="cuda", generator=g) * out).to(dt)
        s["gamma"] = (1 + randn(K, std=0.1)) / out.sqrt()  # gamma / s
        s["h"] = torch.empty(T, K, dtype=dt, device="cuda")
        s["xq"] = torch.empty(T, K, dtype=torch.int8, device="cuda")
        s["act"] = torch.empty(T if c["gran"] == "token" else 1, device="cuda")
        s["y"] = torch.empty(T, K, dtype=torch.bfloat16, device="cuda")
        if c["gran"] == "static":
            s["act"].fill_(0.03)
        return s
    if c["kind"] == "dispatch":
        K, R = c["K"], T * c["top_k"]
        s["ids"], _ = _route(c, g, c["E"])
        if c["dtype"] == "i8":
            s["x"], s["scale"], s["scale_s"] = codes(T, K), steps(T), torch.zeros(R, device="cuda")
        else:
            s["x"], s["scale"], s["scale_s"] = randn(T, K, dtype=DTYPES[c["dtype"]]), None, None
        s["xs"] = torch.zeros(R, K, dtype=s["x"].dtype, device="cuda")
        s["offsets"] = torch.empty(c["E"] + 1, dtype=torch.int32, device="cuda")
        s["pos"] = torch.empty(T, c["top_k"], dtype=torch.int32, device="cuda")
    elif c["kind"] == "experts":
        E, N, K, R = c["E"], c["N"], c["K"], T * c["top_k"]
        ids, _ = _route(c, g, E)
        s["offsets"], _ = _places(ids, E)
        s["most"] = int(s["offsets"].diff().max())  # the plain form pads to it
        s["xq"], s["wq"] = codes(R, K), codes(E, N, K)
        s["act"] = steps(R if c["per_token"] else 1)
        s["ws"] = steps(E, N, at=0.001)
        s["bias"] = randn(E, N, std=0.1) if c["bias"] else None
        s["y"] = torch.zeros(R, N, dtype=DTYPES[c["dtype"]], device="cuda")
    else:
        N, R, dt = c["N"], T * c["top_k"], DTYPES[c["dtype"]]
        ids, s["weights"] = _route(c, g, 64)
        _, s["pos"] = _places(ids, 64)
        s["z"] = randn(R, N, dtype=dt)
        if c["kind"] == "combine":
            s["residual"] = randn(T, N, dtype=dt) if c["residual"] else None
            s["y"] = torch.empty(T, N, dtype=dt, device="cuda")
        else:
            s["dy"], s["dxs"] = randn(T, N, dtype=dt), randn(R, N, dtype=dt)
            s["dz"] = torch.zeros(R, N, dtype=dt, device="cuda")
            s["dw"] = torch.empty(T, c["top_k"], device="cuda")
            s["dx"] = torch.empty(T, N, dtype=dt, device="cuda")
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    s, c = state, state["case"]
    if own:
        return _run_own(s, c)
    return {"norm": _norm, "dispatch": _dispatch, "experts": _experts, "combine": _combine,
            "grad": _grad}[c["kind"]](s, c)


def _run_own(s, c):
    import w8a8_int8_gemm_calib_b200 as sq

    if "workspace" not in s:
        s["workspace"] = sq.Workspace()  # kept between passes
    if c["kind"] == "norm":
        sq.sq_add_rms_smooth_quant_act(s["x"], s["residual"], s["h"], s["xq"], s["act"], s["gamma"],
                                       eps=EPS, per_token=c["gran"] == "token",
                                       per_tensor_dynamic=c["gran"] == "tensor")
        torch.mul(s["xq"], s["act"][:, None], out=s["y"])  # the codes' values
        return [s["h"], s["act"], s["y"]]
    if c["kind"] == "dispatch":
        sq.sq_moe_sort(s["ids"], c["E"], s["offsets"], s["pos"], workspace=s["workspace"])
        sq.sq_moe_gather(s["x"], s["pos"], s["xs"], scale=s["scale"], scale_s=s["scale_s"])
        return [s["offsets"], s["pos"], s["xs"], s["scale_s"]]
    if c["kind"] == "experts":
        sq.sq_gemm_w8a8_grouped(s["xq"], s["wq"], s["offsets"], s["act"], s["ws"], s["y"],
                                per_token=c["per_token"], bias=s["bias"])
        return s["y"]
    if c["kind"] == "combine":
        return sq.sq_moe_combine(s["z"], s["pos"], s["y"], weights=s["weights"],
                                 residual=s["residual"])
    sq.sq_moe_combine_grad(s["dy"], s["pos"], z=s["z"], weights=s["weights"], dz=s["dz"],
                           dweights=s["dw"])
    sq.sq_moe_combine(s["dxs"], s["pos"], s["dx"])
    return [s["dz"], s["dw"], s["dx"]]


def _norm(s, c):
    h = (s["x"].float() + s["residual"].float()).to(s["x"].dtype)
    hf = h.float()
    y = hf * torch.rsqrt(hf.square().mean(1, keepdim=True) + EPS) * s["gamma"]
    if c["gran"] == "static":
        act = s["act"]
    else:
        peak = y.abs().amax(1) if c["gran"] == "token" else y.abs().amax().reshape(1)
        act = peak.clamp(min=1e-7) / 127
    q = (y / act[:, None]).round().clamp(-127, 127)
    return [h, act, (q * act[:, None]).to(torch.bfloat16)]


def _dispatch(s, c):
    off, pos = _places(s["ids"], c["E"])
    R, k = s["xs"].shape[0], c["top_k"]
    to = torch.where(pos < 0, R, pos).long().reshape(-1)  # row R: assignments that go nowhere
    xs = torch.zeros(R + 1, c["K"], dtype=s["x"].dtype, device="cuda")
    xs[to] = s["x"].repeat_interleave(k, 0)
    if s["scale"] is None:
        return [off, pos, xs[:R], None]
    scale_s = torch.zeros(R + 1, device="cuda")
    scale_s[to] = s["scale"].repeat_interleave(k)
    return [off, pos, xs[:R], scale_s[:R]]


def _experts(s, c):
    off, R, E = s["offsets"], s["xq"].shape[0], c["E"]
    r = torch.arange(R, device="cuda")
    e = (r[:, None] >= off[None, 1:]).sum(1)
    live = e < E
    e = e.clamp(max=E - 1)
    at = torch.where(live, r - off[e], s["most"])  # place s["most"]: rows of no expert
    x = torch.zeros(E, s["most"] + 1, c["K"], device="cuda")
    x[e, at] = s["xq"].float()
    acc = (x @ s["wq"].float().transpose(1, 2))[e, at]
    act = s["act"][:, None] if c["per_token"] else s["act"]
    y = acc * (act * s["ws"][e])
    if c["bias"]:
        y = y + s["bias"][e]
    return torch.where(live[:, None], y, 0).to(s["y"].dtype)


def _combine(s, c):
    pos = s["pos"].long()
    w = torch.where(pos < 0, 0, s["weights"])
    y = (s["z"][pos.clamp(min=0)].float() * w[..., None]).sum(1)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(s["z"].dtype)


def _grad(s, c):
    pos, R = s["pos"].long(), s["z"].shape[0]
    live = pos >= 0
    dy, at = s["dy"].float(), pos.clamp(min=0)
    dw = torch.where(live, (s["z"][at].float() * dy[:, None]).sum(2), 0)
    dz = torch.zeros(R + 1, c["N"], dtype=s["z"].dtype, device="cuda")
    dz[torch.where(live, pos, R)] = (s["weights"][..., None] * dy[:, None]).to(dz.dtype)
    dx = torch.where(live[..., None], s["dxs"][at].float(), 0).sum(1).to(dz.dtype)
    return [dz[:R], dw, dx]


# ------------------------------------------------------------------ what it takes
def work(case):
    c = case
    T = c["T"]
    size = {"bf16": 2, "f32": 4, "i8": 1}[c["dtype"]]
    if c["kind"] == "norm":
        n, K = T * c["K"], c["K"]
        # x and the residual in, h and the codes out, gamma, a step per row
        return dict(bytes=n * (3 * size + 1) + 4 * K + 4 * T, flops=8 * n)
    R = T * c["top_k"]
    live = R * (1 - c["drop"])
    if c["kind"] == "dispatch":
        # the ids in, places and offsets out; each token read once, each copy written once
        return dict(bytes=R * 12 + 4 * (c["E"] + 1) + (T + live) * (c["K"] * size + 4), flops=R)
    if c["kind"] == "experts":
        N, K, E = c["N"], c["K"], c["E"]
        used = E * (1 - (1 - 1 / E) ** live)  # experts that some row goes to
        return dict(bytes=live * (K + 4 + N * size) + used * N * (K + 4), flops=2 * live * N * K)
    N = c["N"]
    if c["kind"] == "combine":
        return dict(bytes=N * size * (live + T * (2 if c["residual"] else 1)) + 8 * R,
                    flops=2 * live * N)
    # dy and z in, dz out, the copies' gradients in and their tokens' out
    return dict(bytes=N * size * (2 * T + 3 * live) + 12 * R, flops=4 * live * N)


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["kind"] == "norm":
        total = s["x"].double() + s["residual"].double()
        h = total.to(s["x"].dtype).double()  # the norm is taken of h as it is stored
        y = h / (h.pow(2).sum(1, keepdim=True) / c["K"] + EPS).sqrt() * s["gamma"].double()
        if c["gran"] == "static":
            step = s["act"].double()
        elif c["gran"] == "token":
            step = y.abs().max(1).values.clamp_min(1e-7) / 127
        else:
            step = y.abs().max().reshape(1).clamp_min(1e-7) / 127
        return [total, step, torch.clamp(torch.round(y / step[:, None]), -127, 127) * step[:, None]]
    if c["kind"] == "dispatch":
        if s["scale"] is None:
            return None
        T, k = c["T"], c["top_k"]
        scale_s = torch.zeros(T * k, dtype=torch.float64)
        rows = [(e, t) for t, row in enumerate(s["ids"].tolist()) for e in row if e >= 0]
        rows.sort(key=lambda a: a[0])  # stable: by token within an expert
        given = s["scale"].double().cpu()
        scale_s[: len(rows)] = given[torch.tensor([t for _, t in rows], dtype=torch.long)]
        return [None, None, None, scale_s]
    if c["kind"] == "experts":
        off = s["offsets"].tolist()
        y = torch.zeros(s["y"].shape, dtype=torch.float64, device="cuda")
        for e in range(c["E"]):
            a, b = off[e], off[e + 1]
            if a == b:
                continue
            p = s["xq"][a:b].double() @ s["wq"][e].double().t()
            p *= s["act"][a:b, None].double() if c["per_token"] else s["act"].double()
            p *= s["ws"][e].double()
            y[a:b] = p + s["bias"][e].double() if c["bias"] else p
        return y
    pos = s["pos"].long()
    z = s["z"].double()
    w = s["weights"].double()
    if c["kind"] == "combine":
        y = torch.zeros(c["T"], c["N"], dtype=torch.float64, device="cuda")
        if s["residual"] is not None:
            y += s["residual"].double()
        for j in range(c["top_k"]):
            t = torch.nonzero(pos[:, j] >= 0)[:, 0]
            y[t] += w[t, j, None] * z[pos[t, j]]
        return y
    dy, dxs = s["dy"].double(), s["dxs"].double()
    dz, dw, dx = torch.zeros_like(z), torch.zeros_like(w), torch.zeros_like(dy)
    for j in range(c["top_k"]):
        t = torch.nonzero(pos[:, j] >= 0)[:, 0]
        p = pos[t, j]
        dz[p] = w[t, j, None] * dy[t]
        dw[t, j] = torch.einsum("tn,tn->t", dy[t], z[p])
        dx[t] += dxs[p]
    return [dz, dw, dx]
