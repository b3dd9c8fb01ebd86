"""B200 (sm_100a) smoothed W8A8 linear layer: the SmoothQuant hot path.

Thin torch-facing wrappers over the C ABI of include/sq.h, one per entry
point and with the same names.  They only marshal arguments (data pointers,
sizes, the current CUDA stream); every step of the computation runs in the
library's CUDA kernels.  Tensors must be contiguous CUDA tensors, 16-byte
aligned (fresh torch allocations are).

Sources:
* "SmoothQuant 如何解决激活量化难题？为什么适合 W8A8？" §三, §四
* "SmoothQuant：大型语言模型的精准高效训练后量化 — 深度技术评审" §2.2, §2.5, §2.6,
  §5.1 eq. (3), §5.3 eq. (4), §5.5, §6.3
* "嵌入式 SLM 动态权重量化：SmoothQuant 激活异常值迁移与 INT8 部署实战" §二, §三
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from ._lib import (SQ_ACT_PER_TENSOR_DYNAMIC, SQ_ACT_PER_TENSOR_STATIC, SQ_ACT_PER_TOKEN_DYNAMIC, SQ_BF16,
                   SQ_F32, SQ_I8, SQ_I32, SQ_I64, SQError, check, lib)

__all__ = [
    "sq_calib_absmax", "sq_smooth_scales", "sq_fuse_weights_q8",
    "sq_ln_smooth_quant_act", "sq_gemm_workspace_bytes", "sq_gemm_w8a8",
    "sq_sync_status", "sq_selftest_bounded_wait", "SQError", "Workspace",
    "sq_calib_absmax_rms", "sq_rms_smooth_quant_act", "sq_fold_into_producer",
    "sq_alpha_sweep_workspace_bytes", "sq_alpha_sweep", "sq_bmm_w8a8",
    "sq_weight_colmax", "sq_smooth_scales_peaks", "sq_probe_mma_i8", "sq_probe_mma_i8_pair",
    "sq_debug_bounds_enabled", "sq_selftest_bounds_check",
    "sq_add_rms_smooth_quant_act", "sq_moe_sort_workspace_bytes", "sq_moe_sort",
    "sq_moe_gather", "sq_moe_combine", "sq_moe_combine_grad",
    "sq_gemm_w8a8_grouped",
]


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return SQ_F32
    if t.dtype == torch.bfloat16:
        return SQ_BF16
    raise TypeError(f"expected float32 or bfloat16, got {t.dtype}")


def _ptr(t):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def sq_calib_absmax(x, amax, ln_gamma=None, ln_beta=None, ln_eps=1e-5, stream=None):
    """Running per-input-channel peak of X (or of LN(X)) over tokens; amax [K] fp32 in/out."""
    T, K = x.shape
    check(lib.sq_calib_absmax(_ptr(x), _dt(x), T, K, _ptr(ln_gamma), _ptr(ln_beta),
                              ln_eps, _ptr(amax), _stream(stream)), "sq_calib_absmax")
    return amax


def sq_calib_absmax_rms(x, amax, gamma, eps=1e-5, stream=None):
    """Running per-input-channel peak of RMSNorm(X; gamma) over tokens."""
    T, K = x.shape
    check(lib.sq_calib_absmax_rms(_ptr(x), _dt(x), T, K, _ptr(gamma), eps, _ptr(amax),
                                  _stream(stream)), "sq_calib_absmax_rms")
    return amax


def sq_smooth_scales(amax_x, w, alpha, s, inv_s, act_delta_static=None, stream=None):
    """eq. (4) smoothing factors s, 1/s (and the static activation step)."""
    N, K = w.shape
    check(lib.sq_smooth_scales(_ptr(amax_x), _ptr(w), _dt(w), N, K, float(alpha), _ptr(s),
                               _ptr(inv_s), _ptr(act_delta_static), _stream(stream)),
          "sq_smooth_scales")
    return s, inv_s


def sq_weight_colmax(w, amax_w, stream=None):
    """amax_w[k] = max_n |W[n,k]| (the weight half of eq. (4)'s peaks)."""
    N, K = w.shape
    check(lib.sq_weight_colmax(_ptr(w), _dt(w), N, K, _ptr(amax_w), _stream(stream)),
          "sq_weight_colmax")
    return amax_w


def sq_smooth_scales_peaks(amax_x, amax_w, alpha, s, inv_s, act_delta_static=None, stream=None):
    """eq. (4) from both sets of peaks: s, 1/s (and the static step)."""
    K = amax_x.numel()
    check(lib.sq_smooth_scales_peaks(_ptr(amax_x), _ptr(amax_w), K, float(alpha), _ptr(s),
                                     _ptr(inv_s), _ptr(act_delta_static), _stream(stream)),
          "sq_smooth_scales_peaks")
    return s, inv_s


def sq_fuse_weights_q8(w, s, wq, w_scale, gamma=None, beta=None, gamma_out=None,
                       beta_out=None, stream=None):
    """W*s -> per-output-channel INT8 (wq, w_scale); gamma/s, beta/s."""
    N, K = w.shape
    check(lib.sq_fuse_weights_q8(_ptr(w), _dt(w), N, K, _ptr(s), _ptr(wq), _ptr(w_scale),
                                 _ptr(gamma), _ptr(beta), _ptr(gamma_out), _ptr(beta_out),
                                 _stream(stream)), "sq_fuse_weights_q8")
    return wq, w_scale


def sq_ln_smooth_quant_act(x, xq, act_scale, gamma_s=None, beta_s=None, ln_eps=1e-5,
                           inv_s=None, per_token=True, n_clipped=None, stream=None,
                           per_tensor_dynamic=False):
    """Fused LN + smoothing + symmetric INT8 quantizer -> xq (and act_scale).
    per_token: one step per token; else the step in act_scale[0] (static), or
    with per_tensor_dynamic one step from the peak of the whole call."""
    T, K = x.shape
    if per_tensor_dynamic:
        gran = SQ_ACT_PER_TENSOR_DYNAMIC
    else:
        gran = SQ_ACT_PER_TOKEN_DYNAMIC if per_token else SQ_ACT_PER_TENSOR_STATIC
    check(lib.sq_ln_smooth_quant_act(_ptr(x), _dt(x), T, K, _ptr(gamma_s), _ptr(beta_s),
                                     ln_eps, _ptr(inv_s), gran, _ptr(act_scale), _ptr(xq),
                                     _ptr(n_clipped), _stream(stream)),
          "sq_ln_smooth_quant_act")
    return xq, act_scale


def sq_rms_smooth_quant_act(x, xq, act_scale, gamma_s, eps=1e-5, per_token=True,
                            n_clipped=None, stream=None, per_tensor_dynamic=False):
    """RMSNorm (gamma_s = gamma / s) + symmetric INT8 quantizer -> xq (and
    act_scale), granularities as sq_ln_smooth_quant_act."""
    T, K = x.shape
    if per_tensor_dynamic:
        gran = SQ_ACT_PER_TENSOR_DYNAMIC
    else:
        gran = SQ_ACT_PER_TOKEN_DYNAMIC if per_token else SQ_ACT_PER_TENSOR_STATIC
    check(lib.sq_rms_smooth_quant_act(_ptr(x), _dt(x), T, K, _ptr(gamma_s), eps, gran,
                                      _ptr(act_scale), _ptr(xq), _ptr(n_clipped),
                                      _stream(stream)), "sq_rms_smooth_quant_act")
    return xq, act_scale


_ROW_TYPES = {torch.float32: SQ_F32, torch.bfloat16: SQ_BF16, torch.int8: SQ_I8}
_ID_TYPES = {torch.int32: SQ_I32, torch.int64: SQ_I64}


def _arg(t, what, dtype, numel, dev=None):
    """Pointer of a contiguous tensor of this type and size on device `dev`,
    the current one (None: NULL)."""
    if t is None:
        return None
    if t.dtype is not dtype:
        raise TypeError(f"{what}: expected {dtype}, got {t.dtype}")
    if t.numel() != numel:
        raise ValueError(f"{what}: expected {numel} elements, got {t.numel()}")
    if t.get_device() != (torch.cuda.current_device() if dev is None else dev):
        raise ValueError(f"{what}: not on the current CUDA device")
    if not t.is_contiguous():
        raise ValueError(f"{what}: tensors must be contiguous")
    return t.data_ptr()


def _here(stream):
    """The current device and the stream to use, as integers (short calls are
    bound by the host: no Stream object is made)."""
    dev = torch.cuda.current_device()
    if stream is None:
        return dev, torch._C._cuda_getCurrentRawStream(dev)
    return dev, _stream(stream)


def _scratch(workspace, need, what):
    """(pointer, bytes) of a Workspace or a tensor of at least `need` bytes."""
    if not need:
        return None, 0
    if workspace is None:
        raise ValueError(f"{what} needs a workspace of {need} bytes")
    ws = workspace.get(need) if isinstance(workspace, Workspace) else workspace
    if ws.get_device() != torch.cuda.current_device():
        raise ValueError(f"{what}: the workspace is not on the current CUDA device")
    return _ptr(ws), ws.numel() * ws.element_size()


def sq_add_rms_smooth_quant_act(x, residual, h, xq, act_scale, gamma_s, eps=1e-5, per_token=True,
                                n_clipped=None, stream=None, per_tensor_dynamic=False):
    """h = x + residual, then sq_rms_smooth_quant_act of the stored h, in one
    pass -> h, xq (and act_scale).  h may be x or residual itself."""
    T, K = x.shape
    dt = x.dtype
    if per_tensor_dynamic:
        gran = SQ_ACT_PER_TENSOR_DYNAMIC
    else:
        gran = SQ_ACT_PER_TOKEN_DYNAMIC if per_token else SQ_ACT_PER_TENSOR_STATIC
    steps = T if gran == SQ_ACT_PER_TOKEN_DYNAMIC else 1
    dev, st = _here(stream)
    check(lib.sq_add_rms_smooth_quant_act(
        _arg(x, "x", dt, T * K, dev), _arg(residual, "residual", dt, T * K, dev), _dt(x), T, K,
        _arg(gamma_s, "gamma_s", torch.float32, K, dev), eps, gran, _arg(h, "h", dt, T * K, dev),
        _arg(act_scale, "act_scale", torch.float32, steps, dev), _arg(xq, "xq", torch.int8, T * K, dev),
        _arg(n_clipped, "n_clipped", torch.int64, 1, dev), st),
        "sq_add_rms_smooth_quant_act")
    return h, xq, act_scale


def sq_moe_sort_workspace_bytes(T, top_k, E) -> int:
    return int(lib.sq_moe_sort_workspace_bytes(T, top_k, E))


def sq_moe_sort(expert_ids, num_experts, offsets, pos, workspace=None, stream=None):
    """Assignments sorted by expert: expert_ids [T, top_k] int32 or int64 (an
    id outside [0, E): none) -> offsets [E + 1], pos [T, top_k] int32."""
    T, k = expert_ids.shape
    if expert_ids.dtype not in _ID_TYPES:
        raise TypeError(f"expert_ids: expected int32 or int64, got {expert_ids.dtype}")
    ws, nbytes = _scratch(workspace, sq_moe_sort_workspace_bytes(T, k, num_experts), "sq_moe_sort")
    dev, st = _here(stream)
    check(lib.sq_moe_sort(_arg(expert_ids, "expert_ids", expert_ids.dtype, T * k, dev),
                          _ID_TYPES[expert_ids.dtype], T, k, num_experts,
                          _arg(offsets, "offsets", torch.int32, num_experts + 1, dev),
                          _arg(pos, "pos", torch.int32, T * k, dev), ws, nbytes, st),
          "sq_moe_sort")
    return offsets, pos


def sq_moe_gather(x, pos, xs, scale=None, scale_s=None, stream=None):
    """Each token's row (int8, bf16 or fp32), and its step, copied to its
    sorted rows: xs[pos[t, c]] = x[t], scale_s[pos[t, c]] = scale[t]."""
    T, K = x.shape
    R, k = xs.shape[0], pos.shape[1]
    if x.dtype not in _ROW_TYPES:
        raise TypeError(f"x: expected int8, bfloat16 or float32, got {x.dtype}")
    dev, st = _here(stream)
    check(lib.sq_moe_gather(_arg(x, "x", x.dtype, T * K, dev), _ROW_TYPES[x.dtype], T, K,
                            _arg(scale, "scale", torch.float32, T, dev),
                            _arg(pos, "pos", torch.int32, T * k, dev), k, R,
                            _arg(xs, "xs", x.dtype, R * K, dev),
                            _arg(scale_s, "scale_s", torch.float32, R, dev), st),
          "sq_moe_gather")
    return xs, scale_s


def sq_moe_combine(z, pos, y, weights=None, residual=None, stream=None):
    """y[t] = residual[t] + sum_c weights[t, c] * z[pos[t, c]] (weights None:
    1; without weights and residual the gradient of sq_moe_gather).  y may be
    the residual itself."""
    R, N = z.shape
    T, k = pos.shape
    dev, st = _here(stream)
    check(lib.sq_moe_combine(_arg(z, "z", z.dtype, R * N, dev), _dt(z), R, N,
                             _arg(pos, "pos", torch.int32, T * k, dev),
                             _arg(weights, "weights", torch.float32, T * k, dev), T, k,
                             _arg(residual, "residual", z.dtype, T * N, dev),
                             _arg(y, "y", z.dtype, T * N, dev), st), "sq_moe_combine")
    return y


def sq_moe_combine_grad(dy, pos, z=None, weights=None, dz=None, dweights=None, stream=None):
    """Gradients of sq_moe_combine: dz[pos[t, c]] = weights[t, c] * dy[t] and
    dweights[t, c] = <dy[t], z[pos[t, c]]>, each where its output is given.
    For dz no two assignments may share a row (sq_moe_sort's never do)."""
    T, N = dy.shape
    k = pos.shape[1]
    rows = dz if dz is not None else z
    R = 0 if rows is None else rows.shape[0]
    if dweights is not None and z is None:
        raise ValueError("dweights needs z")
    dev, st = _here(stream)
    check(lib.sq_moe_combine_grad(_arg(dy, "dy", dy.dtype, T * N, dev), _dt(dy), T, N,
                                  _arg(pos, "pos", torch.int32, T * k, dev),
                                  _arg(weights, "weights", torch.float32, T * k, dev), k,
                                  _arg(z, "z", dy.dtype, R * N, dev), R,
                                  _arg(dz, "dz", dy.dtype, R * N, dev),
                                  _arg(dweights, "dweights", torch.float32, T * k, dev),
                                  st), "sq_moe_combine_grad")
    return dz, dweights


def sq_fold_into_producer(s, w_scale, bias=None, stream=None):
    """1/s folded into the producing linear: w_scale /= s, bias /= s (in place)."""
    K = s.numel()
    check(lib.sq_fold_into_producer(_ptr(s), K, _ptr(w_scale), _ptr(bias), _stream(stream)),
          "sq_fold_into_producer")
    return w_scale, bias


def sq_alpha_sweep_workspace_bytes(M, N, K) -> int:
    return int(lib.sq_alpha_sweep_workspace_bytes(M, N, K))


def sq_alpha_sweep(amax_x, w, x, y_ref, alphas, ln_gamma=None, ln_beta=None, ln_eps=1e-5,
                   per_token=True, per_tensor_dynamic=False, workspace=None, stream=None):
    """Layer-output error of the smoothed W8A8 layer at each alpha: a CUDA
    tensor of len(alphas) doubles, ||y - y_ref|| / ||y_ref||."""
    N, K = w.shape
    M = x.shape[0]
    if per_tensor_dynamic:
        gran = SQ_ACT_PER_TENSOR_DYNAMIC
    else:
        gran = SQ_ACT_PER_TOKEN_DYNAMIC if per_token else SQ_ACT_PER_TENSOR_STATIC
    need = sq_alpha_sweep_workspace_bytes(M, N, K)
    ws = workspace.get(need) if isinstance(workspace, Workspace) else workspace
    if ws is None:
        ws = torch.empty(need, dtype=torch.uint8, device=x.device)
    a = (ctypes.c_float * len(alphas))(*[float(v) for v in alphas])
    err = torch.empty(len(alphas), dtype=torch.float64, device=x.device)
    check(lib.sq_alpha_sweep(_ptr(amax_x), _ptr(w), _dt(w), N, K, _ptr(x), _dt(x), M,
                             _ptr(ln_gamma), _ptr(ln_beta), ln_eps, _ptr(y_ref), a, len(alphas),
                             gran, _ptr(err), _ptr(ws), ws.numel() * ws.element_size(),
                             _stream(stream)), "sq_alpha_sweep")
    return err


def sq_bmm_w8a8(xq, wq, act_scale, w_scale, y, per_token=True, w_per_channel=True,
                acc_out=None, stream=None):
    """Batched INT8 GEMM: y[b] = (float)(xq[b] @ wq[b]^T) * (as * ws), xq
    [batch, M, K], wq [batch, N, K], y [batch, M, N]."""
    B, M, K = xq.shape
    N = wq.shape[1]
    check(lib.sq_bmm_w8a8(_ptr(xq), _ptr(wq), B, M, N, K, _ptr(act_scale), int(per_token),
                          _ptr(w_scale), int(w_per_channel), _ptr(y), _dt(y), _ptr(acc_out),
                          _stream(stream)), "sq_bmm_w8a8")
    return y


def sq_gemm_workspace_bytes(M, N, K) -> int:
    return int(lib.sq_gemm_workspace_bytes(M, N, K))


class Workspace:
    """Device scratch for the calls that take a workspace, grown on demand.
    They need no particular contents.  A buffer that was outgrown is kept: a
    captured graph may still replay calls that use it.  Each is at least twice
    the one before, so all that are kept are smaller than the one in use."""

    def __init__(self, device=None):
        self.device = device
        self.buf = None
        self._outgrown = []

    def get(self, nbytes: int):
        if nbytes == 0:
            return None
        if self.buf is None or self.buf.numel() < nbytes:
            if self.buf is not None:
                self._outgrown.append(self.buf)
                nbytes = max(nbytes, 2 * self.buf.numel())
            self.buf = torch.empty(nbytes, dtype=torch.uint8, device=self.device or "cuda")
        return self.buf


def sq_gemm_w8a8(xq, wq, act_scale, w_scale, y, per_token=True, acc_out=None,
                 workspace=None, stream=None, bias=None):
    """y = (float)(xq @ wq^T) * (act_scale[t] * w_scale[n]) (+ bias[n]);
    y fp32 or bf16.  With a bias this calls sq_gemm_w8a8_bias."""
    M, K = xq.shape
    N = wq.shape[0]
    need = sq_gemm_workspace_bytes(M, N, K)
    ws = None
    if need:
        if workspace is None:
            raise ValueError(f"sq_gemm_w8a8 needs a workspace of {need} bytes")
        ws = workspace.get(need) if isinstance(workspace, Workspace) else workspace
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    if bias is None:
        check(lib.sq_gemm_w8a8(_ptr(xq), _ptr(wq), M, N, K, _ptr(act_scale), int(per_token),
                               _ptr(w_scale), _ptr(y), _dt(y), _ptr(acc_out), _ptr(ws),
                               nbytes, _stream(stream)), "sq_gemm_w8a8")
    else:
        check(lib.sq_gemm_w8a8_bias(_ptr(xq), _ptr(wq), M, N, K, _ptr(act_scale),
                                    int(per_token), _ptr(w_scale), _ptr(bias), _ptr(y), _dt(y),
                                    _ptr(acc_out), _ptr(ws), nbytes, _stream(stream)),
              "sq_gemm_w8a8_bias")
    return y


def sq_gemm_w8a8_grouped(xq, wq, offsets, act_scale, w_scale, y, per_token=True, bias=None,
                         acc_out=None, stream=None):
    """The experts' GEMM: rows offsets[e] .. offsets[e + 1] - 1 of xq [R, K]
    with wq[e] of [E, N, K], dequantized by act_scale and w_scale [E, N] (+
    bias [E, N]); y [R, N] fp32 or bf16."""
    R, K = xq.shape
    E, N = wq.shape[:2]
    f32 = torch.float32
    dev, st = _here(stream)
    check(lib.sq_gemm_w8a8_grouped(
        _arg(xq, "xq", torch.int8, R * K, dev), _arg(wq, "wq", torch.int8, E * N * K, dev),
        _arg(offsets, "offsets", torch.int32, E + 1, dev), R, N, K, E,
        _arg(act_scale, "act_scale", f32, R if per_token else 1, dev), int(per_token),
        _arg(w_scale, "w_scale", f32, E * N, dev), _arg(bias, "bias", f32, E * N, dev),
        _arg(y, "y", y.dtype, R * N, dev), _dt(y), _arg(acc_out, "acc_out", torch.int32, R * N, dev),
        st), "sq_gemm_w8a8_grouped")
    return y


def sq_sync_status(stream=None):
    """Synchronize the stream and raise SQError if a kernel recorded a fault."""
    check(lib.sq_sync_status(_stream(stream)), "sq_sync_status")


def sq_selftest_bounded_wait(limit_ns: int, stream=None):
    check(lib.sq_selftest_bounded_wait(int(limit_ns), _stream(stream)),
          "sq_selftest_bounded_wait")


def sq_probe_mma_i8(kblocks: int, grid: int, stream=None):
    """Launch the INT8 tensor-core rate probe: grid CTAs, each issuing
    kblocks x 4 tcgen05.mma kind::i8 steps of 128 x 256 x 32 (8,388,608 ops
    per k-block).  Returns the op count; the caller times the launch."""
    check(lib.sq_probe_mma_i8(int(kblocks), int(grid), _stream(stream)), "sq_probe_mma_i8")
    return 8388608 * int(kblocks) * int(grid)


def sq_probe_mma_i8_pair(kblocks: int, pairs: int, stream=None):
    """Launch the CTA-pair INT8 tensor-core rate probe: `pairs` clusters of two
    CTAs issuing kblocks x 4 tcgen05.mma.cta_group::2 steps of 256 x 256 x 32
    (16,777,216 ops per k-block per pair).  Returns the op count."""
    check(lib.sq_probe_mma_i8_pair(int(kblocks), int(pairs), _stream(stream)),
          "sq_probe_mma_i8_pair")
    return 16777216 * int(kblocks) * int(pairs)


def sq_debug_bounds_enabled() -> bool:
    """True for the bounds-checked build (libsq_b200_debug.so)."""
    return bool(lib.sq_debug_bounds_enabled())


def sq_selftest_bounds_check(stream=None):
    """Launch the bounds-check self-test (one thread checks an offset at
    its tensor's end, touching no memory); sq_sync_status() then raises
    SQ_ERR_BOUNDS in the bounds-checked build and nothing otherwise."""
    check(lib.sq_selftest_bounds_check(_stream(stream)), "sq_selftest_bounds_check")
