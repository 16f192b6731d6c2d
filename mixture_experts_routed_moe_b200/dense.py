"""The dense operators around the routed experts: the RMS norm with the
residual's addition, the gated projection of a shared expert and the linear
projection with bias, activation and residual, each with its backward pass.

Thin bindings over the C ABI (``moe_rms_norm``, ``moe_gated_ffn``,
``moe_linear`` and their ``_backward`` forms): they check the tensors, allocate
outputs and workspaces that the caller did not pass, and launch on the current
stream (or ``stream``). All tensors are contiguous and share one CUDA device;
activations, weights and gradients are bfloat16. Nothing synchronises, and
every call can be captured in a CUDA graph after one eager call.
"""
from __future__ import annotations

import contextlib
import typing

import torch

from . import _FLOAT8, ACT, _check, _need, lib

_BF16 = torch.bfloat16
_F32 = torch.float32
_LINEAR_ACT = dict(ACT, none=-1)
_NO_GUARD = contextlib.nullcontext()


def _tensor(t, name, dtype, shape, device):
    """One tensor of the given type and sizes, contiguous, on `device` (a CUDA
    device). The common case is one line: small calls are bound by the host."""
    if (isinstance(t, torch.Tensor) and t.dtype == dtype and t.shape == shape and t.is_contiguous()
            and t.device == device):
        return t.data_ptr()
    _need(t, name, (dtype,), len(shape), shape, cuda=False)
    raise ValueError(f"{name} is on {t.device}, x on {device}: all tensors must share one CUDA device")


def _optional(t, name, dtype, shape, device):
    return None if t is None else _tensor(t, name, dtype, shape, device)


def _first(t, name):
    """The tensor that fixes the token count and the device: (T, columns, device)."""
    if not (isinstance(t, torch.Tensor) and t.dtype == _BF16 and t.dim() == 2 and t.is_contiguous() and t.is_cuda):
        _need(t, name, (_BF16,), 2, cuda=False)
        raise ValueError(f"{name} must be on a CUDA device, not {t.device}")
    T, n = t.shape
    return T, n, t.device


def _launch(device, stream):
    """(guard, raw stream) of a call on `device`. Under the guard the device is
    the current one and the caller's stream, if given, the current stream, so
    outputs and workspaces allocated there belong to the stream that uses them."""
    index = device.index
    if stream is not None:
        if stream.device != device:
            raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
        return torch.cuda.stream(stream), stream.cuda_stream
    guard = _NO_GUARD if torch.cuda.current_device() == index else torch.cuda.device(index)
    return guard, torch._C._cuda_getCurrentRawStream(index)


def _output(t, name, like, shape, device):
    """The caller's bf16 output tensor after its checks, or a new one (of
    like's type and device: `like` is an input)."""
    if t is None:
        return torch.empty_like(like) if like.shape == shape else like.new_empty(shape)
    _tensor(t, name, _BF16, shape, device)
    return t


def _workspace(ws, need, device):
    if ws is None:
        return torch.empty(need, dtype=torch.uint8, device=device)
    _need(ws, "workspace", (torch.uint8,), 1, cuda=False)
    if ws.device != device:
        raise ValueError(f"workspace is on {ws.device}, x on {device}: all tensors must share one CUDA device")
    return ws


def _act(act, table):
    if act not in table:
        raise ValueError(f"act: {act!r}, expected one of {', '.join(sorted(table))}")
    return table[act]


class RMSNormOutput(typing.NamedTuple):
    """What ``rms_norm`` gives: ``y`` bf16 [T,H]; ``residual`` the residual
    stream after the addition (x itself when no residual was given); with
    quantize, ``codes`` float8_e4m3fn [T,H] and ``scales`` fp32 [T,H/128]; with
    rstd, ``rstd`` fp32 [T] for ``rms_norm_backward``."""

    y: torch.Tensor | None
    residual: torch.Tensor
    codes: torch.Tensor | None = None
    scales: torch.Tensor | None = None
    rstd: torch.Tensor | None = None


def rms_norm(x, weight, residual=None, eps: float = 1e-6, quantize: bool = False, rstd: bool = False, out=None,
             residual_out=None, stream=None) -> RMSNormOutput:
    """moe_rms_norm: s = x + residual (rounded to bf16, the residual stream),
    y = s * (mean(s^2) + eps)^(-1/2) * weight. ``out`` and ``residual_out`` may be
    x or residual for an in-place step. ``quantize`` adds y in the form of the
    FP8 experts' activations (H a multiple of 128)."""
    T, H, device = _first(x, "x")
    w = _tensor(weight, "weight", _BF16, (H,), device)
    r = _optional(residual, "residual", _BF16, (T, H), device)
    guard, st = _launch(device, stream)
    with guard:
        y = _output(out, "out", x, (T, H), device)
        s, sp = x, None
        if residual is not None:
            s = _output(residual_out, "residual_out", x, (T, H), device)
            sp = s.data_ptr()
        elif residual_out is not None:
            raise ValueError("residual_out was given without a residual")
        codes = scales = rs = None
        if quantize:
            codes = torch.empty((T, H), dtype=_FLOAT8, device=device)
            scales = torch.empty((T, H // 128), dtype=_F32, device=device)
        if rstd:
            rs = torch.empty((T,), dtype=_F32, device=device)
        _check(lib().moe_rms_norm(x.data_ptr(), r, w, T, H, eps, y.data_ptr(), sp,
                                  None if codes is None else codes.data_ptr(),
                                  None if scales is None else scales.data_ptr(),
                                  None if rs is None else rs.data_ptr(), st), "moe_rms_norm")
    return RMSNormOutput(y, s, codes, scales, rs)


def rms_norm_backward(dy, s, weight, rstd, dresidual=None, dx=None, dw=None, workspace=None, stream=None):
    """moe_rms_norm_backward: (dx bf16 [T,H], dw bf16 [H]) from the gradient dy at
    y and dresidual at the residual stream; s, weight and rstd are the
    forward's (``RMSNormOutput.residual`` and ``.rstd``). dx is the gradient of x
    and of the residual alike."""
    T, H, device = _first(dy, "dy")
    sp = _tensor(s, "s", _BF16, (T, H), device)
    w = _tensor(weight, "weight", _BF16, (H,), device)
    r = _tensor(rstd, "rstd", _F32, (T,), device)
    dr = _optional(dresidual, "dresidual", _BF16, (T, H), device)
    guard, st = _launch(device, stream)
    with guard:
        dx = _output(dx, "dx", dy, (T, H), device)
        dw = _output(dw, "dw", weight, (H,), device)
        L = lib()
        ws = _workspace(workspace, L.moe_rms_norm_backward_workspace_size(T, H), device)
        _check(L.moe_rms_norm_backward(dy.data_ptr(), sp, w, r, dr, T, H, dx.data_ptr(), dw.data_ptr(), ws.data_ptr(),
                                       ws.numel(), st), "moe_rms_norm_backward")
    return dx, dw


def _gate_up_sizes(w_gate_up, H, device):
    _need(w_gate_up, "w_gate_up", (_BF16,), 2, cuda=False)
    twoI = w_gate_up.shape[0]
    if twoI % 2 != 0:
        raise ValueError(f"w_gate_up: {twoI} rows, expected 2*I (gate rows, then up rows)")
    return twoI // 2, _tensor(w_gate_up, "w_gate_up", _BF16, (twoI, H), device)


def gated_ffn(x, w_gate_up, act: str = "silu", save: bool = False, out=None, stream=None):
    """moe_gated_ffn: h = act(x Wg^T) * (x Wu^T) in one kernel, w_gate_up [2I,H]
    the gate rows and then the up rows (one expert's layout). Returns h bf16
    [T,I]; with save, (h, gu) with the fp32 pre-activations [T,2I] that
    ``gated_ffn_backward`` takes."""
    a = _act(act, ACT)
    T, H, device = _first(x, "x")
    I, w = _gate_up_sizes(w_gate_up, H, device)
    guard, st = _launch(device, stream)
    with guard:
        h = _output(out, "out", x, (T, I), device)
        gu = torch.empty((T, 2 * I), dtype=_F32, device=device) if save else None
        _check(lib().moe_gated_ffn(x.data_ptr(), w, T, H, I, a, h.data_ptr(), gu.data_ptr() if save else None, st),
               "moe_gated_ffn")
    return (h, gu) if save else h


def gated_ffn_backward(dh, x, w_gate_up, gu, act: str = "silu", dx=None, dw=None, workspace=None, stream=None):
    """moe_gated_ffn_backward: (dx bf16 [T,H], dw bf16 [2I,H]) from dh [T,I], with
    x, w_gate_up and the gu that the forward kept."""
    a = _act(act, ACT)
    T, H, device = _first(x, "x")
    I, w = _gate_up_sizes(w_gate_up, H, device)
    d = _tensor(dh, "dh", _BF16, (T, I), device)
    g = _tensor(gu, "gu", _F32, (T, 2 * I), device)
    guard, st = _launch(device, stream)
    with guard:
        dx = _output(dx, "dx", x, (T, H), device)
        dw = _output(dw, "dw", w_gate_up, (2 * I, H), device)
        L = lib()
        ws = _workspace(workspace, L.moe_gated_ffn_backward_workspace_size(T, I), device)
        _check(L.moe_gated_ffn_backward(d, x.data_ptr(), w, g, T, H, I, a, dx.data_ptr(), dw.data_ptr(), ws.data_ptr(),
                                        ws.numel(), st), "moe_gated_ffn_backward")
    return dx, dw


def linear(x, w, bias=None, act: str = "none", residual=None, save: bool = False, out=None, stream=None):
    """moe_linear: y = act(x W^T + bias) + residual, w [N,K], rounded once. ``out``
    may be residual. Returns y bf16 [T,N]; with save, (y, z) with the fp32
    pre-activation [T,N] that ``linear_backward`` takes (None without an
    activation: the backward pass needs none)."""
    a = _act(act, _LINEAR_ACT)
    T, K, device = _first(x, "x")
    _need(w, "w", (_BF16,), 2, cuda=False)
    N = w.shape[0]
    wp = _tensor(w, "w", _BF16, (N, K), device)
    b = _optional(bias, "bias", _BF16, (N,), device)
    r = _optional(residual, "residual", _BF16, (T, N), device)
    guard, st = _launch(device, stream)
    with guard:
        y = _output(out, "out", x, (T, N), device)
        z = torch.empty((T, N), dtype=_F32, device=device) if save and act != "none" else None
        _check(lib().moe_linear(x.data_ptr(), wp, b, r, T, K, N, a, y.data_ptr(),
                                None if z is None else z.data_ptr(), st), "moe_linear")
    return (y, z) if save else y


def linear_backward(dy, x, w, z=None, act: str = "none", bias: bool = False, dx=None, dw=None, workspace=None,
                    stream=None):
    """moe_linear_backward: (dx bf16 [T,K], dw bf16 [N,K], db bf16 [N] or None)
    from dy [T,N], with x, w and, for an activation, the z that the forward
    kept. ``bias`` asks for db; the residual's gradient is dy itself."""
    a = _act(act, _LINEAR_ACT)
    T, K, device = _first(x, "x")
    _need(w, "w", (_BF16,), 2, cuda=False)
    N = w.shape[0]
    wp = _tensor(w, "w", _BF16, (N, K), device)
    d = _tensor(dy, "dy", _BF16, (T, N), device)
    zp = _optional(z, "z", _F32, (T, N), device)
    guard, st = _launch(device, stream)
    with guard:
        dx = _output(dx, "dx", x, (T, K), device)
        dw = _output(dw, "dw", w, (N, K), device)
        db = torch.empty((N,), dtype=_BF16, device=device) if bias else None
        L = lib()
        ws = _workspace(workspace, L.moe_linear_backward_workspace_size(T, N, a, int(bool(bias))), device)
        _check(L.moe_linear_backward(d, x.data_ptr(), wp, zp, T, K, N, a, dx.data_ptr(), dw.data_ptr(),
                                     None if db is None else db.data_ptr(), ws.data_ptr(), ws.numel(), st),
               "moe_linear_backward")
    return dx, dw, db
