"""The dense operators around the routed experts: the RMS norm with the
residual's addition, the gated projection of a shared expert and the linear
projection with bias, activation and residual, each with its backward pass.

Thin bindings over the C ABI (``moe_rms_norm``, ``moe_gated_ffn``,
``moe_linear`` and their ``_backward`` forms): they check the tensors, allocate
outputs and workspaces that the caller did not pass, and launch on the current
stream. All tensors are contiguous and share one CUDA device; activations,
weights and gradients are bfloat16. Nothing synchronises, and every call can be
captured in a CUDA graph after one eager call.

``stream`` takes a call to another stream, its new outputs and workspaces
included. It does not wait there for whoever wrote the inputs, nor keep them
alive: order that stream behind the writer's (``stream.wait_stream``), and hold
inputs, or call their ``record_stream``, until its work is done.

Gradients are explicit calls, not autograd's: a result carries no graph, also
where an input requires grad, and ``backward()`` does not reach what came before.
"""
from __future__ import annotations

import contextlib
import typing

import torch

from . import _FLOAT8, ACT, _check, _need, lib

_BF16 = torch.bfloat16
_F32 = torch.float32
_LINEAR_ACT = dict(ACT, none=-1)
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


@contextlib.contextmanager
def _on(device, stream):
    if stream is None:
        with torch.cuda.device(device):
            yield
    else:
        if stream.device != device:
            raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
        with torch.cuda.stream(stream):
            yield


# Every entry point passes a call for another device than the current one, or with a
# stream, once through itself with that device and stream current (_on): outputs and
# workspaces allocated inside then belong to the stream that uses them.
def _elsewhere(index, stream):
    return stream is not None or index != _current_device()


def _tensor(t, name, dtype, shape, index):
    """The address of a tensor of the given type and sizes, contiguous, on CUDA
    device `index`."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.is_contiguous()
            and t.get_device() == index):
        return t.data_ptr()
    _need(t, name, (dtype,), len(shape), shape, cuda=False)
    raise ValueError(f"{name} is on {t.device}, not cuda:{index}: all tensors must share one CUDA device")


def _first(t, name):
    """The tensor that fixes the token count and the device: (shape, device index)."""
    if not (isinstance(t, torch.Tensor) and t.dtype is _BF16 and t.dim() == 2 and t.is_contiguous() and t.is_cuda):
        _need(t, name, (_BF16,), 2, cuda=False)
        raise ValueError(f"{name} must be on a CUDA device, not {t.device}")
    return t.shape, t.get_device()


def _output(t, name, like, shape, index):
    """(tensor, address) of the caller's bf16 output after its checks, or of a new
    one of the type and device of the input `like`."""
    if t is None:
        t = torch.empty_like(like) if like.shape == shape else like.new_empty(*shape)
        return t, t.data_ptr()
    return t, _tensor(t, name, _BF16, shape, index)


def _rows(t, name):
    """Rows of a weight matrix; its type, columns and device are checked by _tensor."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        _need(t, name, (_BF16,), 2, cuda=False)
    return t.shape[0]


def _workspace(ws, need, like):
    if ws is None:
        return like.new_empty(need // 2)  # (bf16, as `like` is; sizes are multiples of 256 bytes)
    _need(ws, "workspace", (torch.uint8,), 1, cuda=False)
    if ws.device != like.device:
        raise ValueError(f"workspace is on {ws.device}, not {like.device}: all tensors must share one CUDA device")
    return ws


def _act(act, table):
    if act not in table:
        raise ValueError(f"act: {act!r}, expected one of {', '.join(sorted(table))}")
    return table[act]


class RMSNormOutput(typing.NamedTuple):
    """What ``rms_norm`` gives: ``y`` bf16 [T,H]; ``residual`` the residual
    stream after the addition (x itself when no residual was given, None when y
    took its place); with quantize, ``codes`` float8_e4m3fn [T,H] and ``scales``
    fp32 [T,H/128]; with rstd, ``rstd`` fp32 [T] for ``rms_norm_backward``."""

    y: torch.Tensor | None
    residual: torch.Tensor | None
    codes: torch.Tensor | None = None
    scales: torch.Tensor | None = None
    rstd: torch.Tensor | None = None


def rms_norm(x, weight, residual=None, eps: float = 1e-6, quantize: bool = False, rstd: bool = False, out=None,
             residual_out=None, stream=None) -> RMSNormOutput:
    """moe_rms_norm: s = x + residual (rounded to bf16, the residual stream),
    y = s * (mean(s^2) + eps)^(-1/2) * weight. ``out`` and ``residual_out`` may be
    x or residual for an in-place step (without a residual, out = x overwrites the
    stream: the result's ``residual`` is None then). ``quantize`` adds y in the form
    of the FP8 experts' activations (H a multiple of 128). ``stream``: launch there."""
    shape, dev = _first(x, "x")
    if _elsewhere(dev, stream):
        with _on(x.device, stream):
            return rms_norm(x, weight, residual, eps, quantize, rstd, out, residual_out)
    T, H = shape
    w = _tensor(weight, "weight", _BF16, (H,), dev)
    r = sp = cp = kp = rp = codes = scales = rs = None
    s = x
    if residual is not None:
        r = _tensor(residual, "residual", _BF16, shape, dev)
        s, sp = _output(residual_out, "residual_out", x, shape, dev)
    elif residual_out is not None:
        raise ValueError("residual_out was given without a residual")
    xp = x.data_ptr()
    y, yp = _output(out, "out", x, shape, dev)
    if yp == xp and residual is None and T:
        s = None  # x holds y after the call
    if quantize:
        codes = torch.empty_like(x, dtype=_FLOAT8)
        scales = x.new_empty(T, H // 128, dtype=_F32)
        cp, kp = codes.data_ptr(), scales.data_ptr()
    if rstd:
        rs = x.new_empty(T, dtype=_F32)
        rp = rs.data_ptr()
    _check(lib().moe_rms_norm(xp, r, w, T, H, eps, yp, sp, cp, kp, rp, _raw_stream(dev)), "moe_rms_norm")
    return RMSNormOutput(y, s, codes, scales, rs)


def rms_norm_backward(dy, s, weight, rstd, dresidual=None, dx=None, dw=None, workspace=None, stream=None):
    """moe_rms_norm_backward: (dx bf16 [T,H], dw bf16 [H]) from the gradient dy at
    y and dresidual at the residual stream; s, weight and rstd are the
    forward's (``RMSNormOutput.residual`` and ``.rstd``). dx is the gradient of x
    and of the residual alike. ``stream``: launch there."""
    shape, dev = _first(dy, "dy")
    if _elsewhere(dev, stream):
        with _on(dy.device, stream):
            return rms_norm_backward(dy, s, weight, rstd, dresidual, dx, dw, workspace)
    T, H = shape
    sp = _tensor(s, "s", _BF16, shape, dev)
    w = _tensor(weight, "weight", _BF16, (H,), dev)
    r = _tensor(rstd, "rstd", _F32, (T,), dev)
    dr = None if dresidual is None else _tensor(dresidual, "dresidual", _BF16, shape, dev)
    dx, dxp = _output(dx, "dx", dy, shape, dev)
    dw, dwp = _output(dw, "dw", weight, (H,), dev)
    L = lib()
    ws = _workspace(workspace, L.moe_rms_norm_backward_workspace_size(T, H), dy)
    _check(L.moe_rms_norm_backward(dy.data_ptr(), sp, w, r, dr, T, H, dxp, dwp, ws.data_ptr(), ws.nbytes,
                                   _raw_stream(dev)), "moe_rms_norm_backward")
    return dx, dw


def _gate_up(w_gate_up, H, dev):
    """(I, address) of the [2I,H] weight."""
    twoI = _rows(w_gate_up, "w_gate_up")
    if twoI % 2 != 0:
        raise ValueError(f"w_gate_up: {twoI} rows, expected 2*I (gate rows, then up rows)")
    return twoI // 2, _tensor(w_gate_up, "w_gate_up", _BF16, (twoI, H), dev)


def gated_ffn(x, w_gate_up, act: str = "silu", save: bool = False, out=None, stream=None):
    """moe_gated_ffn: h = act(x Wg^T) * (x Wu^T) in one kernel, w_gate_up [2I,H]
    the gate rows and then the up rows (one expert's layout). Returns h bf16
    [T,I]; with save, (h, gu) with the fp32 pre-activations [T,2I] that
    ``gated_ffn_backward`` takes. ``stream``: launch there."""
    a = _act(act, ACT)
    (T, H), dev = _first(x, "x")
    if _elsewhere(dev, stream):
        with _on(x.device, stream):
            return gated_ffn(x, w_gate_up, act, save, out)
    I, w = _gate_up(w_gate_up, H, dev)
    h, hp = _output(out, "out", x, (T, I), dev)
    gu = x.new_empty(T, 2 * I, dtype=_F32) if save else None
    _check(lib().moe_gated_ffn(x.data_ptr(), w, T, H, I, a, hp, gu.data_ptr() if save else None,
                               _raw_stream(dev)), "moe_gated_ffn")
    return (h, gu) if save else h


def gated_ffn_backward(dh, x, w_gate_up, gu, act: str = "silu", dx=None, dw=None, workspace=None, stream=None):
    """moe_gated_ffn_backward: (dx bf16 [T,H], dw bf16 [2I,H]) from dh [T,I], with
    x, w_gate_up and the gu that the forward kept. ``stream``: launch there."""
    a = _act(act, ACT)
    shape, dev = _first(x, "x")
    if _elsewhere(dev, stream):
        with _on(x.device, stream):
            return gated_ffn_backward(dh, x, w_gate_up, gu, act, dx, dw, workspace)
    T, H = shape
    I, w = _gate_up(w_gate_up, H, dev)
    d = _tensor(dh, "dh", _BF16, (T, I), dev)
    g = _tensor(gu, "gu", _F32, (T, 2 * I), dev)
    dx, dxp = _output(dx, "dx", x, shape, dev)
    dw, dwp = _output(dw, "dw", w_gate_up, (2 * I, H), dev)
    L = lib()
    ws = _workspace(workspace, L.moe_gated_ffn_backward_workspace_size(T, I), x)
    _check(L.moe_gated_ffn_backward(d, x.data_ptr(), w, g, T, H, I, a, dxp, dwp, ws.data_ptr(), ws.nbytes,
                                    _raw_stream(dev)), "moe_gated_ffn_backward")
    return dx, dw


def linear(x, w, bias=None, act: str = "none", residual=None, save: bool = False, out=None,
           stream=None):
    """moe_linear: y = act(x W^T + bias) + residual, w [N,K], rounded once. ``out``
    may be residual. Returns y bf16 [T,N]; with save, (y, z) with the bf16
    pre-activation [T,N] that ``linear_backward`` takes (None without an
    activation: the backward pass needs none). ``stream``: launch there."""
    a = _act(act, _LINEAR_ACT)
    (T, K), dev = _first(x, "x")
    if _elsewhere(dev, stream):
        with _on(x.device, stream):
            return linear(x, w, bias, act, residual, save, out)
    N = _rows(w, "w")
    wp = _tensor(w, "w", _BF16, (N, K), dev)
    b = None if bias is None else _tensor(bias, "bias", _BF16, (N,), dev)
    r = None if residual is None else _tensor(residual, "residual", _BF16, (T, N), dev)
    y, yp = _output(out, "out", x, (T, N), dev)
    z = x.new_empty(T, N) if save and act != "none" else None
    _check(lib().moe_linear(x.data_ptr(), wp, b, r, T, K, N, a, yp, None if z is None else z.data_ptr(),
                            _raw_stream(dev)), "moe_linear")
    return (y, z) if save else y


def linear_backward(dy, x, w, z=None, act: str = "none", bias: bool = False, dx=None, dw=None, workspace=None,
                    stream=None):
    """moe_linear_backward: (dx bf16 [T,K], dw bf16 [N,K], db bf16 [N] or None)
    from dy [T,N], with x, w and, for an activation, the z that the forward
    kept. ``bias`` asks for db; the residual's gradient is dy itself.
    ``stream``: launch there."""
    a = _act(act, _LINEAR_ACT)
    shape, dev = _first(x, "x")
    if _elsewhere(dev, stream):
        with _on(x.device, stream):
            return linear_backward(dy, x, w, z, act, bias, dx, dw, workspace)
    T, K = shape
    N = _rows(w, "w")
    wp = _tensor(w, "w", _BF16, (N, K), dev)
    d = _tensor(dy, "dy", _BF16, (T, N), dev)
    zp = None if z is None else _tensor(z, "z", _BF16, (T, N), dev)
    dx, dxp = _output(dx, "dx", x, shape, dev)
    dw, dwp = _output(dw, "dw", w, (N, K), dev)
    db = w.new_empty(N) if bias else None
    L = lib()
    ws = _workspace(workspace, L.moe_linear_backward_workspace_size(T, N, a, int(bool(bias))), x)
    _check(L.moe_linear_backward(d, x.data_ptr(), wp, zp, T, K, N, a, dxp, dwp, None if db is None else db.data_ptr(),
                                 ws.data_ptr(), ws.nbytes, _raw_stream(dev)), "moe_linear_backward")
    return dx, dw, db
