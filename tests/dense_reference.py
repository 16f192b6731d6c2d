"""Plain 64-bit forms of the dense operators, with the error bounds that the
GPU tests hold the kernels to.

The bounds count roundings. bf16 outputs are rounded once: half a step,
2^-8 of the value. A tensor-core sum over K products takes K/16 additions of
fp32, each off by at most two steps of the running sum (the 16 products of one
instruction are aligned and truncated, then added): (K/16 + 1) 2^-22 of the
sum of the magnitudes. The activations are a few fp32 operations and one
approximate exponential: 2^-18 of the value.
"""
from __future__ import annotations

import math

import torch

HALF = 2.0 ** -8  # half a bf16 step, relative
TINY = 2.0 ** -126  # below it bf16 values are subnormal
FP32 = 2.0 ** -18  # a handful of fp32 operations and an approximate exponential


def act(name, z):
    """(f, f') of the activation in 64 bits."""
    if name == "silu":
        s = torch.sigmoid(z)
        return z * s, s * (1 + z * (1 - s))
    if name == "gelu":
        q = 0.5 * (1 + torch.erf(z / math.sqrt(2)))
        return z * q, q + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "relu":
        return z.clamp(min=0), (z > 0).double()
    return z, torch.ones_like(z)


SLOPE = {"silu": 1.1, "gelu": 1.13, "relu": 1.0, "none": 1.0}  # largest |f'|
CURVE = {"silu": 0.5, "gelu": 0.8, "relu": 0.0, "none": 0.0}  # largest |f''|


def product(a, b):
    """a b^T in 64 bits, and the bound of a tensor-core sum of it."""
    a, b = a.double(), b.double()
    return a @ b.t(), (a.shape[1] / 16 + 1) * 2.0 ** -22 * (a.abs() @ b.abs().t())


def check(got, ref, bound, what):
    got = got.double()
    assert got.shape == ref.shape, what
    assert torch.isfinite(got).all(), f"{what}: not finite"
    over = (got - ref).abs() / (bound + TINY)
    assert over.numel() == 0 or float(over.max()) <= 1.0, f"{what}: {float(over.max()):.3g} times its bound"


def check_fro(got, ref, limit, what):
    n = float(ref.norm())
    rel = float((got.double() - ref).norm()) / n if n else 0.0
    assert rel <= limit, f"{what}: relative error {rel:.3g}"


def gated(x, w, name):
    I = w.shape[0] // 2
    z, dz = product(x, w)
    g, u, eg, eu = z[:, :I], z[:, I:], dz[:, :I], dz[:, I:]
    f, _ = act(name, g)
    h = f * u
    bound = HALF * h.abs() + SLOPE[name] * eg * (u.abs() + eu) + f.abs() * eu + FP32 * (f.abs() + eg) * u.abs()
    return h, z, bound * (1 + HALF), dz + 2.0 ** -24 * z.abs()


def gated_grads(dh, x, w, name):
    """dx, dw with their bounds: the pre-activations' error, the rounding of
    dg and du to bf16 and the products' sums, all in the worst case."""
    I = w.shape[0] // 2
    z, ez = product(x, w)
    g, u, eg, eu = z[:, :I], z[:, I:], ez[:, :I], ez[:, I:]
    f, d = act(name, g)
    dh = dh.double()
    a = dh.abs()
    dgu = torch.cat([dh * u * d, dh * f], 1)
    edge = (g.abs() <= eg).double() if name == "relu" else 0.0  # the slope jumps at zero
    e = torch.cat([a * (eu * (d.abs() + CURVE[name] * eg) + u.abs() * (CURVE[name] * eg + edge)) + FP32 * a * u.abs(),
                   a * (SLOPE[name] * eg) + FP32 * a * f.abs()], 1)
    e = e + HALF * (dgu.abs() + e)
    return _grads(dgu, e, x, w)


def _grads(d, e, x, w):
    dx, dw = d @ w.double(), d.t() @ x.double()
    ex = e @ w.double().abs() + (d.shape[1] / 16 + 1) * 2.0 ** -22 * ((d.abs() + e) @ w.double().abs())
    ew = e.t() @ x.double().abs() + (d.shape[0] / 16 + 1) * 2.0 ** -22 * ((d.abs() + e).t() @ x.double().abs())
    return dx, dw, ex + HALF * (dx.abs() + ex), ew + HALF * (dw.abs() + ew)


def linear(x, w, bias, name, residual):
    z, ez = product(x, w)
    if bias is not None:
        z = z + bias.double()
        ez = ez + 2.0 ** -24 * (z.abs() + ez)
    f, _ = act(name, z)
    y, e = f, SLOPE[name] * ez + (FP32 * f.abs() if name != "none" else 0.0)
    if residual is not None:
        y = y + residual.double()
        e = e + 2.0 ** -24 * (y.abs() + e)
    return y, z, e + HALF * (y.abs() + e), ez


def linear_grads(dy, x, w, bias, name):
    z, ez = product(x, w)
    if bias is not None:
        z = z + bias.double()
        ez = ez + 2.0 ** -24 * (z.abs() + ez)
    _, d = act(name, z)
    dy = dy.double()
    dz = dy * d
    if name == "none":
        e = torch.zeros_like(dz)
        eb = e
    else:
        edge = (z.abs() <= ez).double() if name == "relu" else 0.0
        kept = ez + HALF * (z.abs() + ez)  # the forward keeps z in bf16
        eb = dy.abs() * (CURVE[name] * kept + edge + FP32)
        e = eb + HALF * (dz.abs() + eb)
    dx, dw, ex, ew = _grads(dz, e, x, w)
    db = dz.sum(0)
    s = eb.sum(0) + dz.shape[0] * 2.0 ** -24 * (dz.abs() + eb).sum(0)
    return dx, dw, db, ex, ew, s + HALF * (db.abs() + s)


NORM = 2.0 ** -17  # sums of squares, rsqrt and scalings in fp32, relative


def norm(x, weight, residual, eps):
    s = x.double() if residual is None else (x.double() + residual.double()).to(torch.bfloat16).double()
    r = 1 / (s.square().mean(1, keepdim=True) + eps).sqrt()
    y = s * r * weight.double()
    return s, r[:, 0], y


def norm_grads(dy, s, weight, eps, dresidual):
    s, dy, w = s.double(), dy.double(), weight.double()
    H = s.shape[1]
    r = 1 / (s.square().mean(1, keepdim=True) + eps).sqrt()
    t, xh = dy * w, s * r
    dot, mag = (t * xh).mean(1, keepdim=True), (t * xh).abs().mean(1, keepdim=True)
    dx = r * (t - xh * dot)
    bound = r * NORM * (t.abs() + xh.abs() * (dot.abs() + mag))
    if dresidual is not None:
        dx = dx + dresidual.double()
        bound = bound + 2.0 ** -24 * dx.abs()
    dw = (dy * xh).sum(0)
    ew = (dy * xh).abs().sum(0) * (NORM + s.shape[0] * 2.0 ** -24)
    return dx, dw, bound + HALF * (dx.abs() + bound), ew + HALF * (dw.abs() + ew)
