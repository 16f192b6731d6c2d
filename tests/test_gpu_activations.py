"""The activations and their slopes through the dense operators over the whole range of
pre-activations: where gelu's and silu's tails run out of fp32, and far beyond.

Weights with a single one in a row make a pre-activation the product of two bf16 numbers,
exact in fp32, and let the elementwise gradients through the products that follow as
they are. The references are in 64 bits (erfc keeps the accuracy of the negative tail)."""
import math

import pytest
import torch

import dense_reference as R
import mixture_experts_routed_moe_b200 as moe

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
FLUSH = 2.0 ** -126  # exponentials and reciprocals below it are zero


def values():
    """bf16 numbers over -14 ... 14, the ends of both exponentials and far beyond."""
    v = torch.cat([torch.linspace(-14, 14, 449, dtype=torch.float64), torch.linspace(-92, 92, 185, dtype=torch.float64),
                   torch.tensor([-0.75, -1.2784, 0.0, 1e-3, -1e-3, 1e-30, -1e-30, 1e4, -1e4, 1e30, -1e30],
                                dtype=torch.float64)])
    v = torch.unique(v.to(BF).double())
    v = torch.cat([v, v.new_full((-v.numel() % 8,), 0.5)])  # a multiple of 8
    return v.to(BF).cuda()


def exact(name, z):
    """(f, f', bound of f, bound of f') in 64 bits. The kernels' steps: an exponential whose
    argument z log2 e (silu) or z^2/2 log2 e (gelu) is rounded once or twice in fp32, as is the
    constant, which is 2^-23 |z| or 2^-23 z^2 of the result; 2^-22 for the hardware's
    exponential; and a reciprocal, a fitted polynomial (7e-7) and products, together below
    2^-18. What is below 2^-126 on the way is zero: |z| 2^-126 of f."""
    if name == "relu":
        return z.clamp(min=0), (z > 0).double(), torch.zeros_like(z), torch.zeros_like(z)
    a = z.abs()
    if name == "silu":
        p = torch.sigmoid(z)
        rel = 2.0 ** -18 + 2.0 ** -23 * a.clamp(max=100)  # (from 88 on p is zero or one)
        f, d = z * p, p * (1 + z * torch.sigmoid(-z))
        # (1 - p from a rounded p: 2^-24, times z, and z ends at 17 where p is one)
        slope = p * (1 + a * torch.sigmoid(-z)) * rel + (z > 0) * 17 * 2.0 ** -22
        return f, d, f.abs() * rel + a * FLUSH, slope + (1 + a).square().clamp(max=1e8) * FLUSH
    q = 0.5 * torch.special.erfc(-z / math.sqrt(2))
    e = z * torch.exp(-z.clamp(-40, 40).square() / 2) / math.sqrt(2 * math.pi)
    rel = 2.0 ** -18 + 2.0 ** -23 * a.clamp(max=14).square()
    return z * q, q + e, (z * q).abs() * rel + a * FLUSH, (q + e.abs()) * rel + (1 + a) * FLUSH


@pytest.mark.parametrize("T", [1, 20, 60, 1000])  # the form of one token and of a few, the cluster form, the tiles
@pytest.mark.parametrize("name", ["silu", "gelu", "relu"])
def test_activation_over_its_range(T, name):
    v = values()
    N, K = v.numel(), 16
    a = (1 + (torch.arange(T, device="cuda") % 37) / 64.0).to(BF)  # bf16 numbers, 1 to 1.6
    x = torch.zeros(T, K, device="cuda", dtype=BF)
    x[:, 0], x[:, 1] = a, 1
    w = torch.zeros(2 * N, K, device="cuda", dtype=BF)
    w[:N, 0], w[N:, 1] = v, 1  # g = a v, u = 1
    z = a.double()[:, None] * v.double()[None, :]
    f, _, bound, _ = exact(name, z)
    h, gu = moe.gated_ffn(x, w, act=name, save=True)
    assert torch.equal(gu[:, :N].double(), z) and bool((gu[:, N:] == 1).all())
    R.check(h, f, R.HALF * (f.abs() + bound) + bound, f"gated {name}")
    y, zs = moe.linear(x, w[:N].contiguous(), act=name, save=True)
    assert torch.equal(zs.double(), z.to(BF).double())
    R.check(y, f, R.HALF * (f.abs() + bound) + bound, f"linear {name}")


@pytest.mark.parametrize("name", ["silu", "gelu", "relu"])
def test_slope_over_its_range(name):
    v = values()
    T, K, N = v.numel(), 16, 8
    x = torch.zeros(T, K, device="cuda", dtype=BF)
    x[:, 0], x[:, 1] = v, 1
    w = torch.zeros(2 * N, K, device="cuda", dtype=BF)
    w[0, 0], w[N, 1] = 1, 1  # the first column's g = v and u = 1; the others' are zero
    dh = torch.zeros(T, N, device="cuda", dtype=BF)
    dh[:, 0] = 0.75
    z = v.double()
    f, d, ef, ed = exact(name, z)
    _, gu = moe.gated_ffn(x, w, act=name, save=True)
    dx, dw = moe.gated_ffn_backward(dh, x, w, gu, act=name)

    def rounded(ref, err, what, got):  # one rounding of the elementwise gradient; the product by one is exact
        R.check(got, ref, err + R.HALF * (ref.abs() + err), what)

    rounded(0.75 * d, 0.75 * ed, f"dg {name}", dx[:, 0])
    rounded(0.75 * f, 0.75 * ef, f"du {name}", dx[:, 1])
    assert not dx[:, 2:].any()
    # dw of the gate's row against u's column of x: the sum of dg over the tokens
    e = 0.75 * ed + R.HALF * 0.75 * (d.abs() + ed)
    e = e.sum() + (T / 16 + 1) * 2.0 ** -22 * (0.75 * d.abs() + e).sum()
    ref = (0.75 * d).sum()
    R.check(dw[0, 1], ref, e + R.HALF * (ref.abs() + e), f"dw {name}")
    _, zs = moe.linear(x, w[:N].contiguous(), act=name, save=True)
    dx, _, db = moe.linear_backward(dh, x, w[:N].contiguous(), zs, act=name, bias=True)
    rounded(0.75 * d, 0.75 * ed, f"dz {name}", dx[:, 0])
    e = 0.75 * ed.sum() + T * 2.0 ** -24 * (0.75 * (d.abs() + ed)).sum()
    R.check(db[0], ref, e + R.HALF * (ref.abs() + e), f"db {name}")


@pytest.mark.parametrize("T,H,I", [(20, 136, 72), (200, 264, 520), (1000, 520, 1032)])
@pytest.mark.parametrize("name", ["silu", "gelu", "relu"])
def test_gated_gradients_of_every_activation(T, H, I, name):
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    x, w, dh = (torch.randn(s, generator=g, device="cuda") for s in ((T, H), (2 * I, H), (T, I)))
    x, w, dh = x.to(BF), (w * H ** -0.5).to(BF), (dh * 0.1).to(BF)
    _, gu = moe.gated_ffn(x, w, act=name, save=True)
    dx, dw = moe.gated_ffn_backward(dh, x, w, gu, act=name)
    rx, rw, ex, ew = R.gated_grads(dh, x, w, name)
    R.check(dx, rx, ex, "dx")
    R.check(dw, rw, ew, "dw")
