"""Calls of the C entry points with optional outputs left out, which the binding never
makes: what is asked for is right, and what is not is not touched."""
import pytest
import torch

import dense_reference as R
import mixture_experts_routed_moe_b200 as moe

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def normal(seed, *shape, std=1.0, mean=0.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").mul_(std).add_(mean).to(BF)


def ptr(t):
    return None if t is None else t.data_ptr()


def stream():
    return torch.cuda.current_stream().cuda_stream


@pytest.mark.parametrize("T,H", [(3, 512), (16, 7168), (700, 2048), (400, 7168), (300, 8320)])
@pytest.mark.parametrize("with_residual", [False, True])
@pytest.mark.parametrize("keep", [False, True])
def test_norm_for_codes_alone(T, H, with_residual, keep):
    x, w = normal(T, T, H), normal(H, H, std=0.2, mean=1.0)
    r = normal(T + 1, T, H) if with_residual else None
    want = moe.rms_norm(x, w, residual=r, quantize=True)
    codes, scales = torch.empty_like(want.codes), torch.empty_like(want.scales)
    s = torch.full_like(x, 7.0) if keep else None
    assert moe.lib().moe_rms_norm(ptr(x), ptr(r), ptr(w), T, H, 1e-6, None, ptr(s), ptr(codes), ptr(scales), None,
                                  stream()) == 0
    assert torch.equal(codes.view(torch.uint8), want.codes.view(torch.uint8)) and torch.equal(scales, want.scales)
    if keep:
        assert torch.equal(s, want.residual)


# dx as a stream of the weights, and in tiles; with dw in one launch and by itself
SIZES = [(8, 264, 136), (40, 2048, 1408), (1000, 520, 1032)]


@pytest.mark.parametrize("T,H,I", SIZES)
@pytest.mark.parametrize("which", ["dx", "dw"])
def test_gated_gradients_one_at_a_time(T, H, I, which):
    x, w, dh = normal(1, T, H), normal(2, 2 * I, H, std=H ** -0.5), normal(3, T, I, std=0.1)
    gu = moe.gated_ffn(x, w, act="gelu", save=True)[1]
    L = moe.lib()
    ws = torch.empty(L.moe_gated_ffn_backward_workspace_size(T, I), dtype=torch.uint8, device="cuda")
    dx = torch.empty_like(x) if which == "dx" else None
    dw = torch.empty_like(w) if which == "dw" else None
    assert L.moe_gated_ffn_backward(ptr(dh), ptr(x), ptr(w), ptr(gu), T, H, I, moe.ACT["gelu"], ptr(dx), ptr(dw),
                                    ptr(ws), ws.numel(), stream()) == 0
    rx, rw, ex, ew = R.gated_grads(dh, x, w, "gelu")
    R.check(*((dx, rx, ex) if which == "dx" else (dw, rw, ew)), which)


@pytest.mark.parametrize("T,K,N", SIZES)
@pytest.mark.parametrize("name", ["none", "silu"])
@pytest.mark.parametrize("which", [("dx",), ("dw",), ("db",), ("dx", "db"), ("dw", "db")])
def test_linear_gradients_some_at_a_time(T, K, N, name, which):
    x, w, dy, b = normal(1, T, K), normal(2, N, K, std=K ** -0.5), normal(3, T, N, std=0.1), normal(4, N, std=0.5)
    z = moe.linear(x, w, bias=b, act=name, save=True)[1]
    L, act = moe.lib(), -1 if name == "none" else moe.ACT[name]
    out = {"dx": torch.empty_like(x), "dw": torch.empty_like(w), "db": torch.empty_like(b)}
    out = {k: v if k in which else None for k, v in out.items()}
    ws = torch.empty(L.moe_linear_backward_workspace_size(T, N, act, int("db" in which)), dtype=torch.uint8,
                     device="cuda")
    assert L.moe_linear_backward(ptr(dy), ptr(x), ptr(w), ptr(z), T, K, N, act, ptr(out["dx"]), ptr(out["dw"]),
                                 ptr(out["db"]), ptr(ws), ws.numel(), stream()) == 0
    rx, rw, rb, ex, ew, eb = R.linear_grads(dy, x, w, b, name)
    for k, ref, bound in (("dx", rx, ex), ("dw", rw, ew), ("db", rb, eb)):
        if k in which:
            R.check(out[k], ref, bound, k)
