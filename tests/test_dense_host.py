"""Host-side refusals of the dense operators: the C entry points reject bad sizes,
pointers, aliases and workspaces before any launch, and the binding rejects
tensors the library could not read safely (no GPU needed)."""
import math

import pytest
import torch

import mixture_experts_routed_moe_b200 as moe
from mixture_experts_routed_moe_b200 import _build

BAD, SPACE = -1, -4
BF = torch.bfloat16


def at(i):
    """Aligned addresses 1 GB apart; never dereferenced by the host checks."""
    return (1 << 40) + (i << 30)


@pytest.fixture(scope="module")
def L():
    _build.build()
    return moe.lib()


def call(fn, base, **change):
    args = dict(base, **change)
    return fn(*args.values())


def norm_args():
    return dict(x=at(0), residual=at(1), weight=at(2), T=4, H=256, eps=1e-6, y=at(3), residual_out=at(4), codes=at(5),
                scales=at(6), rstd=at(7), stream=None)


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(T=(1 << 30) + 1), dict(H=0), dict(H=100), dict(H=65544), dict(eps=0.0), dict(eps=-1.0), dict(eps=math.inf),
    dict(eps=math.nan), dict(x=None), dict(weight=None), dict(codes=None), dict(scales=None), dict(H=264),
    dict(y=None, codes=None, scales=None), dict(x=at(0) + 8), dict(residual=at(1) + 2), dict(weight=at(2) + 8),
    dict(y=at(3) + 4), dict(residual_out=at(4) + 8), dict(codes=at(5) + 1), dict(scales=at(6) + 2),
    dict(rstd=at(7) + 1), dict(y=at(0) + 16), dict(residual_out=at(3)), dict(codes=at(0)), dict(rstd=at(1)),
    dict(scales=at(5)), dict(y=at(2)), dict(residual_out=at(1) + 512)])
def test_norm_refusals(L, bad):
    assert call(L.moe_rms_norm, norm_args(), **bad) == BAD


def test_empty_batches_are_no_ops(L):
    assert call(L.moe_rms_norm, norm_args(), T=0, x=None, y=None) == 0
    assert call(L.moe_gated_ffn, gated_args(), T=0, x=None) == 0
    assert call(L.moe_linear, linear_args(), T=0, x=None, y=None) == 0


def norm_bwd_args(L):
    return dict(dy=at(0), s=at(1), weight=at(2), rstd=at(3), dresidual=at(4), T=4, H=256, dx=at(5), dw=at(6),
                workspace=at(7), bytes=L.moe_rms_norm_backward_workspace_size(4, 256), stream=None)


def test_norm_backward_refusals(L):
    a = norm_bwd_args(L)
    for bad in (dict(T=-1), dict(H=100), dict(dy=None), dict(s=None), dict(weight=None), dict(rstd=None), dict(dx=None),
                dict(dw=None), dict(workspace=None), dict(dy=at(0) + 8), dict(workspace=at(7) + 128), dict(dx=at(1)),
                dict(dx=at(0) + 16), dict(dw=at(2)), dict(dw=at(5)), dict(workspace=at(4)), dict(rstd=at(3) + 2)):
        assert call(L.moe_rms_norm_backward, a, **bad) == BAD, bad
    assert call(L.moe_rms_norm_backward, a, bytes=a["bytes"] - 1) == SPACE
    assert L.moe_rms_norm_backward_workspace_size(4, 100) == 0
    assert L.moe_rms_norm_backward_workspace_size(-1, 256) == 0
    # one fp32 row for each block of the first pass: two of 512 threads on each of 148 SMs
    assert L.moe_rms_norm_backward_workspace_size(10 ** 6, 4096) == 296 * 4096 * 4


def gated_args():
    return dict(x=at(0), w=at(1), T=4, H=64, I=128, act=0, h=at(2), gu=at(3), stream=None)


@pytest.mark.parametrize("bad", [dict(T=-1), dict(H=12), dict(I=4), dict(I=(1 << 20) + 8), dict(act=3), dict(act=-1),
                                 dict(x=None), dict(w=None), dict(h=None), dict(x=at(0) + 8), dict(gu=at(3) + 8),
                                 dict(h=at(0)), dict(h=at(1) + 64), dict(gu=at(2)), dict(gu=at(1))])
def test_gated_refusals(L, bad):
    assert call(L.moe_gated_ffn, gated_args(), **bad) == BAD


def test_gated_backward_refusals(L):
    need = L.moe_gated_ffn_backward_workspace_size(4, 128)
    assert need >= 4 * 256 * 2
    a = dict(dh=at(0), x=at(1), w=at(2), gu=at(3), T=4, H=64, I=128, act=0, dx=at(4), dw=at(5), workspace=at(6),
             bytes=need, stream=None)
    for bad in (dict(T=-1), dict(H=12), dict(act=-1), dict(dh=None), dict(gu=None), dict(workspace=None),
                dict(workspace=at(6) + 16), dict(dx=at(1)), dict(dx=at(0)), dict(dw=at(2)), dict(dw=at(4)),
                dict(workspace=at(3)), dict(dx=at(4) + 2)):
        assert call(L.moe_gated_ffn_backward, a, **bad) == BAD, bad
    assert call(L.moe_gated_ffn_backward, a, bytes=need - 1) == SPACE
    assert call(L.moe_gated_ffn_backward, a, dx=None, dw=None) == 0  # nothing asked for
    assert L.moe_gated_ffn_backward_workspace_size(4, 12) == 0


def linear_args():
    return dict(x=at(0), w=at(1), bias=at(2), residual=at(3), T=4, K=64, N=128, act=-1, y=at(4), z=at(5), stream=None)


@pytest.mark.parametrize("bad", [dict(T=-1), dict(K=12), dict(N=0), dict(act=3), dict(act=-2), dict(x=None),
                                 dict(w=None), dict(y=None), dict(bias=at(2) + 2), dict(residual=at(3) + 8),
                                 dict(y=at(0)), dict(y=at(3) + 16), dict(z=at(4)), dict(z=at(3)), dict(y=at(2))])
def test_linear_refusals(L, bad):
    assert call(L.moe_linear, linear_args(), **bad) == BAD


def test_linear_backward_refusals(L):
    size = L.moe_linear_backward_workspace_size
    need = size(4, 128, 1, 1)
    assert need > size(4, 128, 1, 0) > size(4, 128, -1, 0) > 0
    assert size(4, 12, 0, 0) == 0 and size(4, 128, 5, 0) == 0
    a = dict(dy=at(0), x=at(1), w=at(2), z=at(3), T=4, K=64, N=128, act=1, dx=at(4), dw=at(5), db=at(6),
             workspace=at(7), bytes=need, stream=None)
    for bad in (dict(T=-1), dict(K=12), dict(N=12), dict(act=3), dict(z=None), dict(dy=None), dict(dx=at(0)),
                dict(dw=at(2)), dict(db=at(5)), dict(workspace=at(1)), dict(workspace=at(7) + 8), dict(dx=at(4) + 8)):
        assert call(L.moe_linear_backward, a, **bad) == BAD, bad
    assert call(L.moe_linear_backward, a, bytes=need - 1) == SPACE
    assert call(L.moe_linear_backward, a, dx=None, dw=None, db=None, bytes=size(4, 128, 1, 0)) == 0


def test_binding_refuses_what_the_library_cannot_see():
    x, w = torch.zeros((4, 64), dtype=BF), torch.zeros((64,), dtype=BF)
    wl, wg = torch.zeros((128, 64), dtype=BF), torch.zeros((256, 64), dtype=BF)
    for f in (lambda: moe.rms_norm(x, w), lambda: moe.gated_ffn(x, wg), lambda: moe.linear(x, wl),
              lambda: moe.rms_norm_backward(x, x, w, torch.zeros(4)),
              lambda: moe.gated_ffn_backward(torch.zeros((4, 128), dtype=BF), x, wg, torch.zeros((4, 256))),
              lambda: moe.linear_backward(torch.zeros((4, 128), dtype=BF), x, wl)):
        with pytest.raises(ValueError, match="must be on a CUDA device"):
            f()
    with pytest.raises(ValueError, match="x: dtype"):
        moe.rms_norm(x.float(), w)
    with pytest.raises(ValueError, match="x: 1-D"):
        moe.linear(w, wl)
    with pytest.raises(ValueError, match="x must be contiguous"):
        moe.gated_ffn(torch.zeros((64, 4), dtype=BF).t(), wg)
    with pytest.raises(TypeError):
        moe.linear(None, wl)
    with pytest.raises(ValueError, match="act"):
        moe.gated_ffn(x, wg, act="none")
    with pytest.raises(ValueError, match="act"):
        moe.linear(x, wl, act="tanh")


def test_quantized_forward_refusals(L):
    """moe_forward_quantized takes e4m3 experts only, and needs codes and scales."""
    import ctypes

    args = [at(i) for i in range(1, 10)]

    def run(s, codes, scales, need=1 << 40):
        return L.moe_forward_quantized(ctypes.byref(s), codes, scales, *args[2:8], at(20), at(21), need, None)

    s = moe.make_shape(4, 256, 256, 8, 2, "e4m3")
    assert run(s, None, at(1)) == BAD and run(s, at(0), None) == BAD
    assert run(s, at(0) + 8, at(1)) == BAD and run(s, at(0), at(1) + 2) == BAD
    assert run(s, at(0), at(1), 16) == SPACE
    for other in ("bf16", "e2m1"):
        assert run(moe.make_shape(4, 256, 256, 8, 2, other), at(0), at(1)) == -2
    assert run(moe.make_shape(4, 100, 256, 8, 2, "e4m3"), at(0), at(1)) == BAD
    assert run(moe.make_shape(0, 256, 256, 8, 2, "e4m3"), None, None) == 0


def test_block_and_quantized_binding_refusals():
    f8 = torch.float8_e4m3fn
    T, H, I, E, k = 4, 256, 256, 8, 2
    idx, w = torch.zeros((T, k), dtype=torch.int32), torch.zeros((T, k))
    ok = dict(codes=torch.zeros((T, H), dtype=f8), scales=torch.zeros((T, H // 128)), topk_idx=idx, topk_w=w,
              w_gate_up=torch.zeros((E, 2 * I, H), dtype=f8), w_down=torch.zeros((E, H, I), dtype=f8),
              sw_gate_up=torch.zeros((E, 2 * I // 128, H // 128), dtype=torch.uint8),
              sw_down=torch.zeros((E, H // 128, I // 128), dtype=torch.uint8))
    for bad, msg in ((dict(codes=torch.zeros((T, H), dtype=BF)), "codes: dtype"),
                     (dict(scales=torch.zeros((T, H // 128 + 1))), "scales: shape"),
                     (dict(w_gate_up=torch.zeros((E, 2 * I, H), dtype=BF), w_down=torch.zeros((E, H, I), dtype=BF),
                           sw_gate_up=None, sw_down=None), "need e4m3 experts"),
                     (dict(), "CUDA device")):
        with pytest.raises(ValueError, match=msg):
            moe.forward_quantized(**dict(ok, **bad))
    layer = moe.MoELayer(ok["w_gate_up"], ok["w_down"], k)
    with pytest.raises(ValueError, match="both shared_gate_up and shared_down"):
        moe.MoEBlock(layer, torch.ones(H, dtype=BF), torch.zeros((E, H), dtype=BF), shared_down=torch.zeros((H, I)))
