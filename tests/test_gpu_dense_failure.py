"""Waits of the dense GEMMs that give up, without a fault: one CTA of each cluster issues
no loads, so that its own waits and its peers' run into a short limit. Each call returns
with NaN in what it did not compute, and the next one gives the right bits."""
import time

import pytest
import torch

import mixture_experts_routed_moe_b200 as moe

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
LIMIT_NS = 20_000_000  # 20 ms


def normal(seed, *shape, std=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").mul_(std).to(BF)


def stalled(f):
    """f() with the loads withheld, and the seconds it took."""
    torch.cuda.synchronize()
    try:
        moe.set_test_hooks(stall_gate_up_loads=True, wait_limit_ns=LIMIT_NS)
        t = time.perf_counter()
        out = f()
        torch.cuda.synchronize()
        return out, time.perf_counter() - t
    finally:
        moe.set_test_hooks()


# clusters of eight, four, two and one; one token tile and several; whole and half SMs
SPLIT = [(40, 7168, 136), (33, 2048, 1408), (64, 2048, 7168), (100, 512, 4096), (333, 2040, 1000), (40, 64, 264)]


@pytest.mark.parametrize("T,K,N", SPLIT)
@pytest.mark.parametrize("op", ["linear", "gated", "dx"])
def test_a_cluster_whose_partials_never_come(T, K, N, op):
    x, w = normal(1, T, K), normal(2, 2 * N if op == "gated" else N, K, std=K ** -0.5)
    d = normal(3, T, N)
    call = {"linear": lambda: moe.linear(x, w), "gated": lambda: moe.gated_ffn(x, w),
            "dx": lambda: moe.linear_backward(d, x, w)[0]}[op]
    want = call()
    for _ in range(2):
        got, seconds = stalled(call)
        assert torch.isnan(got).all()
        assert seconds < 1.0  # the short limit ended the waits
        assert torch.equal(call(), want)


# tiles of CTA pairs, of which the leader's loads are on their way when it gives up, and of
# single CTAs; fewer K steps than the ring has stages, so that the producer is done by then, and more
TILES = [(4096, 2048, 1408), (4096, 136, 2048), (1000, 520, 2056), (700, 64, 520), (2050, 2048, 4104)]


@pytest.mark.parametrize("T,K,N", TILES)
@pytest.mark.parametrize("op", ["linear", "gated", "backward"])
def test_tiles_whose_loads_never_come(T, K, N, op):
    x, w = normal(1, T, K), normal(2, 2 * N if op == "gated" else N, K, std=K ** -0.5)
    d = normal(3, T, N)
    call = {"linear": lambda: [moe.linear(x, w, residual=d)], "gated": lambda: [moe.gated_ffn(x, w)],
            "backward": lambda: list(moe.linear_backward(d, x, w)[:2])}[op]
    want = call()
    for _ in range(2):
        got, seconds = stalled(call)
        assert all(bool(torch.isnan(t).all()) for t in got)
        assert seconds < 1.0
        assert all(torch.equal(a, b) for a, b in zip(call(), want))


@pytest.mark.parametrize("T,H,I", [(40, 512, 264), (333, 2040, 1000), (700, 64, 520), (4096, 136, 2048)])
@pytest.mark.parametrize("name", ["silu", "gelu", "relu"])
def test_kept_pre_activations_are_marked_too(T, H, I, name):
    """Through the C entry points, into buffers that held finite numbers: with the output, g
    and u and z are NaN, so that no gradient is formed of what was never computed."""
    x, wg, wd = normal(1, T, H), normal(2, 2 * I, H, std=H ** -0.5), normal(3, I, H, std=H ** -0.5)
    h, y, z = (torch.ones((T, I), device="cuda", dtype=BF) for _ in range(3))
    gu = torch.ones((T, 2 * I), device="cuda")
    L, act, st = moe.lib(), moe.ACT[name], torch.cuda.current_stream().cuda_stream

    def both():
        assert L.moe_gated_ffn(x.data_ptr(), wg.data_ptr(), T, H, I, act, h.data_ptr(), gu.data_ptr(), st) == 0
        assert L.moe_linear(x.data_ptr(), wd.data_ptr(), None, None, T, H, I, act, y.data_ptr(), z.data_ptr(), st) == 0

    both()
    want = [t.clone() for t in (h, gu, y, z)]
    stalled(both)
    for t in (h, gu, y, z):
        assert torch.isnan(t).all()
    both()
    assert all(torch.equal(a, b) for a, b in zip((h, gu, y, z), want))
