"""The dense operators together and around the routed experts: whole blocks
against the oracle's experts and 64-bit dense forms, a training step of a shared
expert against differences, streams, graphs, and waits that give up."""
import numpy as np
import pytest
import torch

import dense_reference as R
import mixture_experts_routed_moe_b200 as moe
from mixture_experts_routed_moe_b200 import inputs as G
from oracle import moe_oracle as O
from parity import ExpertView

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def normal(seed, *shape, std=1.0, mean=0.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").mul_(std).add_(mean).to(BF)


def block_of(wl, seed, Is=192, shared=True):
    W = G.make_weights(wl, seed, device="cuda")
    layer = moe.MoELayer(W["w_gate_up"], W["w_down"], wl.k, W.get("sw_gate_up"), W.get("sw_down"))
    extra = {}
    if shared:
        extra = dict(shared_gate_up=normal(3, 2 * Is, wl.H, std=wl.H ** -0.5),
                     shared_down=normal(4, wl.H, Is, std=Is ** -0.5))
    return moe.MoEBlock(layer, normal(1, wl.H, std=0.2, mean=1.0), G.make_router_weights(wl, seed, device="cuda"),
                        **extra), W


BLOCKS = [G.Workload("block", 64, 256, 256, 8, 2), G.Workload("block", 1, 256, 128, 16, 4),
          G.Workload("block", 301, 512, 256, 16, 4), G.Workload("block", 5, 256, 256, 8, 2, wdtype="e4m3"),
          G.Workload("block", 300, 512, 256, 8, 2, wdtype="e4m3"),
          G.Workload("block", 40, 256, 256, 8, 2, wdtype="e2m1")]


@pytest.mark.parametrize("wl", BLOCKS, ids=lambda w: f"{w.wdtype}-{w.T}")
@pytest.mark.parametrize("shared", [True, False])
def test_block_against_the_oracle(wl, shared):
    """norm -> router -> experts -> shared expert with the routed sum as its
    residual. The oracle routes and runs the experts on the device's own norm
    output; the dense parts are compared in 64 bits."""
    block, W = block_of(wl, 7, shared=shared)
    x, res = normal(11, wl.T, wl.H), normal(12, wl.T, wl.H)
    y, s = block(x, res)
    s_ref, _, n_ref = R.norm(x, block.w_norm, res, block.eps)
    assert torch.equal(s.double(), s_ref)
    fp8 = wl.wdtype == "e4m3"
    n = moe.rms_norm(x, block.w_norm, residual=res, eps=block.eps, quantize=fp8)
    R.check(n.y, n_ref, (R.HALF + 2 * R.NORM) * n_ref.abs(), "norm")
    idx, w, lg = moe.router(n.y, block.w_router, wl.k, logits=True)
    ridx, rw, _ = O.route(lg.cpu().numpy(), wl.k)
    assert np.array_equal(idx.cpu().numpy(), ridx)
    xn = n.y.float().cpu().numpy()
    if fp8:  # value = code * scale: quantising these again gives the same codes
        xn = (n.codes.float().view(wl.T, -1, 128) * n.scales[:, :, None]).reshape(wl.T, wl.H).cpu().numpy()
        routed = O.moe_forward_fp8(xn, ridx, rw, ExpertView(W["w_gate_up"], True), ExpertView(W["sw_gate_up"], True),
                                   ExpertView(W["w_down"], True), ExpertView(W["sw_down"], True))
    elif wl.wdtype == "e2m1":
        routed = O.moe_forward_fp4(xn, ridx, rw, *(W[k].cpu().numpy() for k in
                                                   ("w_gate_up", "sw_gate_up", "w_down", "sw_down")))
    else:
        routed = O.moe_forward(xn, ridx, rw, ExpertView(W["w_gate_up"]), ExpertView(W["w_down"]))
    ref = torch.from_numpy(np.asarray(routed, dtype=np.float64)).cuda()
    if shared:
        h = R.gated(n.y, block.shared_gate_up, "silu")[0]
        ref = ref + h @ block.shared_down.double().t()
    # the experts' own tolerance (5e-3 bf16, 3e-2 FP8), and one bf16 rounding each of h, the routed sum and y
    R.check_fro(y, ref, (3e-2 if fp8 else 5e-3) + 3 * R.HALF / 2, "block")


@pytest.mark.parametrize("T,path", [(5, "decode"), (40, "prefill"), (300, "prefill"), (300, "decode"), (1, "auto")])
def test_quantized_forward_equals_forward_on_its_codes(T, path):
    """Codes and scales that the layer would form itself give the layer's bits:
    x on the e4m3 grid with power-of-two scales quantises to itself."""
    wl = G.Workload("q", T, 512, 256, 8, 2, wdtype="e4m3")
    _, logits = G.make_activations(wl, 3)
    W = G.make_weights(wl, 3, device="cuda")
    codes = normal(5, T, wl.H, std=64.0).float().to(torch.float8_e4m3fn)
    c = codes.view(T, -1, 128)
    c[:, :, 0] = torch.tensor(448.0).to(torch.float8_e4m3fn).cuda()  # each group's largest, so amax / 448 is the scale
    scales = torch.exp2(torch.randint(-6, 3, (T, wl.H // 128), device="cuda").float())
    x = (c.float() * scales[:, :, None]).view(T, wl.H).to(BF)
    idx, w = moe.route(logits.cuda(), wl.k)
    args = (idx, w, W["w_gate_up"], W["w_down"], W["sw_gate_up"], W["sw_down"])
    want, _ = moe.forward(x, *args, path=path)
    got, ws = moe.forward_quantized(codes, scales, *args, path=path)
    assert moe.read_device_status(ws) == 0
    assert torch.equal(got, want)


def test_shared_expert_training_step_against_differences():
    """norm -> gated -> linear + residual, and back: every gradient of the chain
    against central differences of the 64-bit chain."""
    T, H, I = 24, 64, 40
    x, res, wn = normal(1, T, H), normal(2, T, H), normal(3, H, std=0.2, mean=1.0)
    wg, wd, b = normal(4, 2 * I, H, std=H ** -0.5), normal(5, H, I, std=I ** -0.5), normal(6, H, std=0.1)
    dy, ds = normal(7, T, H, std=0.5), normal(8, T, H, std=0.5)
    n = moe.rms_norm(x, wn, residual=res, rstd=True)
    h, gu = moe.gated_ffn(n.y, wg, save=True)
    y = moe.linear(h, wd, bias=b, residual=n.residual)
    # backward: y = linear(h) + s, so dy also reaches the residual stream
    dh, dwd, db = moe.linear_backward(dy, h, wd, bias=True)
    dn, dwg = moe.gated_ffn_backward(dh, n.y, wg, gu)
    dx, dwn = moe.rms_norm_backward(dn, n.residual, wn, n.rstd, dresidual=(dy.float() + ds.float()).to(BF))

    def loss(s, wn, wg, wd, b):
        r = 1 / (s.square().mean(1, keepdim=True) + 1e-6).sqrt()
        z = (s * r * wn) @ wg.t()
        g, u = z[:, :I], z[:, I:]
        out = (g * torch.sigmoid(g) * u) @ wd.t() + b + s
        return (out * dy.double()).sum() + (s * ds.double()).sum()

    at = [t.double() for t in (n.residual, wn, wg, wd, b)]
    rng = np.random.default_rng(0)
    for k, grad in enumerate((dx, dwn, dwg, dwd, db)):
        flat = grad.double().reshape(-1)
        scale = float(flat.square().mean().sqrt())
        for i in rng.choice(flat.numel(), size=min(25, flat.numel()), replace=False):
            e = 2.0 ** -10
            moved = []
            for sgn in (1, -1):
                a = [t.clone() for t in at]
                a[k].reshape(-1)[int(i)] += sgn * e
                moved.append(float(loss(*a)))
            num = (moved[0] - moved[1]) / (2 * e)
            # the chain's bf16 roundings (n, h, dg, du, dn: 2^-8 each of terms of the gradient's size), and e^2
            assert abs(num - float(flat[int(i)])) <= 6 * R.HALF * (abs(num) + scale) + 1e-3


def _ops():
    """Every operator as a call on fixed inputs, returning its outputs."""
    T, H, I = 200, 256, 136
    x, res, wn = normal(1, T, H), normal(2, T, H), normal(3, H, mean=1.0)
    wg, wd, b, dh, dy = (normal(4, 2 * I, H, std=0.06), normal(5, H, I, std=0.08), normal(6, H), normal(7, T, I),
                         normal(8, T, H))
    n = moe.rms_norm(x, wn, residual=res, rstd=True)
    h, gu = moe.gated_ffn(x, wg, save=True)
    _, z = moe.linear(h, wd, bias=b, act="gelu", save=True)
    torch.cuda.synchronize()
    return {
        "rms_norm": lambda **k: list(moe.rms_norm(x, wn, residual=res, quantize=True, rstd=True, **k)),
        "rms_norm_backward": lambda **k: list(moe.rms_norm_backward(dy, n.residual, wn, n.rstd, dresidual=x, **k)),
        "gated_ffn": lambda **k: list(moe.gated_ffn(x, wg, act="gelu", save=True, **k)),
        "gated_ffn_backward": lambda **k: list(moe.gated_ffn_backward(dh, x, wg, gu, **k)),
        "linear": lambda **k: list(moe.linear(h, wd, bias=b, act="silu", residual=res, save=True, **k)),
        "linear_backward": lambda **k: list(moe.linear_backward(dy, h, wd, z, act="gelu", bias=True, **k)),
    }


def _same(a, b):
    return all(torch.equal(u.view(torch.uint8), v.view(torch.uint8)) for u, v in zip(a, b))


@pytest.mark.parametrize("name", ["rms_norm", "rms_norm_backward", "gated_ffn", "gated_ffn_backward", "linear",
                                  "linear_backward"])
def test_streams_and_graphs(name):
    """The same bits on another stream (given or current), from two calls at
    once, and from two graphs captured and replayed several times."""
    op = _ops()[name]
    want = op()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    a, b = op(stream=s1), op(stream=s2)  # may overlap: each call has its own workspace
    with torch.cuda.stream(s2):
        c = op()
    torch.cuda.synchronize()
    assert _same(a, want) and _same(b, want) and _same(c, want)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = op()
        graphs.append((g, out))
    for _ in range(3):
        for g, out in graphs:
            for t in out:
                t.view(torch.uint8).zero_()
            g.replay()
        torch.cuda.synchronize()
        for _, out in graphs:
            assert _same(out, want)


def test_arguments_by_name():
    x, w, wg, wl = normal(1, 3, 64), normal(2, 64), normal(3, 32, 64), normal(4, 24, 64)
    assert torch.equal(moe.rms_norm(x=x, weight=w).y, moe.rms_norm(x, w).y)
    assert torch.equal(moe.gated_ffn(w_gate_up=wg, x=x, act="gelu"), moe.gated_ffn(x, wg, act="gelu"))
    assert torch.equal(moe.linear(w=wl, x=x, stream=torch.cuda.current_stream()), moe.linear(x, wl))


def test_stream_of_another_kind_is_refused():
    x, w = normal(1, 2, 64), normal(2, 64)
    if torch.cuda.device_count() > 1:
        with pytest.raises(ValueError, match="stream is on"):
            moe.rms_norm(x, w, stream=torch.cuda.Stream(device=1))
    with pytest.raises(ValueError, match="is on cpu"):
        moe.rms_norm(x, w.cpu())
    with pytest.raises(moe.MoeError):
        moe.rms_norm(x, w, residual=x, residual_out=x, out=x)  # the two outputs in one buffer


@pytest.mark.parametrize("wl", BLOCKS[:1] + BLOCKS[3:5], ids=lambda w: f"{w.wdtype}-{w.T}")
def test_block_in_a_graph(wl):
    block, _ = block_of(wl, 5)
    x, res = normal(1, wl.T, wl.H), normal(2, wl.T, wl.H)
    block(x, res)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y, s = block(x, res)
    for seed in (8, 9):
        x.copy_(normal(seed, wl.T, wl.H))
        g.replay()
        torch.cuda.synchronize()
        want = block(x, res)
        assert torch.equal(y, want[0]) and torch.equal(s, want[1])


def test_empty_batches():
    H, I = 64, 72
    x, wn, wg, wd = normal(1, 0, H), normal(2, H), normal(3, 2 * I, H), normal(4, H, I)
    n = moe.rms_norm(x, wn, residual=x, rstd=True)
    assert n.y.shape == (0, H) and n.rstd.shape == (0,)
    dx, dw = moe.rms_norm_backward(x, x, wn, n.rstd)
    assert dx.shape == (0, H) and not dw.any()
    h, gu = moe.gated_ffn(x, wg, save=True)
    assert h.shape == (0, I)
    dx, dw = moe.gated_ffn_backward(h, x, wg, gu)
    assert dx.shape == (0, H) and not dw.any()
    y = moe.linear(h, wd, bias=normal(5, H), residual=x)
    assert y.shape == (0, H)
    dh, dw, db = moe.linear_backward(y, h, wd, bias=True)
    assert dh.shape == (0, I) and not dw.any() and not db.any()


@pytest.mark.parametrize("T", [3, 700])
def test_nan_and_infinite_rows_stay_in_their_rows(T):
    """A NaN or an infinity in a token's row reaches that row's outputs only."""
    H, I = 128, 264
    x, wg = normal(1, T, H), normal(2, 2 * I, H, std=0.1)
    wd, b = normal(3, H, I, std=0.1), normal(4, H)
    clean = moe.gated_ffn(x, wg)
    y0 = moe.linear(clean, wd, bias=b, act="gelu")
    bad = x.clone()
    bad[1, 5], bad[2, 7] = float("nan"), float("inf")
    h = moe.gated_ffn(bad, wg)
    y = moe.linear(h, wd, bias=b, act="gelu")
    keep = [0] + list(range(3, T))
    assert torch.equal(h[keep], clean[keep]) and torch.equal(y[keep], y0[keep])
    assert torch.isnan(h[1]).all() and torch.isnan(y[1]).all()


@pytest.mark.parametrize("T", [40, 700])
def test_a_wait_that_gives_up_marks_the_outputs(T):
    """With loads withheld and a 20 ms limit the GEMMs' waits run out: the call
    returns, every output is NaN, and the next call gives the right bits."""
    H, I = 512, 264
    x, wg, wd = normal(1, T, H), normal(2, 2 * I, H, std=0.05), normal(3, H, I, std=0.1)
    want = moe.gated_ffn(x, wg)
    y_want = moe.linear(want, wd)
    torch.cuda.synchronize()
    try:
        moe.set_test_hooks(stall_gate_up_loads=True, wait_limit_ns=20_000_000)
        h, gu = moe.gated_ffn(x, wg, save=True)
        y = moe.linear(want, wd)
        dx, dw, _ = moe.linear_backward(y_want, want, wd)
        torch.cuda.synchronize()
    finally:
        moe.set_test_hooks()
    for t in (h, y, dx, dw):
        assert torch.isnan(t).all()
    assert torch.equal(moe.gated_ffn(x, wg), want) and torch.equal(moe.linear(want, wd), y_want)


def test_offsets_beyond_32_bits():
    """Rows whose element offsets pass 2^31 (and byte offsets 2^32): the last rows
    equal the same rows computed alone."""
    T, H, I = 270_000, 64, 8192  # h: 2.2e9 elements
    x, wg = normal(1, T, H), normal(2, 2 * I, H, std=0.1)
    h = moe.gated_ffn(x, wg)
    want, bound = R.gated(x[-5:], wg, "silu")[::2]
    R.check(h[-5:], want, bound, "h")
    wd, b = normal(3, H, I, std=0.01), normal(4, H)
    y = moe.linear(h, wd, bias=b, residual=x)
    want, _, bound, _ = R.linear(h[-5:], wd, b, "none", x[-5:])
    R.check(y[-5:], want, bound, "y")
    w = normal(5, I, std=0.1, mean=1.0)
    n = moe.rms_norm(h, w, residual=h, residual_out=h, quantize=True)
    few = moe.rms_norm(h[-5:].contiguous(), w, quantize=True)  # (h holds the sums now)
    assert torch.equal(n.y[-5:], few.y) and torch.equal(n.scales[-5:], few.scales)
    assert torch.equal(n.codes[-5:].view(torch.uint8), few.codes.view(torch.uint8))
