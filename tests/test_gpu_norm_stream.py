"""What the RMS norm hands on as the residual stream: through the C entry point with and
without a residual, into a buffer of its own or the input's, and the binding's result
where the normalised rows take the input's place."""
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


def c_norm(x, residual, w, y, residual_out, codes=None, scales=None):
    at = [None if t is None else t.data_ptr() for t in (x, residual, w, y, residual_out, codes, scales)]
    status = moe.lib().moe_rms_norm(*at[:3], *x.shape, 1e-6, *at[3:], None, torch.cuda.current_stream().cuda_stream)
    assert status == 0
    torch.cuda.synchronize()


# one size at least for each form of the kernel: a warp or a block a row, 1 to 8 vectors a
# thread, few rows and many, with codes the lean forms too; rows that fill no vector group
STREAM = [(5, 64), (3, 512), (33, 1024), (129, 2040), (700, 4096), (3, 7168), (700, 7168), (400, 8200), (3, 16392)]
STREAM_CODES = [(5, 256), (3, 512), (33, 1024), (129, 2048), (700, 2048), (400, 5120), (3, 7168), (400, 6144),
                (400, 7168), (400, 8192), (300, 8320), (3, 16512)]


@pytest.mark.parametrize("T,H,quantize", [(T, H, False) for T, H in STREAM] + [(T, H, True) for T, H in STREAM_CODES])
@pytest.mark.parametrize("with_residual", [False, True])
def test_residual_out_holds_the_stream(T, H, quantize, with_residual):
    """s = x + residual, or x without a residual, into a buffer of its own; the other
    outputs are those of a call that does not ask for it."""
    x, w = normal(T, T, H), normal(H, H, std=0.2, mean=1.0)
    r = normal(T + 1, T, H) if with_residual else None
    want = moe.rms_norm(x, w, residual=r, quantize=quantize)
    kept = x.clone()
    around = torch.full((T + 2, H), 7.0, device="cuda", dtype=BF)
    y = torch.full_like(x, 7.0)
    codes = torch.empty((T, H), device="cuda", dtype=torch.float8_e4m3fn) if quantize else None
    scales = torch.empty((T, H // 128), device="cuda") if quantize else None
    c_norm(x, r, w, y, around[1:T + 1], codes, scales)
    s = R.norm(x, w, r, 1e-6)[0]
    assert torch.equal(around[1:T + 1].double(), s)
    assert bool((around[0] == 7).all()) and bool((around[T + 1] == 7).all())
    assert torch.equal(x, kept) and torch.equal(y, want.y)
    if quantize:
        assert torch.equal(codes.view(torch.uint8), want.codes.view(torch.uint8))
        assert torch.equal(scales, want.scales)


@pytest.mark.parametrize("T,H", [(5, 64), (700, 4096), (400, 8200)])
def test_stream_without_a_residual_in_place(T, H):
    """residual_out may be x, and y may be x while the stream goes elsewhere."""
    x, w = normal(T, T, H), normal(H, H, std=0.2, mean=1.0)
    want = moe.rms_norm(x, w).y
    a, y = x.clone(), torch.empty_like(x)
    c_norm(a, None, w, y, a)
    assert torch.equal(a, x) and torch.equal(y, want)
    a, s = x.clone(), torch.full_like(x, 7.0)
    c_norm(a, None, w, a, s)
    assert torch.equal(s, x) and torch.equal(a, want)


def test_stream_is_not_claimed_where_y_took_its_place():
    """Without a residual the stream is x itself; in place it is gone, so none is handed on."""
    x, w = normal(1, 6, 64), normal(2, 64, mean=1.0)
    want = moe.rms_norm(x, w, rstd=True)
    assert want.residual is x
    for name in (lambda t: t, lambda t: t.view(6, 64)):  # the same memory by either name
        a = x.clone()
        got = moe.rms_norm(a, w, rstd=True, out=name(a))
        assert torch.equal(got.y, want.y) and torch.equal(got.rstd, want.rstd)
        assert got.residual is None
        with pytest.raises(TypeError, match="s must be"):
            moe.rms_norm_backward(x, got.residual, w, got.rstd)
    a, r = x.clone(), normal(3, 6, 64)
    got = moe.rms_norm(a, w, residual=r, out=a)  # with a residual the stream has a buffer of its own
    assert torch.equal(got.residual.double(), R.norm(x, w, r, 1e-6)[0])
    none = x[:0]
    assert moe.rms_norm(none, w).residual is none and moe.rms_norm(none, w, out=none).residual is none
