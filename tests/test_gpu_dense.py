"""The dense operators on the GPU against their 64-bit forms: the RMS norm with
the residual, the gated projection, the linear projection, forward and backward,
at the sizes where tiles, clusters and vectors end, and a whole block of them."""
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


# ---- RMS norm ---------------------------------------------------------------

NORM_SIZES = [(1, 2048), (1, 8), (3, 64), (129, 128), (5, 1024), (7, 1032), (33, 2040), (64, 4096), (2, 7168),
              (301, 8192), (3, 8200), (2, 16384), (2, 32776), (1, 65536)]


# batches whose rows outnumber the blocks, at widths with 1, 2 and 4 vectors a thread
NORM_MANY = [(1500, 1032), (2500, 2048), (1000, 4096), (1203, 4104), (700, 7168), (801, 8192), (611, 8200),
             (500, 16384)]


@pytest.mark.parametrize("T,H", NORM_SIZES + NORM_MANY)
@pytest.mark.parametrize("residual", [False, True])
def test_rms_norm(T, H, residual):
    x, w = normal(T + H, T, H), normal(H, H, std=0.2, mean=1.0)
    r = normal(T * 3 + H, T, H, std=2.0) if residual else None
    n = moe.rms_norm(x, w, residual=r, eps=1e-5, rstd=True)
    s, rs, y = R.norm(x, w, r, 1e-5)
    assert torch.equal(n.residual.double(), s)
    assert torch.allclose(n.rstd.double(), rs, rtol=R.NORM, atol=0)
    R.check(n.y, y, (R.HALF + 2 * R.NORM) * y.abs(), "y")


@pytest.mark.parametrize("T,H", [(1, 128), (16, 2048), (77, 7168), (3, 1152), (130, 4096), (1, 65536),
                                 (2500, 2048), (700, 7168), (500, 16384),
                                 (700, 4224), (500, 5120), (1300, 1024), (900, 2048), (1500, 1152), (800, 4096),
                                 (400, 5248), (390, 6144), (333, 8192), (310, 8320)])
@pytest.mark.parametrize("residual", [True, False])
def test_rms_norm_codes(T, H, residual):
    x, w, r = normal(1, T, H), normal(2, H, std=0.2, mean=1.0), normal(3, T, H)
    x[0, :128] = 0
    r[0, :128] = 0  # an all-zero group: scale 1, codes 0
    r = r if residual else None
    n = moe.rms_norm(x, w, residual=r, eps=1e-6, quantize=True)
    plain = moe.rms_norm(x, w, residual=r, eps=1e-6)
    assert torch.equal(n.y, plain.y) and torch.equal(n.residual, plain.residual)
    _, _, y = R.norm(x, w, r, 1e-6)
    g = y.view(T, H // 128, 128)
    amax = g.abs().amax(2)
    ref = torch.where(amax > 0, amax / 448, torch.ones_like(amax))
    assert torch.allclose(n.scales.double(), ref, rtol=3 * R.NORM, atol=0)
    assert float(n.scales[0, 0]) == 1.0 and not n.codes[0, :128].float().any()
    # half a step of e4m3: 2^-4 of the value, and 2^-10 of the scale below the smallest normal
    got = n.codes.float().view(T, H // 128, 128).double() * n.scales.double()[:, :, None]
    bound = (2.0 ** -4 + 4 * R.NORM) * g.abs() + 2.0 ** -10 * ref[:, :, None] * (1 + 4 * R.NORM)
    R.check(got, g, bound, "codes")


@pytest.mark.parametrize("H", [512, 2048, 7168, 8192, 16384])
def test_rms_norm_rows_do_not_depend_on_the_batch(H):
    """A row's result is the same bits alone and among many rows."""
    x, r, w = normal(1, 1000, H), normal(2, 1000, H), normal(3, H, mean=1.0)
    many = moe.rms_norm(x, w, residual=r, rstd=True)
    few = moe.rms_norm(x[990:993].contiguous(), w, residual=r[990:993].contiguous(), rstd=True)
    assert torch.equal(few.y, many.y[990:993]) and torch.equal(few.rstd, many.rstd[990:993])


def test_rms_norm_small_and_large_rows():
    """A zero row gives zeros (eps carries the root), rows near the ends of
    fp32's squares keep their scale, and a NaN stays in its row."""
    H = 512
    x = normal(5, 6, H)
    x[1] = 0
    x[2] *= 1e-15
    x[3] *= 1e15
    x[4, 7] = float("nan")
    w = torch.ones(H, dtype=BF, device="cuda")
    n = moe.rms_norm(x, w, eps=1e-6, quantize=True)
    _, _, y = R.norm(x, w, None, 1e-6)
    keep = [0, 1, 2, 3, 5]
    R.check(n.y[keep], y[keep], (R.HALF + 2 * R.NORM) * y[keep].abs(), "y")
    assert not n.y[1].any() and torch.isnan(n.y[4]).all()
    assert (n.scales[1] == 1).all()


def test_rms_norm_in_place():
    x, r, w = normal(1, 9, 1024), normal(2, 9, 1024), normal(3, 1024, mean=1.0)
    want = moe.rms_norm(x, w, residual=r)
    x2, r2 = x.clone(), r.clone()
    got = moe.rms_norm(x2, w, residual=r2, out=x2, residual_out=r2)
    assert got.y is x2 and got.residual is r2
    assert torch.equal(x2, want.y) and torch.equal(r2, want.residual)


@pytest.mark.parametrize("T,H", [(1, 8), (1, 2048), (2, 64), (297, 512), (700, 2040), (64, 4096), (33, 7168), (3, 8200),
                                 (1000, 2048), (5, 16384), (3, 65536)] + NORM_MANY)
@pytest.mark.parametrize("residual", [False, True])
def test_rms_norm_backward(T, H, residual):
    s, w, dy = normal(T, T, H, std=1.5), normal(H, H, std=0.2, mean=1.0), normal(T + 1, T, H, std=0.1)
    dr = normal(T + 2, T, H, std=0.1) if residual else None
    n = moe.rms_norm(s, w, eps=1e-5, rstd=True)
    dx, dw = moe.rms_norm_backward(dy, s, w, n.rstd, dresidual=dr)
    rx, rw, ex, ew = R.norm_grads(dy, s, w, 1e-5, dr)
    R.check(dx, rx, ex, "dx")
    R.check(dw, rw, ew, "dw")
    again = moe.rms_norm_backward(dy, s, w, n.rstd, dresidual=dr)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


def test_rms_norm_gradient_against_differences():
    """dx and dw agree with central differences of the 64-bit form."""
    T, H = 3, 64
    s, w, dy = normal(1, T, H), normal(2, H, std=0.2, mean=1.0), normal(3, T, H)
    n = moe.rms_norm(s, w, eps=1e-2, rstd=True)
    dx, dw = moe.rms_norm_backward(dy, s, w, n.rstd)

    def loss(s64, w64):
        r = 1 / (s64.square().mean(1, keepdim=True) + 1e-2).sqrt()
        return float((s64 * r * w64 * dy.double()).sum())

    e = 2.0 ** -12
    for i in range(0, H, 9):
        d = torch.zeros(T, H, dtype=torch.float64, device="cuda")
        d[1, i] = e
        num = (loss(s.double() + d, w.double()) - loss(s.double() - d, w.double())) / (2 * e)
        # half a step of bf16, and the differences' own error of order e^2
        assert abs(num - float(dx[1, i])) <= R.HALF * abs(num) + 1e-4
        d = torch.zeros(H, dtype=torch.float64, device="cuda")
        d[i] = e
        num = (loss(s.double(), w.double() + d) - loss(s.double(), w.double() - d)) / (2 * e)
        assert abs(num - float(dw[i])) <= R.HALF * abs(num) + 1e-4


# ---- gated projection -------------------------------------------------------

GATED = [(1, 8, 8), (1, 2048, 1408), (2, 64, 64), (16, 72, 200), (17, 2040, 1000), (32, 7168, 264), (64, 512, 72),
         (65, 128, 136), (128, 64, 8), (129, 1000, 520), (200, 264, 1032), (333, 2040, 1000), (1000, 520, 2056),
         (2500, 128, 4104), (4096, 256, 1408)]


@pytest.mark.parametrize("T,H,I", GATED)
@pytest.mark.parametrize("name", ["silu", "gelu", "relu"])
def test_gated_ffn(T, H, I, name):
    x, w = normal(T + I, T, H), normal(H + I, 2 * I, H, std=H ** -0.5)
    h, gu = moe.gated_ffn(x, w, act=name, save=True)
    ref, z, bound, ez = R.gated(x, w, name)
    R.check(gu, z, ez, "gu")
    R.check(h, ref, bound, "h")
    assert torch.equal(moe.gated_ffn(x, w, act=name), h)


@pytest.mark.parametrize("T,H,I", GATED)
def test_gated_ffn_backward(T, H, I):
    name = ["silu", "gelu", "relu"][(T + I) % 3]
    x, w, dh = normal(T, T, H), normal(H, 2 * I, H, std=H ** -0.5), normal(I, T, I, std=0.1)
    _, gu = moe.gated_ffn(x, w, act=name, save=True)
    dx, dw = moe.gated_ffn_backward(dh, x, w, gu, act=name)
    rx, rw, ex, ew = R.gated_grads(dh, x, w, name)
    R.check(dx, rx, ex, "dx")
    R.check(dw, rw, ew, "dw")
    # two roundings of 2^-8 at most each, independent: well under 5e-3 in norm
    R.check_fro(dx, rx, 5e-3, "dx")
    R.check_fro(dw, rw, 5e-3, "dw")


# ---- linear projection ------------------------------------------------------

LINEAR = [(1, 8, 8), (1, 1408, 2048), (3, 200, 72), (16, 2048, 7168), (33, 72, 1000), (64, 2056, 136), (65, 64, 64),
          (130, 520, 264), (256, 1000, 2040), (777, 136, 520), (2050, 264, 4104), (4096, 768, 2048)]


@pytest.mark.parametrize("T,K,N", LINEAR)
@pytest.mark.parametrize("name,bias,residual", [("none", False, False), ("none", True, True), ("silu", True, False),
                                                ("gelu", False, True), ("relu", True, True)])
def test_linear(T, K, N, name, bias, residual):
    x, w = normal(T + K, T, K), normal(K + N, N, K, std=K ** -0.5)
    b = normal(N, N, std=0.5) if bias else None
    r = normal(T, T, N) if residual else None
    y, z = moe.linear(x, w, bias=b, act=name, residual=r, save=True)
    ref, zr, bound, ez = R.linear(x, w, b, name, r)
    R.check(y, ref, bound, "y")
    if name == "none":
        assert z is None
    else:
        R.check(z, zr, ez + R.HALF * (zr.abs() + ez), "z")
    assert torch.equal(moe.linear(x, w, bias=b, act=name, residual=r), y)
    if residual:
        r2 = r.clone()
        assert torch.equal(moe.linear(x, w, bias=b, act=name, residual=r2, out=r2), y)


@pytest.mark.parametrize("T,K,N", LINEAR)
@pytest.mark.parametrize("name,bias", [("none", False), ("none", True), ("gelu", True), ("silu", False)])
def test_linear_backward(T, K, N, name, bias):
    x, w, dy = normal(T, T, K), normal(N, N, K, std=K ** -0.5), normal(K, T, N, std=0.1)
    b = normal(N, N, std=0.5) if bias else None
    _, z = moe.linear(x, w, bias=b, act=name, save=True)
    dx, dw, db = moe.linear_backward(dy, x, w, z, act=name, bias=bias)
    rx, rw, rb, ex, ew, eb = R.linear_grads(dy, x, w, b, name)
    R.check(dx, rx, ex, "dx")
    R.check(dw, rw, ew, "dw")
    R.check_fro(dx, rx, 5e-3, "dx")
    R.check_fro(dw, rw, 5e-3, "dw")
    if bias:
        R.check(db, rb, eb, "db")
    else:
        assert db is None


# ---- one token --------------------------------------------------------------

# four, eight and sixteen warps to a row, a K below one load a lane, ends inside a lane's, a
# warp's and a batch's loads, outputs that end inside a unit, and large weights
ONE = [(8, 8), (16, 4104), (264, 72), (1032, 8), (1000, 2040), (2056, 1032), (2048, 8192), (4096, 8), (4104, 24),
       (8200, 520), (7168, 2048), (16392, 40), (24584, 2056)]


@pytest.mark.parametrize("K,N", ONE)
@pytest.mark.parametrize("name,bias,residual,save", [("none", False, False, False), ("none", True, True, False),
                                                     ("gelu", True, True, True), ("relu", False, True, True)])
def test_linear_one_token(K, N, name, bias, residual, save):
    x, w = normal(K, 1, K), normal(K + N, N, K, std=K ** -0.5)
    b = normal(N, N, std=0.5) if bias else None
    r = normal(N + 1, 1, N) if residual else None
    around = torch.full((3, N), 7.0, device="cuda", dtype=BF)
    out = moe.linear(x, w, bias=b, act=name, residual=r, out=around[1:2], save=save)
    z = out[1] if save else None
    ref, zr, bound, ez = R.linear(x, w, b, name, r)
    R.check(around[1:2], ref, bound, "y")
    assert bool((around[0] == 7).all()) and bool((around[2] == 7).all())
    if save:
        R.check(z, zr, ez + R.HALF * (zr.abs() + ez), "z")


@pytest.mark.parametrize("K,N", ONE)
@pytest.mark.parametrize("name,save", [("silu", False), ("gelu", True)])
def test_gated_one_token(K, N, name, save):
    x, w = normal(K, 1, K), normal(K + N, 2 * N, K, std=K ** -0.5)
    around = torch.full((3, N), 7.0, device="cuda", dtype=BF)
    got = moe.gated_ffn(x, w, act=name, out=around[1:2], save=save)
    ref, z, bound, ez = R.gated(x, w, name)
    R.check(around[1:2], ref, bound, "h")
    assert bool((around[0] == 7).all()) and bool((around[2] == 7).all())
    if save:
        R.check(got[1], z, ez, "gu")


def test_one_token_keeps_a_bad_row_to_its_output():
    x, w = normal(1, 1, 1000), normal(2, 520, 1000, std=0.03)
    y = moe.linear(x, w)
    w[77, 999] = float("nan")
    w[130, 0] = float("inf")
    bad = moe.linear(x, w)
    rest = torch.ones(520, dtype=torch.bool, device="cuda")
    rest[77] = rest[130] = False
    assert bool(bad[0, 77].isnan()) and bool(bad[0, 130].isinf())
    assert torch.equal(bad[:, rest], y[:, rest])


# ---- a few tokens -----------------------------------------------------------

# the group of eight tokens that ends, K and N as above, weights on either side of the rules
# between the forms; 16-byte rows and bases as well as 32-byte ones
FEW = [(2, 8, 8), (5, 40, 24), (7, 1408, 2048), (8, 2056, 1032), (9, 16, 4104), (12, 4096, 136), (15, 7168, 264),
       (16, 2048, 9480), (16, 5120, 5000), (17, 1032, 520), (23, 8192, 72), (24, 2048, 4736), (25, 2048, 1408)]


@pytest.mark.parametrize("T,K,N", FEW)
@pytest.mark.parametrize("shift", [0, 8])
@pytest.mark.parametrize("name,bias,residual,save", [("none", False, False, False), ("silu", True, True, True)])
def test_linear_few_tokens(T, K, N, shift, name, bias, residual, save):
    x, w = normal(T, T * K + shift)[shift:].view(T, K), normal(K + N, N * K + shift, std=K ** -0.5)[shift:].view(N, K)
    b = normal(N, N, std=0.5) if bias else None
    r = normal(N + 1, T, N) if residual else None
    around = torch.full((T + 2, N), 7.0, device="cuda", dtype=BF)
    out = moe.linear(x, w, bias=b, act=name, residual=r, out=around[1:T + 1], save=save)
    ref, zr, bound, ez = R.linear(x, w, b, name, r)
    R.check(around[1:T + 1], ref, bound, "y")
    assert bool((around[0] == 7).all()) and bool((around[T + 1] == 7).all())
    if save:
        R.check(out[1], zr, ez + R.HALF * (zr.abs() + ez), "z")
    if residual:
        assert torch.equal(moe.linear(x, w, bias=b, act=name, residual=r, out=r), around[1:T + 1])


@pytest.mark.parametrize("T,K,N", FEW)
@pytest.mark.parametrize("shift", [0, 8])
@pytest.mark.parametrize("name,save", [("silu", False), ("relu", True)])
def test_gated_few_tokens(T, K, N, shift, name, save):
    x = normal(T, T * K + shift)[shift:].view(T, K)
    w = normal(K + N, 2 * N * K + shift, std=K ** -0.5)[shift:].view(2 * N, K)
    around = torch.full((T + 2, N), 7.0, device="cuda", dtype=BF)
    got = moe.gated_ffn(x, w, act=name, out=around[1:T + 1], save=save)
    ref, z, bound, ez = R.gated(x, w, name)
    R.check(around[1:T + 1], ref, bound, "h")
    assert bool((around[0] == 7).all()) and bool((around[T + 1] == 7).all())
    if save:
        R.check(got[1], z, ez, "gu")


@pytest.mark.parametrize("T", [3, 11, 20])
def test_few_tokens_keep_bad_rows_apart(T):
    x, w = normal(1, T, 1000), normal(2, 520, 1000, std=0.03)
    y = moe.linear(x, w)
    w[77, 999] = float("nan")
    x[2, 0] = float("inf")
    bad = moe.linear(x, w)
    assert bool(bad[:, 77].isnan().all()) and not bool(bad[2].isfinite().any())
    rows = torch.arange(T, device="cuda") != 2
    cols = torch.arange(520, device="cuda") != 77
    assert torch.equal(bad[rows][:, cols], y[rows][:, cols])
