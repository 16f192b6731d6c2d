"""What the dense operators of a mixture-of-experts block cost, as calls a program makes.

Three operators surround the routed experts in such a block: the residual addition with the
root-mean-square norm ahead of the router (its output optionally in e4m3 codes with 1x128 scales,
the form FP8 experts take), the gated projection of a shared expert that every token passes, and
the projection back with bias, activation and the residual (the routed experts' sum) in its
epilogue. Each comes as an inference call and as a training step (forward and backward).

``listed()`` and ``draw(rng)`` give cases, ``prepare(case, seed)`` what a program has in hand,
``run(state)`` one pass, ``work(case)`` the bytes and operations it cannot do without and
``exact(case, seed)`` the result in 64 bits. ``own`` selects the library's kernels; without it
``run`` computes the plain form in 32 bits with elementary torch operations.
"""
import math

import torch

own = False

EPS = 1e-6
E4M3_MAX = 448.0
GROUP = 128


def listed():
    return [
        # one token of a decode step: the latency of the norm itself
        {"name": "norm_one_token", "op": "rms_norm", "T": 1, "H": 2048, "residual": True, "quantize": False, "train": False},
        # a prompt of the prefill-shaped layer
        {"name": "norm_prompt", "op": "rms_norm", "T": 8192, "H": 2048, "residual": True, "quantize": False, "train": False},
        # the large FP8 layer's batch: bf16 for the router, e4m3 codes and scales for the experts
        {"name": "norm_e4m3", "op": "rms_norm", "T": 4096, "H": 7168, "residual": True, "quantize": True, "train": False},
        # a training step of a ragged batch: forward and backward
        {"name": "norm_train", "op": "rms_norm", "T": 4099, "H": 4096, "residual": True, "quantize": False, "train": True},
        # one token through the shared expert of the decode-shaped layer
        {"name": "gated_one_token", "op": "gated_ffn", "T": 1, "H": 2048, "I": 1408, "act": "silu", "train": False},
        # a decode batch through the large layer's shared expert
        {"name": "gated_decode", "op": "gated_ffn", "T": 16, "H": 7168, "I": 2048, "act": "silu", "train": False},
        # a ragged batch between decode and prompt, sizes that fill no tile
        {"name": "gated_ragged", "op": "gated_ffn", "T": 333, "H": 2040, "I": 1000, "act": "gelu", "train": False},
        # a long prompt through the widest layer's gated projection
        {"name": "gated_prompt", "op": "gated_ffn", "T": 4096, "H": 4096, "I": 14336, "act": "silu", "train": False},
        # a training step of the decode-shaped layer's shared expert
        {"name": "gated_train", "op": "gated_ffn", "T": 4096, "H": 2048, "I": 1408, "act": "silu", "train": True},
        # a decode batch projected back and added to the routed experts' sum
        {"name": "linear_decode", "op": "linear", "T": 16, "K": 2048, "N": 7168, "bias": False, "act": "none", "residual": True, "train": False},
        # a prompt projected back and added to the routed experts' sum
        {"name": "linear_prompt", "op": "linear", "T": 8192, "K": 1408, "N": 2048, "bias": True, "act": "none", "residual": True, "train": False},
        # a training step of an ungated projection with bias and activation, sizes that fill no tile
        {"name": "linear_train", "op": "linear", "T": 2050, "K": 2048, "N": 4104, "bias": True, "act": "gelu", "residual": True, "train": True},
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi):
    return max(8, _spread(rng, lo, hi) // 8 * 8)


def draw(rng):
    op = rng.choice(["rms_norm", "gated_ffn", "linear"])
    train = rng.random() < 0.4
    if op == "rms_norm":
        quantize = not train and rng.random() < 0.4
        H = GROUP * max(1, _spread(rng, 128, 8192) // GROUP) if quantize else _size(rng, 64, 8192)
        return {"op": op, "T": _spread(rng, 1, 8192), "H": H, "residual": rng.random() < 0.7, "quantize": quantize, "train": train}
    T = _spread(rng, 1, 8192)
    a, b = _size(rng, 64, 8192), _size(rng, 64, 8192)
    while T * a * b > 4096 * 4096 * 4096:
        T, a, b = max(1, T // 2), max(8, a // 16 * 8), b
    if op == "gated_ffn":
        return {"op": op, "T": T, "H": a, "I": b, "act": rng.choice(["silu", "gelu", "relu"]), "train": train}
    return {"op": op, "T": T, "K": a, "N": b, "bias": rng.random() < 0.5, "act": rng.choice(["none", "silu", "gelu", "relu"]),
            "residual": rng.random() < 0.5, "train": train}


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * (seed % 1000003) + 17)

    def normal(*shape, std=1.0, mean=0.0):
        return torch.randn(shape, generator=g, device="cuda").mul_(std).add_(mean).to(torch.bfloat16)

    s = {"case": case}
    T = case["T"]
    if case["op"] == "rms_norm":
        H = case["H"]
        s["x"] = normal(T, H)
        s["residual"] = normal(T, H, std=2.0) if case["residual"] else None
        s["weight"] = normal(H, std=0.1, mean=1.0)
        if case["train"]:
            s["dy"] = normal(T, H, std=0.1)
            s["dresidual"] = normal(T, H, std=0.1) if case["residual"] else None
    elif case["op"] == "gated_ffn":
        H, I = case["H"], case["I"]
        s["x"] = normal(T, H)
        s["w"] = normal(2 * I, H, std=1.0 / math.sqrt(H))
        if case["train"]:
            s["dh"] = normal(T, I, std=0.1)
    else:
        K, N = case["K"], case["N"]
        s["x"] = normal(T, K)
        s["w"] = normal(N, K, std=1.0 / math.sqrt(K))
        s["bias"] = normal(N, std=0.5) if case["bias"] else None
        s["residual"] = normal(T, N) if case["residual"] else None
        if case["train"]:
            s["dy"] = normal(T, N, std=0.1)
    return s


# ---- the library's calls ----------------------------------------------------

def _own_rms_norm(s, c):
    import mixture_experts_routed_moe_b200 as moe

    if not c["train"]:
        n = moe.rms_norm(s["x"], s["weight"], residual=s["residual"], eps=EPS, quantize=c["quantize"])
        return {"y": n.y, "residual": n.residual if c["residual"] else None, "codes": n.codes, "scales": n.scales}
    n = moe.rms_norm(s["x"], s["weight"], residual=s["residual"], eps=EPS, rstd=True)
    dx, dw = moe.rms_norm_backward(s["dy"], n.residual, s["weight"], n.rstd, dresidual=s["dresidual"])
    return {"y": n.y, "residual": n.residual if c["residual"] else None, "dx": dx, "dw": dw}


def _own_gated_ffn(s, c):
    import mixture_experts_routed_moe_b200 as moe

    if not c["train"]:
        return {"h": moe.gated_ffn(s["x"], s["w"], act=c["act"])}
    h, gu = moe.gated_ffn(s["x"], s["w"], act=c["act"], save=True)
    dx, dw = moe.gated_ffn_backward(s["dh"], s["x"], s["w"], gu, act=c["act"])
    return {"h": h, "dx": dx, "dw": dw}


def _own_linear(s, c):
    import mixture_experts_routed_moe_b200 as moe

    if not c["train"]:
        return {"y": moe.linear(s["x"], s["w"], bias=s["bias"], act=c["act"], residual=s["residual"])}
    y, z = moe.linear(s["x"], s["w"], bias=s["bias"], act=c["act"], residual=s["residual"], save=True)
    dx, dw, db = moe.linear_backward(s["dy"], s["x"], s["w"], z, act=c["act"], bias=c["bias"])
    return {"y": y, "dx": dx, "dw": dw, "db": db}


# ---- the plain form: elementary operations in 32 bits, rounded once ---------

def _act(name, z):
    """The activation and its derivative."""
    if name == "silu":
        p = 1 / (1 + torch.exp(-z))
        return z * p, p * (1 + z * (1 - p))
    if name == "gelu":
        p = 0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
        return z * p, p + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    if name == "relu":
        m = (z > 0).to(z.dtype)
        return z * m, m
    return z, torch.ones_like(z)


def _plain_rms_norm(s, c):
    x, w = s["x"], s["weight"].float()
    # the norm is that of the residual stream's value, which is held in bf16
    r = (x.float() + s["residual"].float()).to(x.dtype) if c["residual"] else x
    v = r.float()
    rstd = torch.rsqrt((v * v).mean(1, keepdim=True) + EPS)
    xh = v * rstd
    y = xh * w
    out = {"y": y.to(x.dtype), "residual": r if c["residual"] else None}
    if c["train"]:
        dy = s["dy"].float()
        t = dy * w
        dx = rstd * (t - xh * (t * xh).mean(1, keepdim=True))
        if c["residual"]:
            dx = dx + s["dresidual"].float()
        out["dx"], out["dw"] = dx.to(x.dtype), (dy * xh).double().sum(0).to(x.dtype)
        return out
    codes = scales = None
    if c["quantize"]:
        yg = y.view(c["T"], c["H"] // GROUP, GROUP)
        a = yg.abs().amax(2, keepdim=True)
        sc = torch.where(a > 0, a / E4M3_MAX, torch.ones_like(a))
        codes = (yg / sc).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(c["T"], c["H"])
        scales = sc.squeeze(2)
    out["codes"], out["scales"] = codes, scales
    return out


def _plain_gated_ffn(s, c):
    x, w, I = s["x"].float(), s["w"].float(), c["I"]
    gu = x @ w.t()
    g, u = gu[:, :I], gu[:, I:]
    a, d = _act(c["act"], g)
    h = (a * u).to(s["x"].dtype)
    if not c["train"]:
        return {"h": h}
    dh = s["dh"].float()
    dgu = torch.cat([dh * u * d, dh * a], 1)
    return {"h": h, "dx": (dgu @ w).to(h.dtype), "dw": (dgu.t() @ x).to(h.dtype)}


def _plain_linear(s, c):
    x, w = s["x"].float(), s["w"].float()
    z = x @ w.t()
    if c["bias"]:
        z = z + s["bias"].float()
    y, d = _act(c["act"], z)
    if c["residual"]:
        y = y + s["residual"].float()
    y = y.to(s["x"].dtype)
    if not c["train"]:
        return {"y": y}
    dz = s["dy"].float() * d
    return {"y": y, "dx": (dz @ w).to(y.dtype), "dw": (dz.t() @ x).to(y.dtype),
            "db": dz.double().sum(0).to(y.dtype) if c["bias"] else None}


def run(state):
    c = state["case"]
    if own:
        return {"rms_norm": _own_rms_norm, "gated_ffn": _own_gated_ffn, "linear": _own_linear}[c["op"]](state, c)
    return {"rms_norm": _plain_rms_norm, "gated_ffn": _plain_gated_ffn, "linear": _plain_linear}[c["op"]](state, c)


def work(case):
    T = case["T"]
    if case["op"] == "rms_norm":
        n, H = T * case["H"], case["H"]
        res = 2 if case["residual"] else 0
        if case["train"]:
            # in: x, residual, dy, the gradient at the residual, weight; out: y, residual, dx, dw
            return {"bytes": n * (2 + res + 2 + res + 2 + res + 2) + 4 * H, "flops": 14 * n}
        q = n + 4 * n // GROUP if case["quantize"] else 0
        return {"bytes": n * (2 + res + 2 + res) + q + 2 * H, "flops": 5 * n}
    if case["op"] == "gated_ffn":
        H, I = case["H"], case["I"]
        fwd = {"bytes": 2 * (T * H + 2 * I * H + T * I), "flops": 4 * T * H * I}
        if not case["train"]:
            return fwd
        return {"bytes": fwd["bytes"] + 2 * (T * I + T * H + 2 * I * H), "flops": 12 * T * H * I}
    K, N = case["K"], case["N"]
    b = 2 * N if case["bias"] else 0
    fwd = {"bytes": 2 * (T * K + N * K + T * N) + b + (2 * T * N if case["residual"] else 0), "flops": 2 * T * K * N}
    if not case["train"]:
        return fwd
    return {"bytes": fwd["bytes"] + 2 * (T * N + T * K + N * K) + b, "flops": 6 * T * K * N}


# ---- the definition in 64 bits ----------------------------------------------

def _exact_gate(name, z):
    """(f(z), f'(z)) of the activation, from its definition."""
    if name == "silu":
        sig = torch.sigmoid(z)
        return z * sig, sig + z * sig * torch.sigmoid(-z)
    if name == "gelu":
        phi = torch.special.ndtr(z)
        return z * phi, phi + z * torch.exp(-z.square() / 2) / math.sqrt(2 * math.pi)
    if name == "relu":
        return z.clamp(min=0), (z > 0).double()
    return z, torch.ones_like(z)


def exact(case, seed):
    s = {k: v.double() if isinstance(v, torch.Tensor) else v for k, v in prepare(case, seed).items()}
    if case["op"] == "rms_norm":
        v = s["x"]
        if case["residual"]:
            v = (v + s["residual"]).to(torch.bfloat16).double()
        H = case["H"]
        inv = 1 / torch.sqrt(torch.linalg.vector_norm(v, dim=1, keepdim=True).square() / H + EPS)
        y = v * s["weight"] * inv
        out = {"y": y, "residual": v if case["residual"] else None}
        if case["train"]:
            # y_i = w_i v_i r, r = (|v|^2/H + eps)^(-1/2): dv_j = r w_j dy_j - r^3 v_j / H * sum_i dy_i w_i v_i
            dot = torch.einsum("th,h,th->t", s["dy"], s["weight"], v)[:, None]
            dv = inv * s["weight"] * s["dy"] - inv**3 * v * dot / H
            if case["residual"]:
                dv = dv + s["dresidual"]
            out["dx"], out["dw"] = dv, torch.einsum("th,th,t->h", s["dy"], v, inv[:, 0])
            return out
        out["codes"] = out["scales"] = None
        if case["quantize"]:
            blocks = y.reshape(-1, GROUP)
            top = blocks.abs().max(dim=1).values
            unit = torch.where(top == 0, 1.0, top / E4M3_MAX)
            out["codes"] = (blocks / unit[:, None]).reshape(y.shape)
            out["scales"] = unit.reshape(case["T"], H // GROUP)
        return out
    x, w = s["x"], s["w"]
    if case["op"] == "gated_ffn":
        I = case["I"]
        wg, wu = w[:I], w[I:]
        g, u = torch.einsum("th,ih->ti", x, wg), torch.einsum("th,ih->ti", x, wu)
        f, df = _exact_gate(case["act"], g)
        out = {"h": f * u}
        if case["train"]:
            dg, du = s["dh"] * u * df, s["dh"] * f
            out["dx"] = torch.einsum("ti,ih->th", dg, wg) + torch.einsum("ti,ih->th", du, wu)
            out["dw"] = torch.cat([torch.einsum("ti,th->ih", dg, x), torch.einsum("ti,th->ih", du, x)])
        return out
    z = torch.einsum("tk,nk->tn", x, w)
    if case["bias"]:
        z = z + s["bias"]
    f, df = _exact_gate(case["act"], z)
    out = {"y": f + s["residual"] if case["residual"] else f}
    if case["train"]:
        dz = s["dy"] * df
        out["dx"] = torch.einsum("tn,nk->tk", dz, w)
        out["dw"] = torch.einsum("tn,tk->nk", dz, x)
        out["db"] = dz.sum(0) if case["bias"] else None
    return out
