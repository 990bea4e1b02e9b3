"""The transformer-block operators beside the dense product, as workloads: what each is called
with, what it computes in plain torch, and what it has to move and compute.

Operators (all on row-major activations, one row per token):
  rms_norm            h = x + residual; y = h / sqrt(mean(h^2) + eps) * weight, y in x's type or
                      in 8 bits (e4m3, one scale a row)
  rms_norm_backward   the gradients of x (and of the residual, which is the same) and weight
  linear              act(a b + bias) + residual, with 16-bit operands, or with 8-bit operands
                      and their scales; optionally the value before the activation as well
  linear_backward     the gradients of a, b and bias
`own` selects between the plain forms (elementary torch in 32 bits) and the package's kernels.
"""
import math

import torch

own = False

EPS = 1e-5
E4M3_MAX = 448.0
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # one token of a served model: the norm before a projection, where latency counts
        {"name": "norm8_one_token", "op": "norm8", "rows": 1, "dim": 4096, "type": "bf16"},
        # a long prompt (or a batch of them) at the largest width
        {"name": "norm8_prompt", "op": "norm8", "rows": 8192, "dim": 8192, "type": "bf16"},
        # a training step's norm, with odd sizes: rows that start at any 2-byte address
        {"name": "norm_train_odd", "op": "norm", "rows": 4095, "dim": 4093, "type": "f16"},
        # the same norm's backward pass in a training step
        {"name": "norm_backward", "op": "norm_bwd", "rows": 8192, "dim": 4096, "type": "bf16"},
        # one token through an up-projection: the weights are read once, nothing else counts
        {"name": "linear_one_token", "op": "linear", "m": 1, "n": 16384, "k": 4096,
         "type": "bf16", "w": "nk", "act": "gelu_tanh", "bias": True, "residual": False,
         "pre": False},
        # a small layer
        {"name": "linear_512", "op": "linear", "m": 512, "n": 512, "k": 512, "type": "f16",
         "w": "kn", "act": "gelu", "bias": True, "residual": True, "pre": False},
        # odd sizes in every direction: an output projection with its residual
        {"name": "linear_odd", "op": "linear", "m": 4095, "n": 4097, "k": 4093, "type": "f16",
         "w": "kn", "act": "none", "bias": True, "residual": True, "pre": False},
        # a training step's up-projection, which keeps what its backward pass needs
        {"name": "linear_train", "op": "linear", "m": 8192, "n": 8192, "k": 8192,
         "type": "bf16", "w": "nk", "act": "gelu_tanh", "bias": True, "residual": False,
         "pre": True},
        # its backward pass
        {"name": "linear_backward", "op": "linear_bwd", "m": 4096, "n": 4096, "k": 4096,
         "type": "bf16", "w": "nk", "act": "gelu_tanh", "bias": True},
        # a small layer's backward pass
        {"name": "linear_backward_small", "op": "linear_bwd", "m": 1024, "n": 768, "k": 128,
         "type": "f16", "w": "kn", "act": "silu", "bias": True},
        # a few requests' tokens through an 8-bit projection with its residual
        {"name": "linear8_few_tokens", "op": "linear8", "m": 16, "n": 8192, "k": 8192,
         "type": "bf16", "act": "none", "bias": False, "residual": True},
        # a prompt through it
        {"name": "linear8_prompt", "op": "linear8", "m": 8192, "n": 8192, "k": 8192,
         "type": "bf16", "act": "silu", "bias": True, "residual": False},
    ]


def _size(rng, lo, hi):
    """A size spread over the logarithm of [lo, hi]: as it falls, or rounded to 8 or 64."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    r = rng.choice((1, 8, 64))
    return max(lo, min(hi, n // r * r if n >= r else n))


def draw(rng):
    op = rng.choice(("norm8", "norm", "norm_bwd", "linear", "linear", "linear_bwd", "linear8",
                     "linear8"))
    case = {"op": op, "type": rng.choice(("bf16", "f16"))}
    if op.startswith("norm"):
        case.update(rows=_size(rng, 1, 8192), dim=_size(rng, 64, 8192))
        return case
    top = 4096 if op == "linear_bwd" else 8192
    case.update(m=_size(rng, 1, top), n=_size(rng, 16, top), k=_size(rng, 16, top),
                act=rng.choice(("none", "relu", "gelu", "gelu_tanh", "silu")),
                bias=rng.random() < 0.5)
    if op != "linear8":
        case["w"] = rng.choice(("nk", "kn"))
    if op != "linear_bwd":
        case["residual"] = rng.random() < 0.5
    if op == "linear":
        case["pre"] = rng.random() < 0.3
    return case


# ---- inputs ----------------------------------------------------------------------------------

def _normal(gen, shape, std, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).mul_(std).to(dtype)


def _stream(gen, rows, dim, dtype):
    """A residual stream: about N(0, 1), with a few channels that are much larger."""
    big = 1.0 + 15.0 * (torch.rand(dim, generator=gen, device="cuda") < 0.004).float()
    return (torch.randn((rows, dim), generator=gen, device="cuda") * big).to(dtype)


def _rows16(rows, dim, dtype):
    """rows x dim whose rows start 16 elements apart or a multiple of it."""
    return torch.zeros((rows, -(-dim // 16) * 16), dtype=dtype, device="cuda")[:, :dim]


def _e4m3_rows(v):
    """Rows of v in 8 bits and one scale a row, as the norm (or an export of weights) gives."""
    amax = v.abs().amax(1)
    scale = torch.where(amax > 0, amax / E4M3_MAX, torch.ones_like(amax))
    q = _rows16(v.shape[0], v.shape[1], torch.float8_e4m3fn)
    q.copy_((v / scale[:, None]).to(torch.float8_e4m3fn))
    return q, scale


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, dt = case["op"], TYPES[case["type"]]
    s = dict(case)
    if op in ("norm8", "norm"):
        s["x"] = _normal(gen, (case["rows"], case["dim"]), 0.3, dt)
        s["res"] = _stream(gen, case["rows"], case["dim"], dt)
        s["weight"] = (1.0 + 0.2 * torch.randn(case["dim"], generator=gen, device="cuda")).to(dt)
        return s
    if op == "norm_bwd":
        s["h"] = _stream(gen, case["rows"], case["dim"], dt)
        s["weight"] = (1.0 + 0.2 * torch.randn(case["dim"], generator=gen, device="cuda")).to(dt)
        s["rstd"] = (s["h"].float().square().mean(1) + EPS).rsqrt()
        s["dy"] = _normal(gen, (case["rows"], case["dim"]), 0.02, dt)
        s["dh"] = _normal(gen, (case["rows"], case["dim"]), 0.02, dt)
        return s
    m, n, k = case["m"], case["n"], case["k"]
    std = 1.0 / math.sqrt(k)
    s["bias_v"] = _normal(gen, (n,), 0.1, dt) if case["bias"] else None
    if op == "linear8":
        s["a"], s["scale_a"] = _e4m3_rows(torch.randn((m, k), generator=gen, device="cuda"))
        w, s["scale_b"] = _e4m3_rows(torch.randn((n, k), generator=gen, device="cuda") * std)
        s["b"] = w.t()
    else:
        s["a"] = _normal(gen, (m, k), 1.0, dt)
        w = _normal(gen, (n, k) if case["w"] == "nk" else (k, n), std, dt)
        s["b"] = w.t() if case["w"] == "nk" else w
    if case.get("residual"):
        s["res"] = _stream(gen, m, n, dt)
    if op == "linear_bwd":
        s["dc"] = _normal(gen, (m, n), 0.02, dt)
        s["pre_v"] = _normal(gen, (m, n), 1.0, dt) if case["act"] != "none" else None
    return s


# ---- one pass --------------------------------------------------------------------------------

def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import dense_gemm_f16f32_amd as g
    op = s["op"]
    if op == "norm8":
        r = g.rms_norm(s["x"], s["weight"], s["res"], eps=EPS, out_dtype=torch.float8_e4m3fn)
        return {"y": r.y, "scale": r.scale, "h": r.h}
    if op == "norm":
        r = g.rms_norm(s["x"], s["weight"], s["res"], eps=EPS, with_rstd=True)
        return {"y": r.y, "h": r.h, "rstd": r.rstd}
    if op == "norm_bwd":
        dx, dweight = g.rms_norm_backward(s["dy"], s["h"], s["weight"], s["rstd"], dh=s["dh"])
        return {"dx": dx, "dweight": dweight}
    if op == "linear_bwd":
        da, db, dbias = g.linear_backward(s["dc"], s["a"], s["b"], s["pre_v"],
                                          activation=s["act"], bias_grad=s["bias"])
        return {"da": da, "db": db, "dbias": dbias}
    if op == "linear8":
        return g.linear(s["a"], s["b"], s["bias_v"], s.get("res"), activation=s["act"],
                        scale_a=s["scale_a"], scale_b=s["scale_b"], out_dtype=TYPES[s["type"]])
    if s["pre"]:
        out, pre = g.linear(s["a"], s["b"], s["bias_v"], s.get("res"), activation=s["act"],
                            with_pre=True)
        return {"out": out, "pre": pre}
    return g.linear(s["a"], s["b"], s["bias_v"], s.get("res"), activation=s["act"])


def _act(v, act):
    if act == "relu":
        return v.clamp(min=0)
    if act == "gelu":
        return 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
    if act == "silu":
        return v / (1 + torch.exp(-v))
    return v


def _act_slope(v, act):
    if act == "relu":
        return (v > 0).to(v.dtype)
    if act == "gelu":
        return (0.5 * (1 + torch.erf(v * math.sqrt(0.5)))
                + v * torch.exp(-0.5 * v * v) / math.sqrt(2 * math.pi))
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (v + 0.044715 * v * v * v))
        return 0.5 * (1 + t) + 0.5 * v * (1 - t * t) * c * (1 + 3 * 0.044715 * v * v)
    if act == "silu":
        p = 1 / (1 + torch.exp(-v))
        return p * (1 + v * (1 - p))
    return torch.ones_like(v)


def _plain(s):
    op, dt = s["op"], TYPES[s["type"]]
    if op in ("norm8", "norm"):
        h = s["x"].float() + s["res"].float()
        rstd = 1 / torch.sqrt((h * h).mean(1, keepdim=True) + EPS)
        y = h * rstd * s["weight"].float()
        if op == "norm":
            return {"y": y.to(dt), "h": h.to(dt), "rstd": rstd[:, 0]}
        amax = y.abs().amax(1, keepdim=True)
        scale = torch.where(amax > 0, amax / E4M3_MAX, torch.ones_like(amax))
        return {"y": (y / scale).to(torch.float8_e4m3fn), "scale": scale[:, 0], "h": h.to(dt)}
    if op == "norm_bwd":
        dy, xh = s["dy"].float(), s["h"].float() * s["rstd"][:, None]
        gw = dy * s["weight"].float()
        dx = s["rstd"][:, None] * (gw - xh * (gw * xh).mean(1, keepdim=True)) + s["dh"].float()
        return {"dx": dx.to(dt), "dweight": (dy * xh).sum(0).to(dt)}
    a, b = s["a"].float(), s["b"].float()
    if op == "linear_bwd":
        dpre = s["dc"].float()
        if s["act"] != "none":
            dpre = dpre * _act_slope(s["pre_v"].float(), s["act"])
        return {"da": (dpre @ b.t()).to(dt), "db": (a.t() @ dpre).to(dt),
                "dbias": dpre.sum(0).to(dt) if s["bias"] else None}
    v = a @ b
    if op == "linear8":
        v = v * s["scale_a"][:, None] * s["scale_b"][None, :]
    if s["bias_v"] is not None:
        v = v + s["bias_v"].float()
    out = _act(v, s["act"])
    if "res" in s:
        out = out + s["res"].float()
    return {"out": out.to(dt), "pre": v.to(dt)} if s.get("pre") else out.to(dt)


# ---- the definition in 64 bits ---------------------------------------------------------------

def _phi(v):
    """The normal distribution's cumulative function."""
    return torch.special.erfc(v / -math.sqrt(2.0)) / 2


def exact(case, seed):
    s = prepare(case, seed)
    op, act = case["op"], case.get("act")
    d = {name: t.to(torch.float64) for name, t in s.items() if isinstance(t, torch.Tensor)}
    if op in ("norm8", "norm"):
        h = d["x"] + d["res"]
        inv = torch.rsqrt(torch.linalg.vector_norm(h, dim=1).square() / case["dim"] + EPS)
        y = torch.einsum("ij,i,j->ij", h, inv, d["weight"])
        if op == "norm":
            return {"y": y, "h": h, "rstd": inv}
        scale = torch.linalg.vector_norm(y, ord=math.inf, dim=1) / E4M3_MAX
        scale[scale == 0] = 1.0
        # e4m3: 3 bits after the leading one, steps of 2^-9 below 2^-6
        q = y / scale[:, None]
        step = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3)
        return {"y": torch.round(q / step) * step, "scale": scale, "h": h}
    if op == "norm_bwd":
        r = d["rstd"].unsqueeze(1)
        gw = d["dy"] * d["weight"]
        dot = (gw * d["h"]).sum(1, keepdim=True)
        dx = d["dh"] + r * gw - r ** 3 * d["h"] * dot / case["dim"]
        return {"dx": dx, "dweight": torch.einsum("ij,ij,i->j", d["dy"], d["h"], d["rstd"])}
    c = math.sqrt(2 / math.pi)
    if op == "linear_bwd":
        dpre = d["dc"]
        if act != "none":
            v = d["pre_v"]
            if act == "relu":
                slope = torch.heaviside(v, torch.zeros((), dtype=v.dtype, device=v.device))
            elif act == "gelu":
                slope = _phi(v) + v * torch.exp(-v.square() / 2) / math.sqrt(2 * math.pi)
            elif act == "gelu_tanh":
                # gelu_tanh(v) = v sigmoid(2 u), u = c (v + 0.044715 v^3)
                p = torch.sigmoid(2 * c * (v + 0.044715 * v ** 3))
                slope = p + v * p * (1 - p) * 2 * c * (1 + 0.134145 * v ** 2)
            else:
                p = torch.sigmoid(v)
                slope = p + v * p * (1 - p)
            dpre = dpre * slope
        return {"da": torch.mm(dpre, d["b"].t().contiguous()),
                "db": torch.mm(d["a"].t().contiguous(), dpre),
                "dbias": torch.sum(dpre, 0) if case["bias"] else None}
    a, b = d["a"], d["b"].contiguous()
    if op == "linear8":
        a, b = a * d["scale_a"].unsqueeze(1), b * d["scale_b"].unsqueeze(0)
    v = torch.mm(a, b)
    if "bias_v" in d:
        v += d["bias_v"]
    if act == "relu":
        out = torch.maximum(v, torch.zeros_like(v))
    elif act == "gelu":
        out = v * _phi(v)
    elif act == "gelu_tanh":
        out = v * torch.sigmoid(2 * c * (v + 0.044715 * v ** 3))
    elif act == "silu":
        out = v * torch.sigmoid(v)
    else:
        out = v
    if "res" in d:
        out = out + d["res"]
    return {"out": out, "pre": v} if case.get("pre") else out


# ---- what a pass cannot do without -------------------------------------------------------------

def work(case):
    op = case["op"]
    if op.startswith("norm"):
        n, r, d = case["rows"] * case["dim"], case["rows"], case["dim"]
        if op == "norm8":     # x, residual in; h, y, scale out
            return {"bytes": 7 * n + 4 * r + 2 * d, "flops": 8 * n}
        if op == "norm":      # x, residual in; h, y, rstd out
            return {"bytes": 8 * n + 4 * r + 2 * d, "flops": 5 * n}
        return {"bytes": 8 * n + 4 * r + 4 * d, "flops": 11 * n}   # dy, h, dh in; dx out
    m, n, k = case["m"], case["n"], case["k"]
    bias = 2 * n if case["bias"] else 0
    if op == "linear8":
        return {"bytes": m * k + n * k + 4 * (m + n) + bias
                + 2 * m * n * (2 if case["residual"] else 1), "flops": 2.0 * m * n * k}
    if op == "linear":
        return {"bytes": 2 * (m * k + k * n) + bias
                + 2 * m * n * (1 + case["residual"] + case["pre"]), "flops": 2.0 * m * n * k}
    return {"bytes": 2 * (m * n * (2 if case["act"] != "none" else 1) + 2 * (m * k + k * n))
            + bias, "flops": 4.0 * m * n * k}
