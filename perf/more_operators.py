"""More operators of a transformer block, as workloads beside perf/operators.py: what each is
called with, what it computes in plain torch, and what it has to move and compute.

Operators (all on row-major activations, one row per token):
  layer_norm            h = x + residual; y = (h - mean) / sqrt(var + eps) * weight + bias, in x's
                        type or in 8 bits (e4m3, one scale a row)
  layer_norm_backward   the gradients of x (and of the residual, which is the same), weight, bias
  linear with int8      act(a b scale_a scale_b + bias) + residual on 8-bit integers with a scale
                        for each token and each output channel; the tokens either come in 8 bits
                        or are quantised in front of it
  pack8                 an activation kept in 8 bits: integers with one power of two for each 32
                        neighbours of a row
  checkpointed layer    a linear layer's forward and backward pass with what is kept in between
                        (its input, its value before the activation) in that form
`own` selects between the plain forms (elementary torch in 32 bits) and the package's kernels.
"""
import math

import torch

own = False

EPS = 1e-5
E4M3_MAX = 448.0
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
# exponents of the smallest scale of a checkpoint: with it, integers up to 127 are f16 (bf16) values
LOWEST = {"bf16": -120, "f16": -24}
ACTS = ("relu", "gelu", "gelu_tanh", "silu")


def listed():
    return [
        # one token of a served model: the norm before an 8-bit projection, where latency counts
        {"name": "layer_norm8_one_token", "op": "ln", "rows": 1, "dim": 4096, "type": "bf16",
         "eight": True},
        # a training step's norm, or a long prompt's, at the largest width
        {"name": "layer_norm_train", "op": "ln", "rows": 8192, "dim": 8192, "type": "bf16",
         "eight": False},
        # its backward pass in a training step
        {"name": "layer_norm_backward", "op": "ln_bwd", "rows": 8192, "dim": 4096, "type": "bf16"},
        # a small one with odd sizes: rows that start at any 2-byte address
        {"name": "layer_norm_backward_odd", "op": "ln_bwd", "rows": 1023, "dim": 1021,
         "type": "f16"},
        # one token through an 8-bit up-projection: the weights are read once, nothing else counts
        {"name": "int8_one_token", "op": "int8", "m": 1, "n": 16384, "k": 4096, "type": "bf16",
         "act": "gelu_tanh", "bias": True, "residual": False, "quantize": False},
        # odd sizes in every direction: an output projection of 16-bit activations
        {"name": "int8_odd", "op": "int8", "m": 4095, "n": 4097, "k": 4093, "type": "f16",
         "act": "none", "bias": True, "residual": True, "quantize": True},
        # a prompt through an 8-bit projection
        {"name": "int8_prompt", "op": "int8", "m": 8192, "n": 8192, "k": 8192, "type": "bf16",
         "act": "silu", "bias": True, "residual": False, "quantize": False},
        # the activations of a small training step
        {"name": "pack8_small", "op": "pack8", "rows": 512, "dim": 512, "type": "f16"},
        # those of a large one; the last block of a row is not whole
        {"name": "pack8_large", "op": "pack8", "rows": 8192, "dim": 8190, "type": "bf16"},
        # a small layer's training step
        {"name": "step8_small", "op": "step8", "m": 1024, "n": 768, "k": 128, "type": "f16",
         "act": "silu", "a_act": "none", "bias": True},
        # an up-projection's training step
        {"name": "step8_up", "op": "step8", "m": 4096, "n": 4096, "k": 4096, "type": "bf16",
         "act": "gelu_tanh", "a_act": "none", "bias": True},
        # a down-projection's, which keeps the value before the activation that it reads; odd sizes
        {"name": "step8_down_odd", "op": "step8", "m": 2047, "n": 1025, "k": 4097, "type": "bf16",
         "act": "none", "a_act": "gelu_tanh", "bias": True},
    ]


def _size(rng, lo, hi):
    """A size spread over the logarithm of [lo, hi]: as it falls, or rounded to 8 or 64."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    r = rng.choice((1, 8, 64))
    return max(lo, min(hi, n // r * r if n >= r else n))


def draw(rng):
    op = rng.choice(("ln", "ln_bwd", "int8", "int8", "pack8", "step8", "step8"))
    case = {"op": op, "type": rng.choice(("bf16", "f16"))}
    if op in ("ln", "ln_bwd", "pack8"):
        case.update(rows=_size(rng, 1, 8192), dim=_size(rng, 16, 8192))
        if op == "ln":
            case["eight"] = rng.random() < 0.5
        return case
    top = 4096 if op == "step8" else 8192
    case.update(m=_size(rng, 1, top), n=_size(rng, 16, top), k=_size(rng, 16, top),
                bias=rng.random() < 0.5)
    if op == "int8":
        case.update(act=rng.choice(("none",) + ACTS), residual=rng.random() < 0.5,
                    quantize=rng.random() < 0.5)
    else:   # an up- or a down-projection
        up = rng.random() < 0.6
        # relu's slope jumps where an integer of the checkpoint turns from 0 to 1: which side a sum
        # in 32 bits falls on says nothing about the kernels
        case.update(act=rng.choice(ACTS[1:]) if up else "none",
                    a_act="none" if up else rng.choice(ACTS))
    return case


# ---- inputs ----------------------------------------------------------------------------------

def _normal(gen, shape, std, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).mul_(std).to(dtype)


def _stream(gen, rows, dim, dtype):
    """A residual stream: about N(0, 1), with a few channels that are much larger and rows that
    are not centred."""
    big = 1.0 + 15.0 * (torch.rand(dim, generator=gen, device="cuda") < 0.004).float()
    v = torch.randn((rows, dim), generator=gen, device="cuda") * big
    return (v + 0.3 * torch.randn((rows, 1), generator=gen, device="cuda")).to(dtype)


def _int8_rows(v):
    """Rows of v in 8-bit integers and one scale a row, as an export of weights gives; rows start
    16 bytes apart or a multiple of it."""
    amax = v.abs().amax(1)
    scale = torch.where(amax > 0, amax / 127.0, torch.ones_like(amax))
    q = torch.zeros((v.shape[0], -(-v.shape[1] // 16) * 16), dtype=torch.int8, device="cuda")
    q = q[:, :v.shape[1]]
    q.copy_(torch.round(v / scale[:, None]).to(torch.int8))
    return q, scale


def _blocks(v):
    """v (rows, dim) with each row as blocks of 32, zeros after its end."""
    rows, dim = v.shape
    out = v.new_zeros((rows, -(-dim // 32) * 32))
    out[:, :dim] = v
    return out.view(rows, -1, 32)


def _pack(v, lowest):
    """(integers, scales) of v in 32 bits: the largest of each 32 neighbours lies in [64, 128)
    scales, and at most 127 are stored."""
    b = _blocks(v)
    top = b.abs().amax(2)
    e = torch.where(top > 0, torch.frexp(top).exponent - 7, lowest).clamp(min=lowest)
    scale = torch.ldexp(torch.ones_like(b[:, :, 0]), e)
    q = torch.round(b / scale[:, :, None]).clamp(-127, 127)
    return q.view(v.shape[0], -1)[:, :v.shape[1]], scale


def _unpack(q, scale):
    return (_blocks(q.float()) * scale.float()[:, :, None]).view(q.shape[0], -1)[:, :q.shape[1]]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, dt = case["op"], TYPES[case["type"]]
    s = dict(case)
    if op in ("ln", "ln_bwd"):
        shape = (case["rows"], case["dim"])
        s["weight"] = (1.0 + 0.2 * torch.randn(case["dim"], generator=gen, device="cuda")).to(dt)
        if op == "ln":
            s["x"] = _normal(gen, shape, 0.3, dt)
            s["res"] = _stream(gen, *shape, dt)
            s["bias_v"] = _normal(gen, (case["dim"],), 0.1, dt)
            return s
        s["h"] = _stream(gen, *shape, dt)
        h = s["h"].float()
        s["mean"] = h.mean(1)
        s["rstd"] = ((h - s["mean"][:, None]).square().mean(1) + EPS).rsqrt()
        s["dy"] = _normal(gen, shape, 0.02, dt)
        s["dh"] = _normal(gen, shape, 0.02, dt)
        return s
    if op == "pack8":
        s["x"] = _stream(gen, case["rows"], case["dim"], dt)
        return s
    m, n, k = case["m"], case["n"], case["k"]
    std = 1.0 / math.sqrt(k)
    s["bias_v"] = _normal(gen, (n,), 0.1, dt) if case["bias"] else None
    if op == "int8":
        a = torch.randn((m, k), generator=gen, device="cuda")
        if case["quantize"]:
            s["a"] = a.to(dt)
        else:
            s["a"], s["scale_a"] = _int8_rows(a)
        w, s["scale_b"] = _int8_rows(torch.randn((n, k), generator=gen, device="cuda") * std)
        s["b"] = w.t()
        if case["residual"]:
            s["res"] = _stream(gen, m, n, dt)
        return s
    z = _normal(gen, (m, k), 1.0, dt)
    s["a"] = z if case["a_act"] == "none" else _act(z.float(), case["a_act"]).to(dt)
    if case["a_act"] != "none":   # kept by the layer that made it
        q, scale = _pack(z.float(), LOWEST[case["type"]])
        s["z"] = torch.zeros((m, -(-k // 16) * 16), dtype=torch.int8, device="cuda")[:, :k]
        s["z"].copy_(q)
        s["z_scale"] = scale.to(torch.float8_e8m0fnu)
    s["b"] = _normal(gen, (n, k), std, dt).t()
    s["dc"] = _normal(gen, (m, n), 0.02, dt)
    return s


# ---- one pass --------------------------------------------------------------------------------

def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import dense_gemm_f16f32_amd as g
    op = s["op"]
    if op == "ln":
        if s["eight"]:
            r = g.layer_norm(s["x"], s["weight"], s["bias_v"], s["res"], eps=EPS,
                             out_dtype=torch.float8_e4m3fn)
            return {"y": r.y, "scale": r.scale, "h": r.h}
        r = g.layer_norm(s["x"], s["weight"], s["bias_v"], s["res"], eps=EPS, with_stats=True)
        return {"y": r.y, "h": r.h, "mean": r.mean, "rstd": r.rstd}
    if op == "ln_bwd":
        dx, dweight, dbias = g.layer_norm_backward(s["dy"], s["h"], s["weight"], s["mean"],
                                                   s["rstd"], dh=s["dh"])
        return {"dx": dx, "dweight": dweight, "dbias": dbias}
    if op == "int8":
        a, scale_a = s["a"], s.get("scale_a")
        if s["quantize"]:
            a, scale_a = g.quantize_rows(a)
        return g.linear(a, s["b"], s["bias_v"], s.get("res"), activation=s["act"],
                        scale_a=scale_a, scale_b=s["scale_b"], out_dtype=TYPES[s["type"]])
    if op == "pack8":
        p = g.pack8(s["x"])
        return {"values": p.values, "scale": p.scale}
    if s["act"] != "none":
        out, pre = g.linear(s["a"], s["b"], s["bias_v"], activation=s["act"], pack_pre=True)
    else:
        out, pre = g.linear(s["a"], s["b"], s["bias_v"]), None
    kept = g.pack8(s["a"]) if s["a_act"] == "none" else g.Packed8(s["z"], s["z_scale"])
    da, db, dbias = g.linear_backward(s["dc"], kept, s["b"], pre, activation=s["act"],
                                      a_activation=s["a_act"], bias_grad=s["bias"])
    return {"out": out, "da": da, "db": db, "dbias": dbias}


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
    if op == "ln":
        h = s["x"].float() + s["res"].float()
        mean = h.mean(1, keepdim=True)
        c = h - mean
        rstd = 1 / torch.sqrt((c * c).mean(1, keepdim=True) + EPS)
        y = c * rstd * s["weight"].float() + s["bias_v"].float()
        if not s["eight"]:
            return {"y": y.to(dt), "h": h.to(dt), "mean": mean[:, 0], "rstd": rstd[:, 0]}
        amax = y.abs().amax(1, keepdim=True)
        scale = torch.where(amax > 0, amax / E4M3_MAX, torch.ones_like(amax))
        return {"y": (y / scale).to(torch.float8_e4m3fn), "scale": scale[:, 0], "h": h.to(dt)}
    if op == "ln_bwd":
        dy, rstd = s["dy"].float(), s["rstd"][:, None]
        xh = (s["h"].float() - s["mean"][:, None]) * rstd
        gw = dy * s["weight"].float()
        dx = rstd * (gw - gw.mean(1, keepdim=True) - xh * (gw * xh).mean(1, keepdim=True))
        return {"dx": (dx + s["dh"].float()).to(dt), "dweight": (dy * xh).sum(0).to(dt),
                "dbias": dy.sum(0).to(dt)}
    if op == "pack8":
        q, scale = _pack(s["x"].float(), LOWEST[s["type"]])
        return {"values": q.to(torch.int8), "scale": scale.to(torch.float8_e8m0fnu)}
    b = s["b"].float()
    if op == "int8":
        a = s["a"].float()
        if s["quantize"]:
            amax = a.abs().amax(1)
            # (torch divides by a number with its rounded reciprocal)
            scale_a = torch.where(amax > 0, amax / torch.full_like(amax, 127),
                                  torch.ones_like(amax))
            a = torch.round(a / scale_a[:, None])
        else:
            scale_a = s["scale_a"]
        v = (a @ b) * scale_a[:, None] * s["scale_b"][None, :]
        if s["bias_v"] is not None:
            v = v + s["bias_v"].float()
        out = _act(v, s["act"])
        return (out + s["res"].float() if "res" in s else out).to(dt)
    a, dpre = s["a"].float(), s["dc"].float()
    v = a @ b
    if s["bias_v"] is not None:
        v = v + s["bias_v"].float()
    if s["act"] != "none":
        dpre = dpre * _act_slope(_unpack(*_pack(v, LOWEST[s["type"]])), s["act"])
    if s["a_act"] == "none":
        kept = _unpack(*_pack(a, LOWEST[s["type"]]))
    else:
        kept = _act(_unpack(s["z"], s["z_scale"]), s["a_act"])
    return {"out": _act(v, s["act"]).to(dt), "da": (dpre @ b.t()).to(dt),
            "db": (kept.t() @ dpre).to(dt), "dbias": dpre.sum(0).to(dt) if s["bias"] else None}


# ---- the definition in 64 bits ---------------------------------------------------------------

def _phi(v):
    """The normal distribution's cumulative function."""
    return torch.special.erfc(v / -math.sqrt(2.0)) / 2


def _value_and_slope(v, act):
    """An activation and its derivative."""
    if act == "none":
        return v, torch.ones_like(v)
    if act == "relu":
        return torch.relu(v), torch.heaviside(v, torch.zeros((), dtype=v.dtype, device=v.device))
    if act == "gelu":
        p, density = _phi(v), torch.exp(-v.square() / 2) / math.sqrt(2 * math.pi)
        return v * p, p + v * density
    if act == "gelu_tanh":   # v sigmoid(2 u), u = c (v + 0.044715 v^3)
        c = math.sqrt(2 / math.pi)
        p = torch.sigmoid(2 * c * (v + 0.044715 * v ** 3))
        return v * p, p + v * p * (1 - p) * 2 * c * (1 + 0.134145 * v ** 2)
    p = torch.sigmoid(v)
    return v * p, p + v * p * (1 - p)


def _kept(v, lowest):
    """v as a checkpoint gives it back, block after block of 32 columns, and the integers and
    scales."""
    back, whole, scales = torch.empty_like(v), torch.empty_like(v), []
    for c in range(0, v.shape[1], 32):
        x = v[:, c:c + 32]
        top = torch.linalg.vector_norm(x, ord=math.inf, dim=1)
        step = torch.floor(torch.log2(top)).sub(6).clamp(min=lowest).exp2().unsqueeze(1)
        whole[:, c:c + 32] = torch.minimum(torch.maximum(torch.round(x / step), step.new_tensor(-127)),
                                           step.new_tensor(127))
        back[:, c:c + 32] = whole[:, c:c + 32] * step
        scales.append(step)
    return back, whole, torch.cat(scales, 1)


def exact(case, seed):
    s = prepare(case, seed)
    op, low = case["op"], LOWEST[case["type"]]
    d = {name: t.to(torch.float64) for name, t in s.items()
         if isinstance(t, torch.Tensor) and t.dtype != torch.float8_e8m0fnu}
    if op == "ln":
        h = d["x"] + d["res"]
        mean = torch.sum(h, 1) / case["dim"]
        var = torch.linalg.vector_norm(h - mean.unsqueeze(1), dim=1).square() / case["dim"]
        inv = torch.rsqrt(var + EPS)
        y = torch.einsum("ij,i,j->ij", h - mean.unsqueeze(1), inv, d["weight"]) + d["bias_v"]
        if not case["eight"]:
            return {"y": y, "h": h, "mean": mean, "rstd": inv}
        scale = torch.linalg.vector_norm(y, ord=math.inf, dim=1) / E4M3_MAX
        scale[scale == 0] = 1.0
        # e4m3: 3 bits after the leading one, steps of 2^-9 below 2^-6
        q = y / scale[:, None]
        step = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3)
        return {"y": torch.round(q / step) * step, "scale": scale, "h": h}
    if op == "ln_bwd":
        n, r = case["dim"], d["rstd"].unsqueeze(1)
        xh = (d["h"] - d["mean"].unsqueeze(1)) * r
        gw = torch.einsum("ij,j->ij", d["dy"], d["weight"])
        along = torch.einsum("ij,ij->i", gw, xh).unsqueeze(1)
        dx = d["dh"] + r / n * (n * gw - torch.sum(gw, 1, keepdim=True) - xh * along)
        return {"dx": dx, "dweight": torch.einsum("ij,ij->j", d["dy"], xh),
                "dbias": torch.einsum("ij->j", d["dy"])}
    if op == "pack8":
        _, whole, scale = _kept(d["x"], low)
        return {"values": whole.to(torch.int8), "scale": scale}
    b = d["b"].contiguous()
    if op == "int8":
        a = d["a"]
        if case["quantize"]:   # the scale is a 32-bit number, and the integers go by it
            top = torch.linalg.vector_norm(s["a"].float(), ord=math.inf, dim=1)
            unit = torch.where(top == 0, torch.ones_like(top), (top.to(torch.float64) / 127).float())
            unit = unit.to(torch.float64)
            a = torch.round(a / unit.unsqueeze(1)) * unit.unsqueeze(1)
        else:
            a = a * d["scale_a"].unsqueeze(1)
        v = torch.mm(a, b * d["scale_b"].unsqueeze(0))
        if "bias_v" in d:
            v += d["bias_v"]
        out = _value_and_slope(v, case["act"])[0]
        return out + d["res"] if "res" in d else out
    v = torch.mm(d["a"], b)
    if "bias_v" in d:
        v += d["bias_v"]
    dpre = d["dc"]
    if case["act"] != "none":
        dpre = dpre * _value_and_slope(_kept(v, low)[0], case["act"])[1]
    if case["a_act"] == "none":
        kept = _kept(d["a"], low)[0]
    else:
        wide = torch.repeat_interleave(s["z_scale"].float().to(torch.float64), 32, dim=1)
        kept = _value_and_slope(d["z"] * wide[:, :case["k"]], case["a_act"])[0]
    return {"out": _value_and_slope(v, case["act"])[0],
            "da": torch.mm(dpre, b.t().contiguous()), "db": torch.mm(kept.t().contiguous(), dpre),
            "dbias": torch.sum(dpre, 0) if case["bias"] else None}


# ---- what a pass cannot do without -------------------------------------------------------------

def work(case):
    op = case["op"]
    if op in ("ln", "ln_bwd", "pack8"):
        r, d = case["rows"], case["dim"]
        n = r * d
        if op == "pack8":     # x in; an integer a value and a byte a block out
            return {"bytes": 3 * n + r * -(-d // 32), "flops": 4 * n}
        if op == "ln_bwd":    # dy, h, dh, mean, rstd, weight in; dx, dweight, dbias out
            return {"bytes": 8 * n + 8 * r + 6 * d, "flops": 15 * n}
        if case["eight"]:     # x, residual, weight, bias in; h, y, scale out
            return {"bytes": 7 * n + 4 * r + 4 * d, "flops": 12 * n}
        return {"bytes": 8 * n + 8 * r + 4 * d, "flops": 9 * n}
    m, n, k = case["m"], case["n"], case["k"]
    bias = 2 * n if case["bias"] else 0
    if op == "int8":
        return {"bytes": m * k * (2 if case["quantize"] else 1) + n * k + 4 * (m + n) + bias
                + 2 * m * n * (2 if case["residual"] else 1), "flops": 2.0 * m * n * k}
    # a, b, bias, dc in (and the kept value where it is not a's); out, da, db, dbias out
    kept = m * k + m * -(-k // 32) if case["a_act"] != "none" else 0
    return {"bytes": 4 * (m * k + k * n + m * n) + 2 * bias + kept, "flops": 6.0 * m * n * k}
