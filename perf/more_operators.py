"""Cases for the gated feed-forward block (both projections, the activation and
the product of the two in one call, and its backward pass) and for products with
4-bit weights that have a scale, and optionally a zero point, for each group of
a row: the quantiser, the plain product and the gated one.

``run`` computes a case in plain torch operations in 32 bits, or, where ``own``
is true, through the package's entry points.
"""
import math

import torch

own = False

REAL = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one decoded token through the block's first half: the weights' bytes bound it
        dict(name="gated_one_token", op="gated", M=1, K=4096, I=8192, x="bf16", act="silu", keep=False),
        # a decode batch
        dict(name="gated_batch", op="gated", M=64, K=2048, I=8192, x="bf16", act="gelu_tanh", keep=False),
        # a long training batch, g and u kept for the backward pass
        dict(name="gated_train", op="gated", M=8192, K=4096, I=8192, x="bf16", act="silu", keep=True),
        # the backward pass of a training batch
        dict(name="backward_train", op="backward", M=4096, K=4096, I=8192, x="bf16", act="silu"),
        # no size a multiple of a tile
        dict(name="backward_ragged", op="backward", M=3001, K=1000, I=2047, x="f16", act="gelu"),
        # a layer's weights quantised once after training; and a small layer with zero points
        dict(name="quantize_large", op="quantize", N=8192, K=8192, w="bf16", group=128, zeros=False),
        dict(name="quantize_small", op="quantize", N=1000, K=520, w="f32", group=32, zeros=True),
        # one decoded token through a projection with 4-bit weights: latency
        dict(name="w4_one_token", op="w4", M=1, N=4096, K=4096, x="bf16", group=128, zeros=False),
        # a decode batch against a wide projection
        dict(name="w4_batch", op="w4", M=64, N=16384, K=8192, x="bf16", group=128, zeros=False),
        # a prompt
        dict(name="w4_prompt", op="w4", M=2048, N=8192, K=4096, x="f16", group=64, zeros=True),
        # one decoded token through the block's first half with 4-bit weights
        dict(name="w4_gated_one_token", op="w4_gated", M=1, K=4096, I=8192, x="bf16", act="silu", group=128,
             zeros=True),
        # a few tokens, odd sizes, small groups
        dict(name="w4_gated_odd", op="w4_gated", M=7, K=1000, I=2047, x="f16", act="gelu_tanh", group=32,
             zeros=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """Mostly multiples of 8, as hidden sizes are; sometimes anything."""
    n = _log(rng, lo, hi)
    return n if rng.random() < 0.15 else max(8, n // 8 * 8)


def draw(rng):
    op = rng.choice(["gated", "gated", "backward", "quantize", "w4", "w4", "w4_gated"])
    x, act = rng.choice(["bf16", "f16"]), rng.choice(["silu", "gelu", "gelu_tanh"])
    group, zeros = rng.choice([32, 64, 128, 128]), rng.random() < 0.5
    if op == "quantize":
        return dict(op=op, N=_log(rng, 100, 16384), K=_width(rng, 100, 8192), w=rng.choice(["bf16", "f16", "f32"]),
                    group=group, zeros=zeros)
    while True:
        m = _log(rng, 1, 128) if rng.random() < 0.6 and op != "backward" else _log(rng, 16, 8192)
        k, i = _width(rng, 128, 8192), _log(rng, 128, 16384)
        if m * k * i <= 2048 * 4096 * 8192:
            break
    if op == "gated":
        return dict(op=op, M=m, K=k, I=i, x=x, act=act, keep=m > 64 and rng.random() < 0.7)
    if op == "backward":
        return dict(op=op, M=m, K=k, I=i, x=x, act=act)
    if op == "w4":
        return dict(op=op, M=m, N=i, K=k, x=x, group=group, zeros=zeros)
    return dict(op=op, M=m, K=k, I=i, x=x, act=act, group=group, zeros=zeros)


# ---------------------------------------------------------------- inputs
def _normal(g, *shape, scale=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def _activations(g, m, k, dtype):
    """Activations with a few columns that are larger than the rest."""
    x = torch.randn(m, k, generator=g, device="cuda")
    x *= torch.where(torch.rand(k, generator=g, device="cuda") < 0.01, 8.0, 1.0)
    return x.to(dtype)


def _groups(w, group):
    """The last dimension as (groups, group), the last one filled up with zeros."""
    n, k = w.shape
    full = w.new_zeros(n, -(-k // group) * group)
    full[:, :k] = w
    return full.view(n, -1, group)


def _pack(codes):
    """Two codes to a byte, the even column in the low half; rows start on 16-byte boundaries."""
    n, k = codes.shape
    even = codes.new_zeros(n, (k + 1) // 2 * 2)
    even[:, :k] = codes
    packed = even[:, 0::2] + even[:, 1::2] * 16
    out = packed.new_zeros(n, (packed.shape[1] + 15) // 16 * 16, dtype=torch.uint8)
    out = out[:, :packed.shape[1]]
    out.copy_(packed)
    return out


def _quantize(w, group, zeros, kind):
    """Codes (0 to 15, one a value), scales in 16 bits and zero points of 16- or
    32-bit weights, in 32 bits."""
    g = _groups(w.float(), group)
    if zeros:
        lo, hi = g.amin(2).clamp(max=0.0), g.amax(2).clamp(min=0.0)
        s = ((hi - lo) * (1 / 15)).to(kind)
    else:
        s = (g.abs().amax(2) * (1 / 7)).to(kind)
    sf = s.float()
    inv = torch.where(sf > 0, 1 / sf, 0.0)
    q = torch.round(g * inv[..., None])
    if zeros:
        z = torch.round(-lo * inv).clamp(0, 15)
        q = (q + z[..., None]).clamp(0, 15)
    else:
        z = None
        q = q.clamp(-8, 7) + 8
    q = q.reshape(w.shape[0], -1)[:, :w.shape[1]]
    return q.to(torch.uint8), s, None if z is None else z.to(torch.uint8)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c = dict(case)
    if c["op"] == "quantize":
        return dict(case=c, w=_normal(g, c["N"], c["K"], scale=c["K"] ** -0.5, dtype=REAL[c["w"]]))
    t = REAL[c["x"]]
    s = dict(case=c, x=_activations(g, c["M"], c["K"], t))
    rows = c["N"] if c["op"] == "w4" else 2 * c["I"]
    w = _normal(g, rows, c["K"], scale=c["K"] ** -0.5, dtype=t)
    if c["op"] in ("gated", "backward"):
        s["w13"] = w
    else:
        codes, s["s"], s["z"] = _quantize(w, c["group"], c["zeros"], t)
        s["q"] = _pack(codes)
    if c["op"] == "backward":
        # what the forward pass kept: gate and up of each token
        s["gu"] = _normal(g, c["M"], 2 * c["I"], scale=1.3, dtype=t)
        s["dh"] = _normal(g, c["M"], c["I"], scale=0.01, dtype=t)
    return s


# ---------------------------------------------------------------- one pass
def _act(g, kind):
    if kind == "silu":
        return g * torch.sigmoid(g)
    if kind == "gelu":
        return 0.5 * g * (1 + torch.erf(g * math.sqrt(0.5)))
    return 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g)))


def _slope(g, kind):
    """The activation's derivative."""
    if kind == "silu":
        p = torch.sigmoid(g)
        return p * (1 + g * (1 - p))
    if kind == "gelu":
        return 0.5 * (1 + torch.erf(g * math.sqrt(0.5))) + g * torch.exp(-0.5 * g * g) * (2 * math.pi) ** -0.5
    a = math.sqrt(2 / math.pi)
    t = torch.tanh(a * (g + 0.044715 * g * g * g))
    return 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * a * (1 + 3 * 0.044715 * g * g)


def _values(s):
    """What codes, scales and zero points stand for, in 32 bits."""
    c, q = s["case"], s["q"]
    codes = torch.stack((q & 15, q >> 4), -1).reshape(q.shape[0], -1)[:, :c["K"]].float()
    z = torch.full_like(s["s"], 8.0, dtype=torch.float32) if s["z"] is None else s["z"].float()
    spread = [v.repeat_interleave(c["group"], 1)[:, :c["K"]] for v in (z, s["s"].float())]
    return (codes - spread[0]) * spread[1]


def run(state):
    s, c = state, state["case"]
    if own:
        import dense_fp16_tensor_gemm_gb300 as gnt
        if c["op"] == "gated":
            return gnt.gated_linear(s["x"], s["w13"], activation=c["act"], keep=c["keep"])
        if c["op"] == "backward":
            return gnt.gated_linear_backward(s["dh"], s["gu"], s["x"], s["w13"], activation=c["act"])
        if c["op"] == "quantize":
            scale = torch.bfloat16 if c["w"] == "f32" else REAL[c["w"]]
            return gnt.quantize_w4(s["w"], group=c["group"], zeros=c["zeros"], scale_dtype=scale)
        if c["op"] == "w4":
            return gnt.linear_w4(s["x"], s["q"], s["s"], s["z"], group=c["group"])
        return gnt.gated_linear_w4(s["x"], s["q"], s["s"], s["z"], group=c["group"], activation=c["act"])
    if c["op"] == "quantize":
        codes, scale, z = _quantize(s["w"], c["group"], c["zeros"], torch.bfloat16 if c["w"] == "f32" else REAL[c["w"]])
        return (_pack(codes), scale, z) if c["zeros"] else (_pack(codes), scale)
    x, t = s["x"].float(), s["x"].dtype
    if c["op"] == "backward":
        g, u = s["gu"].float().chunk(2, 1)
        dh = s["dh"].float()
        dgu = torch.cat((dh * u * _slope(g, c["act"]), dh * _act(g, c["act"])), 1)
        return (dgu @ s["w13"].float()).to(t), (dgu.t() @ x).to(t)
    w = s["w13"].float() if c["op"] == "gated" else _values(s)
    y = x @ w.t()
    if c["op"] == "w4":
        return y.to(t)
    g, u = y.chunk(2, 1)
    h = (_act(g, c["act"]) * u).to(t)
    return (h, y.to(t)) if c.get("keep") else h


# ---------------------------------------------------------------- bytes and operations
def work(case):
    c = case

    def weights(rows):
        groups = -(-c["K"] // c["group"])
        return rows * ((c["K"] + 1) // 2 + (3 if c["zeros"] else 2) * groups)

    if c["op"] == "quantize":
        return {"bytes": c["N"] * c["K"] * SIZE[c["w"]] + weights(c["N"]), "flops": 4 * c["N"] * c["K"]}
    m, k = c["M"], c["K"]
    if c["op"] == "w4":
        return {"bytes": weights(c["N"]) + 2 * m * (k + c["N"]), "flops": 2 * m * k * c["N"]}
    i = c["I"]
    if c["op"] == "w4_gated":
        return {"bytes": weights(2 * i) + 2 * m * (k + i), "flops": 4 * m * k * i}
    if c["op"] == "gated":
        return {"bytes": 2 * (m * k + 2 * i * k + m * i * (3 if c["keep"] else 1)), "flops": 4 * m * k * i}
    return {"bytes": 2 * (3 * m * i + 2 * m * k + 4 * i * k), "flops": 8 * m * k * i}


# ---------------------------------------------------------------- 64 bits
def _curve64(g, kind):
    """The activation and its derivative: g Phi(g) with Phi the logistic or the
    normal distribution function, or the latter's approximation."""
    if kind == "silu":
        phi = 1 / (1 + torch.exp(-g))
        density = phi - phi.square()
    elif kind == "gelu":
        phi = torch.special.ndtr(g)
        density = torch.exp(-g.square() / 2) / math.sqrt(2 * math.pi)
    else:
        # (1 + tanh v) / 2 is the logistic function of 2 v
        v = 2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)
        phi = 1 / (1 + torch.exp(-v))
        density = (phi - phi.square()) * 2 * math.sqrt(2 / math.pi) * (1 + 0.134145 * g.square())
    return g * phi, phi + g * density


def _weights64(s):
    c, q = s["case"], s["q"]
    out = torch.empty(q.shape[0], q.shape[1], 2, dtype=torch.float64, device=q.device)
    out[..., 0], out[..., 1] = q.remainder(16), q.div(16, rounding_mode="floor")
    out = out.view(q.shape[0], -1)[:, :c["K"]]
    of = torch.arange(c["K"], device=q.device) // c["group"]
    out = out - (8.0 if s["z"] is None else s["z"][:, of].double())
    return out * s["s"][:, of].double()


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "quantize":
        # codes and zero points are whole numbers; a scale is its quotient's rounding
        w = s["w"].double()
        parts = [w[:, j:j + c["group"]] for j in range(0, c["K"], c["group"])]
        if c["zeros"]:
            scale = [(p.max(1).values.clamp(min=0) - p.min(1).values.clamp(max=0)) / 15 for p in parts]
        else:
            scale = [torch.linalg.vector_norm(p, math.inf, dim=1) / 7 for p in parts]
        return (None, torch.stack(scale, 1), None) if c["zeros"] else (None, torch.stack(scale, 1))
    x = s["x"].double()
    if c["op"] == "backward":
        gate, up = s["gu"][:, :c["I"]].double(), s["gu"][:, c["I"]:].double()
        value, slope = _curve64(gate, c["act"])
        dh = s["dh"].double()
        dg, du = dh * up * slope, dh * value
        wg, wu = s["w13"][:c["I"]].double(), s["w13"][c["I"]:].double()
        return dg @ wg + du @ wu, torch.cat((dg.t() @ x, du.t() @ x))
    w = s["w13"].double() if c["op"] == "gated" else _weights64(s)
    if c["op"] == "w4":
        return x @ w.t()
    gate, up = x @ w[:c["I"]].t(), x @ w[c["I"]:].t()
    h = _curve64(gate, c["act"])[0] * up
    return (h, torch.cat((gate, up), 1)) if c.get("keep") else h
