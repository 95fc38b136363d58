"""Cases for the 8-bit products with one scale for each block of 128, their
quantiser, the linear layer's training step built from the two, and the
mixture-of-experts layer for a few tokens.

``run`` computes a case in plain torch operations in 32 bits, or, where ``own``
is true, through the package's entry points.
"""
import math

import torch

own = False

F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
F8_MAX = {"e4m3": 448.0, "e5m2": 57344.0}
REAL = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
TINY = 2.0 ** -100  # floor of a block's largest magnitude


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one decoded token through one projection: latency
        dict(name="product_one_token", op="product", batch=1, M=1, N=4096, K=4096, type="e4m3", out="bf16",
             b_rows=128),
        # a decode batch against a wide projection: the weights' bytes bound it
        dict(name="product_skinny", op="product", batch=1, M=64, N=16384, K=8192, type="e4m3", out="f32", b_rows=128),
        # independent ragged products, no size a multiple of a tile, both operands scaled by row
        dict(name="product_ragged_batch", op="product", batch=16, M=3001, N=2047, K=1000, type="e5m2", out="f32",
             b_rows=1),
        # prefill / large training batch: the tensor cores bound it
        dict(name="product_square", op="product", batch=1, M=8192, N=8192, K=8192, type="e4m3", out="bf16",
             b_rows=128),
        # activations of a decode batch before their product
        dict(name="quantize_decode", op="quantize", M=64, K=8192, type="e4m3", x="bf16", rows=1, both=False),
        # activations kept for the backward pass: both orders in one pass
        dict(name="quantize_both", op="quantize", M=8192, K=8192, type="e4m3", x="bf16", rows=1, both=True),
        # forward, input gradient and weight gradient of one linear layer
        dict(name="linear_step", op="linear", M=4096, N=4096, K=4096, x="bf16"),
        dict(name="linear_step_ragged", op="linear", M=3001, N=2047, K=1000, x="f16"),
        # one decoded token through a layer of 64 experts
        dict(name="experts_one_token", op="experts", T=1, E=64, topk=8, H=2048, I=1024, x="bf16", w="bf16",
             masked=False, renorm=True),
        # a decode batch that reaches nearly every expert, weights in 8 bits
        dict(name="experts_batch_8bit", op="experts", T=64, E=64, topk=8, H=2048, I=1024, x="bf16", w="e4m3",
             masked=False, renorm=True),
        # odd sizes, experts masked out, a token with no expert at all
        dict(name="experts_masked_odd", op="experts", T=7, E=10, topk=3, H=1000, I=520, x="f16", w="f16",
             masked=True, renorm=False),
        # few large experts
        dict(name="experts_wide", op="experts", T=16, E=8, topk=2, H=4096, I=8192, x="bf16", w="bf16", masked=False,
             renorm=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["product", "product", "quantize", "linear", "experts", "experts"])
    if op == "product":
        while True:
            c = dict(op=op, batch=rng.choice([1, 1, 1, 2, 5]), M=_log(rng, 1, 8192), N=_log(rng, 100, 16384),
                     K=_log(rng, 100, 8192), type=rng.choice(["e4m3", "e4m3", "e5m2"]),
                     out=rng.choice(["bf16", "f16", "f32"]), b_rows=rng.choice([128, 128, 1]))
            if c["batch"] * c["M"] * c["N"] * c["K"] <= 8192 ** 3:
                return c
    if op == "quantize":
        return dict(op=op, M=_log(rng, 1, 8192), K=_log(rng, 100, 8192), type=rng.choice(["e4m3", "e5m2"]),
                    x=rng.choice(["bf16", "f16", "f32"]), rows=rng.choice([1, 1, 128]), both=rng.random() < 0.5)
    if op == "linear":
        return dict(op=op, M=_log(rng, 100, 4096), N=_log(rng, 200, 4096), K=_log(rng, 200, 4096),
                    x=rng.choice(["bf16", "f16"]))
    x = rng.choice(["bf16", "bf16", "f16"])
    experts = rng.choice([8, 16, 33, 64])
    return dict(op=op, T=_log(rng, 1, 64), E=experts, topk=rng.choice([1, 2, 4, 8]), H=8 * _log(rng, 32, 256),
                I=8 * _log(rng, 16, 128), x=x, w=rng.choice([x, "e4m3"]), masked=rng.random() < 0.4,
                renorm=rng.random() < 0.6)


# ---------------------------------------------------------------- inputs
def _blocks(n):
    return (n + 127) // 128


def _pad(x, rows, cols):
    out = x.new_zeros(*x.shape[:-2], rows, cols)
    out[..., :x.shape[-2], :x.shape[-1]] = x
    return out


def _amax(x, rows):
    """Largest magnitude of each (rows x 128) block of the last two dimensions."""
    m, k = x.shape[-2:]
    p = _pad(x.abs(), _blocks(m) * 128 if rows == 128 else m, _blocks(k) * 128)
    p = p.reshape(*x.shape[:-2], -1, rows, _blocks(k), 128)
    return p.amax(dim=(-3, -1)).clamp(min=TINY)


def _spread(s, rows, m, k):
    """A scale for every element from one for every block."""
    return s.repeat_interleave(rows, -2)[..., :m, :].repeat_interleave(128, -1)[..., :k]


def _quantize(x, rows, kind):
    """Codes and scales, in 32 bits."""
    m, k = x.shape[-2:]
    x = x.float()
    a = _amax(x, rows)
    factor = a.reciprocal() * F8_MAX[kind]
    return (x * _spread(factor, rows, m, k)).to(F8[kind]), a * (1 / F8_MAX[kind])


def _pitched(q):
    """The same codes with rows on 16-byte boundaries, as the quantiser leaves them."""
    out = torch.zeros(*q.shape[:-1], (q.shape[-1] + 15) // 16 * 16, dtype=torch.uint8, device=q.device)
    out = out.view(q.dtype)[..., :q.shape[-1]]
    out.copy_(q)
    return out


def _normal(g, *shape, scale=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def _activations(g, m, k, dtype):
    """Activations with a few columns that are much larger than the rest."""
    x = torch.randn(m, k, generator=g, device="cuda")
    x *= torch.where(torch.rand(k, generator=g, device="cuda") < 0.01, 20.0, 1.0)
    return x.to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c = dict(case)
    if c["op"] == "product":
        a = torch.stack([_activations(g, c["M"], c["K"], torch.bfloat16) for _ in range(c["batch"])])
        b = _normal(g, c["batch"], c["N"], c["K"], scale=0.02)
        qa, sa = _quantize(a, 1, c["type"])
        qb, sb = _quantize(b, c["b_rows"], c["type"])
        # one scale for a row and block: stored with the rows adjacent, as the quantiser leaves them
        sa = sa.transpose(-1, -2).contiguous().transpose(-1, -2)
        if c["b_rows"] == 1:
            sb = sb.transpose(-1, -2).contiguous().transpose(-1, -2)
        s = dict(a=_pitched(qa), sa=sa, b=_pitched(qb), sb=sb)
        if c["batch"] == 1:
            s = {k: v[0] for k, v in s.items()}
    elif c["op"] == "quantize":
        s = dict(x=_activations(g, c["M"], c["K"], REAL[c["x"]]))
    elif c["op"] == "linear":
        w = _normal(g, c["N"], c["K"], scale=c["K"] ** -0.5)
        q, sw = _quantize(w, 128, "e4m3")
        # the weights in both orders, laid out once after each update
        s = dict(x=_activations(g, c["M"], c["K"], REAL[c["x"]]),
                 dy=_normal(g, c["M"], c["N"], scale=0.01, dtype=REAL[c["x"]]),
                 w=_pitched(q), sw=sw, wt=_pitched(q.t()), swt=sw.t().contiguous())
    else:
        x = _normal(g, c["T"], c["H"], dtype=REAL[c["x"]])
        logits = _normal(g, c["T"], c["E"], scale=2.0)
        if c["masked"]:
            off = torch.rand(c["T"], c["E"], generator=g, device="cuda") < 0.4
            off[-1] |= c["T"] > 1  # a token that no expert takes
            logits = logits.masked_fill(off, float("-inf"))
        s = dict(x=x, logits=logits, s13=None, s2=None)
        for name, rows, cols in (("13", 2 * c["I"], c["H"]), ("2", c["H"], c["I"])):
            w = _normal(g, c["E"], rows, cols, scale=cols ** -0.5, dtype=torch.bfloat16)
            if c["w"] == "e4m3":
                q, s["s" + name] = _quantize(w, 128, "e4m3")
                s["w" + name] = _pitched(q)
            else:
                s["w" + name] = w.to(REAL[c["w"]])
    s["case"] = c
    return s


# ---------------------------------------------------------------- one pass
def _values(q, s):
    """What codes and scales stand for, in 32 bits."""
    m, k = q.shape[-2:]
    return q.float() * _spread(s, 1 if s.shape[-2] == m else 128, m, k)


def _linear_plain(s):
    x, dy = s["x"].float(), s["dy"].float()
    w = _values(s["w"], s["sw"])
    xr, xc = _values(*_quantize(x, 1, "e4m3")), _values(*_quantize(x.t(), 1, "e4m3"))
    dr, dc = _values(*_quantize(dy, 1, "e4m3")), _values(*_quantize(dy.t(), 1, "e4m3"))
    t = s["x"].dtype
    return (xr @ w.t()).to(t), (dr @ w).to(t), dc @ xc.t()


def _route(logits, topk, renorm):
    """Chosen experts of each token, best first and ties to the lowest index,
    and their weights; a masked expert (-inf) has weight zero."""
    top, idx = torch.sort(logits, dim=-1, descending=True, stable=True)
    top, idx = top[:, :topk], idx[:, :topk]
    best = top[:, :1]
    e = torch.where(torch.isinf(top), 0.0, torch.exp(top - best))
    every = e if renorm else torch.where(torch.isinf(logits), 0.0, torch.exp(logits - best))
    total = every.sum(-1, keepdim=True)
    return idx, torch.where(total > 0, e / total, 0.0)


def _experts_plain(s):
    c, x = s["case"], s["x"].float()
    idx, p = _route(s["logits"], min(c["topk"], c["E"]), c["renorm"])
    w13, w2, s13, s2 = s["w13"], s["w2"], s["s13"], s["s2"]
    if idx.numel() < c["E"]:  # few tokens: their experts' weights only
        pick = idx.flatten()
        w13, w2 = w13.view(torch.uint8)[pick].view(w13.dtype), w2.view(torch.uint8)[pick].view(w2.dtype)
        s13, s2 = (None, None) if s13 is None else (s13[pick], s2[pick])
    w13 = w13.float() if s13 is None else _values(w13, s13)
    w2 = w2.float() if s2 is None else _values(w2, s2)
    if idx.numel() < c["E"]:
        rows = x.repeat_interleave(idx.shape[1], 0)[:, None]                # (T k, 1, H)
        g, u = torch.matmul(rows, w13.transpose(1, 2)).chunk(2, -1)
        y = torch.matmul(g * torch.sigmoid(g) * u, w2.transpose(1, 2))      # (T k, 1, H)
        y = y.view(*idx.shape, -1) * p[..., None]
        y = torch.where(p[..., None] > 0, y, 0.0).sum(1)
    else:
        g, u = torch.matmul(x, w13.transpose(1, 2)).chunk(2, -1)            # (E, T, I)
        y = torch.matmul(g * torch.sigmoid(g) * u, w2.transpose(1, 2))      # (E, T, H)
        full = torch.zeros_like(s["logits"]).scatter_(1, idx, p)            # (T, E)
        y = torch.where(full.t()[..., None] > 0, y * full.t()[..., None], 0.0).sum(0)
    return y.to(s["x"].dtype)


def run(state):
    s, c = state, state["case"]
    if own:
        import dense_fp16_tensor_gemm_gb300 as gnt
        if c["op"] == "product":
            return gnt.gemm_nt_block128_tensors(s["a"], s["sa"], s["b"], s["sb"], out_dtype=REAL[c["out"]])
        if c["op"] == "quantize":
            return gnt.quantize_block128(s["x"], F8[c["type"]], block_rows=c["rows"], transposed=c["both"])
        if c["op"] == "linear":
            y, saved = gnt.linear_block128(s["x"], s["w"], s["sw"])
            dx, dw = gnt.linear_block128_backward(s["dy"], saved, s["wt"], s["swt"])
            return y, dx, dw
        return gnt.moe_few_tokens(s["x"], s["logits"], s["w13"], s["w2"], topk=min(c["topk"], c["E"]), S13=s["s13"],
                                  S2=s["s2"], renormalize=c["renorm"])
    if c["op"] == "product":
        out = torch.matmul(_values(s["a"], s["sa"]), _values(s["b"], s["sb"]).transpose(-1, -2))
        return out.to(REAL[c["out"]])
    if c["op"] == "quantize":
        q, t = _quantize(s["x"], c["rows"], c["type"])
        if not c["both"]:
            return q, t
        return q, t, *_quantize(s["x"].t(), c["rows"], c["type"])
    if c["op"] == "linear":
        return _linear_plain(s)
    return _experts_plain(s)


# ---------------------------------------------------------------- bytes and operations
def work(case):
    c = case
    size = {"f32": 4, "f16": 2, "bf16": 2, "e4m3": 1, "e5m2": 1}

    def scales(m, k, rows):
        return 4 * (m if rows == 1 else _blocks(m)) * _blocks(k)

    if c["op"] == "product":
        m, n, k = c["M"], c["N"], c["K"]
        per = m * k + n * k + scales(m, k, 1) + scales(n, k, c["b_rows"]) + m * n * size[c["out"]]
        return {"bytes": c["batch"] * per, "flops": 2 * c["batch"] * m * n * k}
    if c["op"] == "quantize":
        m, k = c["M"], c["K"]
        total = m * k * (size[c["x"]] + 1 + c["both"]) + scales(m, k, c["rows"])
        if c["both"]:
            total += scales(k, m, c["rows"])
        return {"bytes": total, "flops": 4 * m * k * (1 + c["both"])}
    if c["op"] == "linear":
        m, n, k = c["M"], c["N"], c["K"]
        # x, dy, the weights (the two orders hold the same values) and their scales; y, dx, dw
        total = 2 * m * k + 2 * m * n + n * k + scales(n, k, 128) + 2 * m * n + 2 * m * k + 4 * n * k
        return {"bytes": total, "flops": 6 * m * n * k}
    t, e, k = c["T"], c["E"], min(c["topk"], c["E"])
    # experts that at least one token is expected to reach; a quarter or so of the masked choices fall away
    reach = e * (1 - (1 - k / e) ** t)
    weights = reach * 3 * c["H"] * c["I"] * size[c["w"]]
    if c["w"] == "e4m3":
        weights += reach * (scales(2 * c["I"], c["H"], 128) + scales(c["H"], c["I"], 128))
    return {"bytes": int(weights + 4 * t * e + 2 * t * c["H"] * size[c["x"]]),
            "flops": 6 * t * k * c["H"] * c["I"]}


# ---------------------------------------------------------------- 64 bits
def _codes64(x, rows, kind):
    """The quantiser's codes (a rounding that is part of its definition, from
    32-bit factors) and scales, as 64-bit values, block by block."""
    x = x.float()
    m, k = x.shape
    lim, mb = F8_MAX[kind], -(-m // rows)
    full = torch.zeros(mb * rows, -(-k // 128) * 128, device=x.device)
    full[:m, :k] = x
    tile = full.view(mb, rows, -1, 128).permute(0, 2, 1, 3)              # (row block, K block, rows, 128)
    top = torch.maximum(tile.abs().flatten(2).max(2).values, torch.tensor(TINY, device=x.device))
    factor = (1 / top) * lim
    q = (tile * factor[..., None, None]).to(F8[kind]).double()
    q = q.permute(0, 2, 1, 3).reshape(full.shape)[:m, :k]
    return q, (top * (1 / lim)).double()


def _scaled64(q, s):
    m, k = q.shape
    rows = torch.arange(m, device=q.device) // (1 if s.shape[0] == m else 128)
    cols = torch.arange(k, device=q.device) // 128
    return q.double() * s.double()[rows][:, cols]


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "product":
        if c["batch"] == 1:
            return _scaled64(s["a"], s["sa"]) @ _scaled64(s["b"], s["sb"]).t()
        return torch.stack([_scaled64(s["a"][i], s["sa"][i]) @ _scaled64(s["b"][i], s["sb"][i]).t()
                            for i in range(c["batch"])])
    if c["op"] == "quantize":
        q, t = _codes64(s["x"], c["rows"], c["type"])
        if not c["both"]:
            return q, t
        return q, t, *_codes64(s["x"].t(), c["rows"], c["type"])
    if c["op"] == "linear":
        w = _scaled64(s["w"], s["sw"])
        y = _scaled64(*_codes64(s["x"], 1, "e4m3")) @ w.t()
        dx = _scaled64(*_codes64(s["dy"], 1, "e4m3")) @ w
        dw = _scaled64(*_codes64(s["dy"].t(), 1, "e4m3")) @ _scaled64(*_codes64(s["x"].t(), 1, "e4m3")).t()
        return y, dx, dw
    logits = s["logits"].double().cpu()
    out = torch.zeros(c["T"], c["H"], dtype=torch.float64, device="cuda")
    chosen = {}
    for t in range(c["T"]):
        row = logits[t].tolist()
        order = [e for e in sorted(range(c["E"]), key=lambda e: (-row[e], e)) if row[e] > -math.inf]
        picks = order[:c["topk"]]
        norm = math.fsum(math.exp(row[e] - row[order[0]]) for e in (picks if c["renorm"] else order))
        for e in picks:
            chosen.setdefault(e, []).append((t, math.exp(row[e] - row[order[0]]) / norm))
    for e, uses in chosen.items():
        w13 = s["w13"][e].double() if s["s13"] is None else _scaled64(s["w13"][e], s["s13"][e])
        w2 = s["w2"][e].double() if s["s2"] is None else _scaled64(s["w2"][e], s["s2"][e])
        at = torch.tensor([t for t, _ in uses], device="cuda")
        p = torch.tensor([v for _, v in uses], dtype=torch.float64, device="cuda")
        g, u = (s["x"][at].double() @ w13.t()).chunk(2, -1)
        out[at] += p[:, None] * ((g / (1 + torch.exp(-g)) * u) @ w2.t())
    return out
